"""pa_decode_weights' scratch where the bound of the lengths is the model's and not the
batch's: what the call allocates follows the tables."""
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.test_gpu_weights import check, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("w", [1, 4])
def test_scratch_of_a_loose_bound(w):
    rows = [100, 30, 77, 64]
    c = setup(rows, w, 16, 2, 128, 16, "bf16", seed=w, width=131072)
    c["ml"] = 131072
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = torch.empty_like(c["q"])
    pa.pa_decode_weights(out, c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["scale"], c["ml"], c["tot"].clone(),
                         queries_per_row=w)
    torch.cuda.synchronize()
    totals = c["tot"].numel() * 4
    assert torch.cuda.max_memory_allocated() - before < totals + (4 << 20)      # by the bound: 34 MB a position and row
    check(c)


def test_lengths_past_the_tables_and_past_the_totals():
    c = setup([64, 30], 1, 4, 1, 128, 16, "f16", seed=15, width=1000)
    lens = c["lens"].clone()
    lens[0] = 900                                    # within the bound, not within the table
    out, err = torch.empty_like(c["q"]), torch.zeros(1, dtype=torch.int32, device=lens.device)
    pa.pa_decode_weights(out, c["q"], c["kc"], c["vc"], c["bt"], lens, c["scale"], 1000, c["tot"].clone(), d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.capi.DEVERR["context_range"]
    with pytest.raises(pa.PAError) as e:
        pa.pa_decode_weights(out, c["q"], c["kc"], c["vc"], c["bt"], lens, c["scale"], 1001, c["tot"].clone())
    assert e.value.status == -3
