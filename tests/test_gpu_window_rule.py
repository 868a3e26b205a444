"""Several positions over one cache on either side of the rule that has them attended
together: the same results from both forms, by the bounds of each."""
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.test_gpu_weights import check, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("G,w,bounds", [(4, 4, (4095, 4096)), (4, 8, (511, 512)), (2, 8, (1023, 1024)), (8, 7, (300,)),
                                        (8, 8, (300,)), (1, 16, (300,)), (4, 15, (511, 512))])
def test_both_sides_of_the_rule(G, w, bounds):
    # the rule is on the bound of the lengths: the same caches, whichever it takes
    for bound in bounds:
        c = setup([300, 5, 129], w, 2 * G, 2, 128, 16, "bf16", seed=G + w, width=bound)
        c["ml"] = bound
        check(c)


@pytest.mark.parametrize("G,w", [(8, 4), (4, 5), (2, 9)])
def test_positions_of_one_cache_have_one_table_row_in_either_form(G, w):
    c = setup([200, 90], w, 2 * G, 2, 128, 16, "f16", seed=w)
    odd = c["bt"].clone()
    odd[w + 2, 1] = odd[0, 0]
    for bound in (200, 8192):
        tot = torch.zeros((2, 2, bound), device=c["q"].device)
        for bt, want in ((c["bt"], 0), (odd, pa.capi.DEVERR["prefix"])):
            err = torch.zeros(1, dtype=torch.int32, device=c["q"].device)
            pa.pa_decode_weights(torch.empty_like(c["q"]), c["q"], c["kc"], c["vc"], bt, c["lens"], c["scale"], bound, tot,
                                 queries_per_row=w, d_err=err)
            torch.cuda.synchronize()
            assert int(err.item()) == want, (bound, want)


@pytest.mark.parametrize("G,w,L", [(4, 4, 100), (4, 4, 8192), (8, 4, 1000), (2, 8, 512), (8, 8, 512), (1, 16, 70)])
def test_a_workspace_of_the_size_that_is_asked_for_is_enough(G, w, L):
    c = setup([L, L // 2], w, 2 * G, 2, 128, 16, "bf16", seed=L)
    n = pa.pa_decode_weights_workspace_bytes(2 * w, 2 * G, 2, 128, 16, L, w)
    ws = torch.full((n + 4096,), 255, dtype=torch.uint8, device=c["q"].device)
    check(c, workspace=ws[:n])
    assert bool((ws[n:] == 255).all())
