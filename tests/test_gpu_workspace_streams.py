"""A call on a stream of its own that allocates its workspace itself: the memory is
not one that work still queued on the current stream uses."""
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.ref64 import make_pool

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def calls():
    lens = [900, 300, 77]
    kc, vc, old, new = make_pool(lens, 2, 128, 16, "bf16", DEV, 5, extra=[64] * 3)
    g = torch.Generator().manual_seed(6)
    q, tot = torch.randn((3, 16, 128), generator=g).bfloat16().to(DEV), torch.rand((3, 2, 900), generator=g).to(DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, t = torch.empty_like(q), torch.empty_like(tot)
    kept, nl, nt = torch.empty((3, 2, 64), dtype=torch.int32, device=DEV), torch.empty_like(n), torch.empty_like(tot)
    one, same = old[:1].repeat(3, 1).contiguous(), torch.full_like(n, 900)
    few = torch.empty_like(q[:2, :4].contiguous()), q[:2, :4].contiguous()
    pairs = torch.tensor([[int(new[0, 0]), int(new[1, 0])], [int(new[0, 1]), int(new[1, 1])]], device=DEV)
    none = torch.empty((0, 2, 128), dtype=torch.bfloat16)
    hostside = (torch.empty(q.shape, dtype=q.dtype), q.cpu(), none, none, torch.empty(0, dtype=torch.int64), old.cpu(), n.cpu())
    pq = torch.randn((8, 16, 128), generator=g).bfloat16().to(DEV)
    pout = torch.empty_like(pq)
    size = pa.pa_decode_weights_workspace_bytes
    return {
        "weights": (size(3, 16, 2, 128, 16, 900),
                    lambda s: pa.pa_decode_weights(out, q, kc, vc, old, n, 0.09, 900, tot, t, stream=s)),
        "several": (size(3, 16, 2, 128, 16, 900, 3),
                   lambda s: pa.pa_decode_weights(out, q, kc, vc, one, same, 0.09, 900, tot[:1], t[:1], queries_per_row=3,
                                                  stream=s)),
        "evict": (pa.lib().pa_evict_workspace_bytes(kc.shape[0]),
                  lambda s: pa.pa_evict(kc, vc, tot, old, n, new, nl, nt, kept, 64, 4, 16, 900, stream=s)),
        "prefix": (pa.pa_decode_common_prefix_workspace_bytes(3, 16, 2, 128, 16, 900, 3, 20),
                   lambda s: pa.pa_decode_common_prefix(out, q, kc, vc, one, same, 0.09, 900, 3, 20, stream=s)),
        "decode": (pa.pa_decode_workspace_bytes(3, 16, 2, 128, 16, 900, 64),
                   lambda s: pa.pa_decode(out, q, kc, vc, old, n, 0.09, 900, 64, stream=s)),
        "shared": (pa.pa_decode_shared_prefix_workspace_bytes(2, 4, 2, 128, 16, 900, 20),
                   lambda s: pa.pa_decode_shared_prefix(*few, kc, vc, one[:2], same[:2], 0.09, 900, 2, 20, stream=s)),
        "copies": (pa.pa_copy_blocks_workspace_bytes(2),
                   lambda s: pa.pa_copy_blocks(kc, vc, pairs, stream=s)),
        "host": (pa.capi.pa_decode_step_host_staging_bytes(3, 16, 2, 128, 16, old.shape[1], 900, 0),
                 lambda s: pa.pa_decode_step_host(*hostside, kc, vc, 0.09, 900, stream=s)),
        "mixed": (pa.lib().pa_mixed_step_workspace_bytes(1, 8, 3, 16, 2, 128, 16, 900, 0),
                  lambda s: pa.pa_mixed_step(pout, pq, old[1:2], [100], [8], out, q, old, n, kc, vc, 0.09, 900, stream=s)),
    }


@pytest.mark.parametrize("name", ["weights", "several", "evict", "prefix", "decode", "shared", "copies", "host", "mixed"])
def test_a_workspace_of_its_own_on_another_stream(name):
    size, call = calls()[name]
    side = torch.cuda.Stream()
    call(None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # freed on the current stream while a copy of it is still to run there
    mine = torch.full((size,), 7, dtype=torch.uint8, device=DEV)
    copy = torch.empty_like(mine)
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    copy.copy_(mine)
    del mine
    call(side)
    torch.cuda.synchronize()
    assert bool((copy == 7).all())
