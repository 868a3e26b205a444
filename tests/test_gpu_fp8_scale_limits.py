"""Writing rows into a block that holds the largest scales there are: exact, as any other."""
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests import ref8
from tests.ref64 import DTYPES

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("byte", [254, 253, 247, 63])
@pytest.mark.parametrize("T", [1, 700])
def test_rows_join_a_block_of_a_given_scale(byte, T):
    Hkv, D, bs = 3, 64, 16
    g = torch.Generator().manual_seed(91)
    nb = T + 2
    kc, ks, vc, vs, _ = ref8.make_pool([nb * bs], Hkv, D, bs, DEV, 92, spare=0)
    for s in (ks, vs):
        s.view(torch.uint8)[:] = byte
    old = [x.clone() for x in (kc, ks, vc, vs)]
    # values of 2^112 to 2^120: from under half of the largest scale's smallest code on
    k, v = ((torch.randn((T, Hkv, D), generator=g) * torch.exp2(torch.randint(112, 121, (T, Hkv, D), generator=g).float()))
            .to(DTYPES["bf16"]).to(DEV) for _ in range(2))
    slots = (torch.randperm(nb, generator=g)[:T] * bs + torch.randint(1, bs, (T,), generator=g)).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_reshape_and_cache_fp8(k, v, kc, vc, ks, vs, slots, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for x, c0, s0, c, s in ((k, old[0], old[1], kc, ks), (v, old[2], old[3], vc, vs)):
        want, e = ref8.store(c0, s0, x.cpu().double(), slots.cpu(), False)
        assert torch.equal(s.cpu().view(torch.uint8).long() - 127, e)
        assert torch.equal(c.cpu().double(), want)
