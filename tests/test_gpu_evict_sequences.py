"""Several sequences of a block manager cut down by one pa_evict: what each keeps
is its own, whatever the pool has left and whether prompts are cached."""
import numpy as np
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.helpers import check_attention, to_f64
from tests.ref64 import attend, evict_choice, gather

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("cache", [True, False])
@pytest.mark.parametrize("spare", [0, 80])
@pytest.mark.parametrize("Hkv,bs,lens", [(2, 16, [200] * 8), (1, 8, [160, 40, 130, 64, 0, 65])])
def test_one_call_over_a_batch(cache, spare, Hkv, bs, lens):
    keep, sink, recent, D, G = 64, 4, 16, 128, 4
    blocks = sum(-(-n // bs) + -(-min(n, keep) // bs) for n in lens) + spare
    g = torch.Generator().manual_seed(bs + spare)
    kc, vc = (torch.randn((blocks, Hkv, bs, D), generator=g).bfloat16().to(DEV) for _ in range(2))
    tot = torch.rand((len(lens), Hkv, max(lens)), generator=g).to(DEV)
    bm = pa.BlockManager(blocks, bs, prefix_cache=cache)
    for s, n in enumerate(lens):
        bm.add_sequence(s, [1000 * s + j for j in range(n)])
    seqs = list(range(len(lens)))
    old = torch.as_tensor(bm.tables(seqs), device=DEV)
    rows = [(gather(kc, old[s], n), gather(vc, old[s], n)) for s, n in enumerate(lens)]
    bm.evict_sequences(seqs, keep)
    new = torch.as_tensor(bm.tables(seqs, -(-keep // bs)), device=DEV)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    nl, nt = torch.empty_like(ctx), torch.empty_like(tot)
    kept = torch.empty((len(lens), Hkv, keep), dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_evict(kc, vc, tot, old, ctx, new, nl, nt, kept, keep, sink, recent, max(lens), d_err=err)
    q = torch.randn((len(lens), Hkv * G, D), generator=g).bfloat16().to(DEV)
    out = torch.empty_like(q)
    pa.pa_decode(out, q, kc, vc, new, nl, 0.09, keep, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    ref = []
    for s, n in enumerate(lens):
        m = min(n, keep)
        assert int(nl[s]) == m == bm.seq_len(s)
        K, V = gather(kc, new[s], m), gather(vc, new[s], m)
        for h in range(Hkv):
            idx = evict_choice(tot[s, h].cpu().numpy(), n, keep, sink, recent)
            assert kept[s, h, :m].tolist() == idx
            assert torch.equal(K[:, h], rows[s][0][idx, h]) and torch.equal(V[:, h], rows[s][1][idx, h])
        ref.append(attend(q[s].cpu().double(), K, V, 0.09)[0])
    check_attention(to_f64(out), torch.stack(ref).numpy(), "bf16", "decode after it")
