"""NaN and infinity in keys and values that some of a window's positions see and
others do not: each position's output is that of its own keys alone."""
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.helpers import check_attention, scale_for, to_f64
from tests.ref64 import DTYPES, attend, gather, make_pool

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def window(rows, ctx, w, G, Hkv, bs, dtype, seed):
    kc, vc, table, _ = make_pool(rows, Hkv, 128, bs, dtype, DEV, seed)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn((len(ctx), G * Hkv, 128), generator=g).to(DTYPES[dtype]).to(DEV)
    return kc, vc, table.repeat_interleave(w, 0).contiguous(), q


def run(kc, vc, bt, q, ctx, w, ml):
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device=DEV)
    tot = torch.zeros((len(ctx) // w, kc.shape[1], ml), device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    pa.pa_decode_weights(out, q, kc, vc, bt, lens, scale_for(128), ml, tot, queries_per_row=w, d_err=err)
    torch.cuda.synchronize()
    return out, tot, int(err.item())


def put(cache, bt, row, j, dims, value, head=None):
    bs = cache.shape[2]
    hs = slice(None) if head is None else head
    cache[int(bt[row, j // bs]), hs, j % bs, dims] = value


def expect(kc, vc, bt, q, ctx, i, drop=()):
    keys = [j for j in range(ctx[i]) if j not in drop]
    K, V = gather(kc, bt[i], ctx[i])[keys], gather(vc, bt[i], ctx[i])[keys]
    return attend(q[i].cpu().double(), K, V, scale_for(128))[0]


@pytest.mark.parametrize("G,Hkv,bs,dtype,w", [(4, 2, 16, "bf16", 8), (8, 1, 64, "f16", 40), (2, 3, 32, "bf16", 9)])
def test_values_reach_only_the_positions_that_see_them(G, Hkv, bs, dtype, w):
    rows = [700, 45]
    ctx = [max(1, n - 3 * (w - 1 - i)) for n in rows for i in range(w)]
    kc, vc, bt, q = window(rows, ctx, w, G, Hkv, bs, dtype, seed=w)
    # (row, key, dimensions, value): a whole V row, some of its dimensions, infinities of both signs
    marks = [(0, rows[0] - 2, slice(None), NAN), (0, rows[0] - 8, slice(3, 7), INF), (0, 640, slice(100, 101), -INF),
             (1, rows[1] - 5, slice(0, 64), NAN)]
    for r, j, d, x in marks:
        put(vc, bt, r * w, j, d, x)
    out, tot, err = run(kc, vc, bt, q, ctx, w, max(rows))
    assert err == 0 and bool(torch.isfinite(tot).all())
    ref = torch.stack([expect(kc, vc, bt, q, ctx, i) for i in range(len(ctx))])
    got = to_f64(out)
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(torch.as_tensor(got)), torch.isnan(ref))
    inf = torch.isinf(ref)
    assert bool(inf.any()) and bool((torch.as_tensor(got)[inf] == ref[inf]).all())
    assert bool((fin.all(-1).all(-1)).any()) and bool((~fin).any())   # some see nothing of it, some do
    clean = torch.where(fin, ref, torch.zeros_like(ref))
    check_attention(torch.where(fin, torch.as_tensor(got), clean).numpy(), clean.numpy(), dtype, "outputs")


def test_beside_table_entries_out_of_the_pool():
    ctx = [100, 90, 80, 70]
    kc, vc, bt, q = window([100], ctx, 4, 4, 1, 16, "bf16", seed=3)
    put(vc, bt, 0, 95, slice(None), NAN)
    good = bt.clone()
    bt[:, 2] = 10 ** 6
    out, _, err = run(kc, vc, bt, q, ctx, 4, 100)
    assert err == pa.capi.DEVERR["block_range"]
    ref = torch.stack([expect(kc, vc, good, q, ctx, i, drop=range(32, 48)) for i in range(4)])
    assert bool(torch.isnan(out[0]).all())
    check_attention(to_f64(out[1:]), ref[1:].numpy(), "bf16", "kept keys")


def test_keys_and_the_mask():
    # a NaN key: the positions that see it are NaN throughout, the others as they were
    ctx = [60, 300, 20, 300, 0]
    kc, vc, bt, q = window([300], ctx, 5, 8, 1, 16, "f16", seed=4)
    put(kc, bt, 0, 150, slice(None), NAN)
    put(vc, bt, 0, 280, slice(None), INF)
    out, tot, err = run(kc, vc, bt, q, ctx, 5, 300)
    assert err == 0
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[3]).all()) and not bool(out[4].any())
    for i in (0, 2):
        check_attention(to_f64(out[i:i + 1]), expect(kc, vc, bt, q, ctx, i)[None].numpy(), "f16", f"position {i}")
