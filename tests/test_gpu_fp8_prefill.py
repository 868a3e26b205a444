"""Prompt chunks over an 8-bit cache, and copies of its blocks.

The cached values enter pa_prefill_batch's kernel exactly, so its numerics apply:
products of 16-bit values in fp32, each weight rounded once to the query's type
(2^-9 of it in bf16, 2^-12 in fp16) and the output once.  With the bounds on scores and
sums of the decode's test, an output is off by at most
  half a step + A (half a step + 2 (2 (D + 8) 2^-24 size + 2^-22) + 2 n 2^-24 + 2^-20),
A the weighted mean of |v|.  In fp16 a weight below 2^-14 of the largest is subnormal and
rounded to a multiple of 2^-24, off by up to 2^-25 however small it is; the weights' sum
is at least the largest one, 1, so that adds up to 2^-25 sum |v_j|, which counts where a
key that takes nearly all of the weight has values far smaller than the others'.  (One row
of the first cases is off by 4 parts in 10^5 of its neighbours that way; rounding the exact
weights to fp16 on the CPU gives the same.)"""
import math

import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests import ref8
from tests.ref64 import DTYPES, half_step

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def make(prefixes, chunks, G, Hkv, bs, dtype, seed, **kw):
    kc, ks, vc, vs, bt = ref8.make_pool([a + b for a, b in zip(prefixes, chunks)], Hkv, 128, bs, DEV, seed, **kw)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn((sum(chunks), G * Hkv, 128), generator=g).to(DTYPES[dtype]).to(DEV)
    return dict(q=q, kc=kc, ks=ks, vc=vc, vs=vs, bt=bt, prefixes=prefixes, chunks=chunks, scale=1 / math.sqrt(128))


def attend(c, err=None, out=None, **kw):
    out = torch.full_like(c["q"], float("nan")) if out is None else out
    pa.pa_prefill_batch_fp8(out, c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["bt"], c["prefixes"], c["chunks"], c["scale"],
                            d_err=err, **kw)
    return out


def check(c, dtype, step=1, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = attend(c, err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert bool(torch.isfinite(out.float()).all())
    kv, vv = ref8.values(c["kc"], c["ks"]), ref8.values(c["vc"], c["vs"])
    at = 0
    h = half_step(dtype)
    for i, (p, n) in enumerate(zip(c["prefixes"], c["chunks"])):
        K, V = ref8.rows_of(kv, c["bt"][i], p + n), ref8.rows_of(vv, c["bt"][i], p + n)
        for r in sorted(set(range(0, n, step)) | ({n - 1} if n else set())):
            m = p + r + 1
            want, mean, size = ref8.attend_sizes(c["q"][at + r].cpu().double(), K[:m], V[:m], c["scale"])
            rel = h + 2 * (2 * (128 + 8) * 2.0 ** -24 * size + 2.0 ** -22) + 2 * m * 2.0 ** -24 + 2.0 ** -20
            bound = want.abs() * h * (1 + 2.0 ** -10) + mean * rel[:, None] + 2.0 ** -25
            if dtype == "f16":
                bound += 2.0 ** -25 * V[:m].abs().sum(0).repeat_interleave(want.shape[0] // V.shape[1], 0)
            assert bool(((out[at + r].cpu().double() - want).abs() <= bound).all()), (i, r)
        at += n
    return out


@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 2), (4, 1), (8, 1)])
@pytest.mark.parametrize("bs,dtype", [(16, "bf16"), (16, "f16"), (32, "bf16"), (64, "f16"), (128, "bf16")])
def test_chunks(G, Hkv, bs, dtype):
    c = make([0, 40, 129, 0, 700], [1, 1, 37, 0, 100], G, Hkv, bs, dtype, seed=G + bs, poison=True, spread=3.0)
    check(c, dtype, step=7)


def test_more_sequences_than_a_launch_takes():
    n = 70
    c = make([(7 * i) % 90 for i in range(n)], [(5 * i) % 12 for i in range(n)], 2, 1, 16, "bf16", seed=5, poison=True)
    check(c, "bf16", step=3)


def test_one_workspace_for_calls_of_all_sizes():
    big = make([500, 100], [300, 200], 8, 2, 16, "bf16", seed=6)
    small = make([10], [5], 8, 2, 16, "bf16", seed=7)
    ws = pa.prefill_fp8_workspace(big["q"], big["kc"], big["prefixes"], big["chunks"])
    ws.fill_(0xff)   # what it holds on entry is ignored
    a = check(big, "bf16", step=50, workspace=ws).clone()
    b = check(small, "bf16", workspace=ws).clone()
    for _ in range(3):
        assert torch.equal(attend(small, workspace=ws), b)
        got = attend(big, workspace=ws)
        torch.cuda.synchronize()
        assert bool(((got.float() - a.float()).abs() <= 2.0 ** -7 * a.float().abs() + 2.0 ** -10).all())


def test_bad_entries_are_flagged_and_other_sequences_unharmed():
    """(what the sequence itself gets is undefined, as in pa_prefill_batch)"""
    c = make([64, 30], [20, 9], 4, 1, 16, "bf16", seed=8, poison=True)
    good = check(c, "bf16").clone()
    for bad in (-3, c["kc"].shape[0]):
        c["bt"][0, 2] = bad
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = attend(c, err)
        torch.cuda.synchronize()
        assert int(err.item()) == pa.capi.DEVERR["block_range"]
        assert bool(((out[20:].float() - good[20:].float()).abs() <= 2.0 ** -7 * good[20:].float().abs() + 2.0 ** -10).all())


def test_nothing_to_do_and_refusals():
    c = make([10, 5], [0, 0], 2, 2, 16, "bf16", seed=9)
    attend(c)
    c = make([10], [6], 2, 2, 16, "bf16", seed=10)
    a = dict(out=torch.zeros_like(c["q"]), query=c["q"], k_cache=c["kc"], v_cache=c["vc"], k_scales=c["ks"], v_scales=c["vs"],
             block_tables=c["bt"], prefix_lens=[10], chunk_lens=[6], scale=0.1)
    pa.pa_prefill_batch_fp8(**a)
    for exc, kw in ((ValueError, dict(chunk_lens=[5])), (ValueError, dict(prefix_lens=[10, 3])),
                    (TypeError, dict(k_cache=c["kc"].bfloat16())), (TypeError, dict(block_tables=c["bt"].long())),
                    (pa.PAError, dict(prefix_lens=[11 + 16])), (pa.PAError, dict(prefix_lens=[-1])), (pa.PAError, dict(scale=0.0)),
                    (pa.PAError, dict(workspace=torch.zeros(512, dtype=torch.uint8, device=DEV)))):
        with pytest.raises(exc):
            pa.pa_prefill_batch_fp8(**{**a, **kw})


def test_replayed_and_on_another_stream():
    c = make([300, 20], [64, 30], 8, 2, 16, "bf16", seed=11)
    ws = pa.prefill_fp8_workspace(c["q"], c["kc"], c["prefixes"], c["chunks"])
    out = attend(c, workspace=ws).clone()
    near = lambda x: bool(((x.float() - out.float()).abs() <= 2.0 ** -7 * out.float().abs() + 2.0 ** -10).all())  # noqa: E731
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = attend(c, stream=s)
    s.synchronize()
    assert near(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attend(c, out=got, workspace=ws)
    for _ in range(2):
        got.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert near(got)


@pytest.mark.parametrize("Hkv,D,bs", [(8, 128, 16), (1, 64, 8), (5, 16, 16), (40, 128, 128)])
def test_copy_blocks(Hkv, D, bs):
    kc, ks, vc, vs, _ = ref8.make_pool([bs * 30], Hkv, D, bs, DEV, seed=12, spread=4.0)
    pairs = torch.tensor([[0, 20], [1, 21], [0, 22], [7, 25]], device=DEV)
    want = []
    for x in (kc, ks, vc, vs):
        y = x.view(torch.uint8).clone()
        y[[20, 21, 22, 25]] = y[[0, 1, 0, 7]]
        want.append(y)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_copy_blocks_fp8(kc, vc, ks, vs, pairs, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for x, y in zip((kc, ks, vc, vs), want):
        assert torch.equal(x.view(torch.uint8), y)
    # conflicting, out of the pool, onto itself: skipped, codes and scales alike
    pairs = torch.tensor([[0, 3], [1, 3], [4, 4], [2, 10 ** 6], [5, 9], [9, 11]], device=DEV)
    y = [x.view(torch.uint8).clone() for x in (kc, ks, vc, vs)]
    for x in y:
        x[11] = x[9]
    pa.pa_copy_blocks_fp8(kc, vc, ks, vs, pairs, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.capi.DEVERR["copy_pair"]
    for x, z in zip((kc, ks, vc, vs), y):
        assert torch.equal(x.view(torch.uint8), z)
    pa.pa_copy_blocks_fp8(kc, vc, ks, vs, pairs[:0])
    with pytest.raises(TypeError):
        pa.pa_copy_blocks_fp8(kc, vc, ks, vs, pairs.int())
    with pytest.raises(ValueError):
        pa.pa_copy_blocks_fp8(kc, vc, ks, vs, pairs.reshape(-1))
