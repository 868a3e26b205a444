"""Decode over an 8-bit cache, against attention over its values in 64 bits.

Tolerance, by arithmetic.  A score in log2 units, s = scale log2(e) sum q_i k_i, is a
sum of D fp32 products of exact values: off by at most (D + 8) 2^-24 of
size = scale log2(e) sum |q_i k_i| (the tensor cores may drop what lies 2^-24 below
the largest term of a step of 32: no more than that bound again), its exponential by
2^-22 of itself more; a weight enters the sum as at least 12 bits (2^-12); the sums
over n keys are off by at most n 2^-24 of the sum of magnitudes, twice (o and l).  So
an output is off by at most
  half a step + A (2 (2 (D + 8) 2^-24 ln(2) size + 2^-22) + 2^-12 + 2 n 2^-24 + 2^-20),
A the weighted mean of |v|."""
import math

import numpy as np
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


def near(got, q, K, V, scale, dtype, n):
    out, mean, size = ref8.attend_sizes(q, K, V, scale)
    D = q.shape[1]
    rel = 2 * (2 * (D + 8) * 2.0 ** -24 * size + 2.0 ** -22) + 2.0 ** -12 + 2 * n * 2.0 ** -24 + 2.0 ** -20
    bound = out.abs() * half_step(dtype) * (1 + 2.0 ** -10) + mean * rel[:, None] + 2.0 ** -25
    err = (got.cpu().double() - out).abs()
    assert bool(torch.isfinite(got.float()).all())
    assert bool((err <= bound).all()), (float((err - bound).max()), float((err / bound).max()))


def make(lens, Hq, Hkv, D, bs, dtype, seed, qsize=1.0, **kw):
    kc, ks, vc, vs, bt = ref8.make_pool(lens, Hkv, D, bs, DEV, seed, **kw)
    g = torch.Generator().manual_seed(seed + 1)
    q = (qsize * torch.randn((len(lens), Hq, D), generator=g)).to(DTYPES[dtype]).to(DEV)
    return dict(q=q, kc=kc, ks=ks, vc=vc, vs=vs, bt=bt, lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                scale=1 / math.sqrt(D), most=max(lens))


def decode(c, err=None, out=None, **kw):
    out = torch.full_like(c["q"], float("nan")) if out is None else out
    pa.pa_decode_fp8(out, c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["bt"], c["lens"], c["scale"], c["most"], d_err=err, **kw)
    return out


def check(c, dtype, lens=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = decode(c, err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    kv, vv = ref8.values(c["kc"], c["ks"]), ref8.values(c["vc"], c["vs"])
    for i, n in enumerate(lens if lens is not None else c["lens"].tolist()):
        near(out[i], c["q"][i].cpu().double(), ref8.rows_of(kv, c["bt"][i], n), ref8.rows_of(vv, c["bt"][i], n), c["scale"],
             dtype, n)
    return out


LENS = [1, 0, 127, 128, 129, 17, 16, 300, 2, 255, 600]


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs,dtype", [(8, "bf16"), (16, "f16"), (16, "bf16"), (32, "bf16"), (64, "f16"), (128, "bf16")])
def test_decode(G, D, bs, dtype):
    c = make(LENS, 2 * G, 2, D, bs, dtype, seed=G + D + bs, poison=True)
    check(c, dtype)


@pytest.mark.parametrize("D,G", [(128, 4), (128, 8), (64, 8), (64, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lens,Hkv", [([1500, 3, 0, 257, 64, 1024], 1),      # every tile a CTA of its own
                                      ([5000, 0, 0, 129], 8),                # shares of one and of two tiles
                                      ([40] * 300 + [3000, 0] + [130] * 40, 3),   # more sequences than are held at a time
                                      ([0, 0, 0, 128, 0], 2)])
def test_shares(D, G, dtype, lens, Hkv):
    c = make(lens, G * Hkv, Hkv, D, 16, dtype, seed=3 + D + G, poison=True)
    if len(lens) > 100:  # the first and last ones, and those around the long one
        c2 = decode(c)
        kv, vv = ref8.values(c["kc"], c["ks"]), ref8.values(c["vc"], c["vs"])
        for i in (0, 1, 7, 299, 300, 301, 302, 341):
            near(c2[i], c["q"][i].cpu().double(), ref8.rows_of(kv, c["bt"][i], lens[i]), ref8.rows_of(vv, c["bt"][i], lens[i]),
                 c["scale"], dtype, lens[i])
    else:
        check(c, dtype)


def test_one_workspace_for_calls_of_all_sizes():
    """The counters that tell who merges are at zero after every call."""
    big = make([5000, 0, 3, 129, 1024], 8 * 2, 2, 128, 16, "bf16", seed=41)
    small = make([200, 700], 8 * 2, 2, 128, 16, "bf16", seed=42)
    ws = pa.decode_fp8_workspace(big["q"], 2, 16, big["most"])
    a, b = check(big, "bf16", workspace=ws).clone(), check(small, "bf16", workspace=ws).clone()
    for _ in range(5):
        assert torch.equal(decode(big, workspace=ws), a)
        assert torch.equal(decode(small, workspace=ws), b)
    torch.cuda.synchronize()
    assert not bool(ws[:4096].any())


@pytest.mark.parametrize("D,G,Hkv", [(128, 8, 1), (128, 2, 1), (64, 4, 1)])
def test_one_long_context_in_many_pieces(D, G, Hkv):
    c = make([40000], G * Hkv, Hkv, D, 64, "bf16", seed=43)
    out = check(c, "bf16")
    for _ in range(3):
        assert torch.equal(decode(c), out)   # whoever merges


def test_a_row_alone_and_in_a_batch():
    """Cut differently, the same up to fp32 sums and one rounding."""
    c = make([2500, 700, 1, 90], 8, 2, 128, 16, "bf16", seed=40)
    out = decode(c)
    for i, n in enumerate(c["lens"].tolist()):
        one = dict(c, q=c["q"][i:i + 1], bt=c["bt"][i:i + 1].contiguous(), lens=c["lens"][i:i + 1], most=n)
        assert bool(((decode(one).float() - out[i].float()).abs() <= 2.0 ** -7 * out[i].float().abs() + 2.0 ** -12).all())


@pytest.mark.parametrize("D,G", [(128, 2), (128, 8), (64, 4)])
def test_scales_far_apart(D, G):
    """Blocks of values 2^60 apart: the smaller ones keep their digits where they alone are attended."""
    lens = [400, 33, 130]
    c = make(lens, G, 1, D, 16, "bf16", seed=21, poison=True)
    t = c["bt"].long()
    vb = c["vs"].view(torch.uint8)
    vb[t[0, 3]] = 127 + 40
    vb[t[0, 7]] = 127 - 20
    vb[t[1, 0]] = 127 - 20                # the attended one of its sequence is the small one
    c["ks"].view(torch.uint8)[t[1, 1]] = 127 - 64
    vb[t[1, 1]] = 127 + 30
    vb[t[2]] = 63                         # all of them at the smallest scale
    check(c, "bf16")


@pytest.mark.parametrize("D,G", [(128, 4), (128, 8), (64, 2)])
def test_peaked_and_flat_weights(D, G):
    c = make([700, 513], G, 1, D, 16, "f16", seed=22, qsize=8.0)   # one key takes nearly everything
    check(c, "f16")
    c["q"].zero_()                                                 # every key alike
    check(c, "f16")


@pytest.mark.parametrize("D,G", [(128, 1), (128, 8), (64, 2)])
@pytest.mark.parametrize("gap", [9.0, 14.0, 18.0])
def test_many_small_weights_beside_a_large_one(D, G, gap):
    """One key `gap` above 6000 others in the exponent: what those add up to is what they
    have of the output (the first key's value is zero), although each weighs e^-gap."""
    n = 6000
    c = make([n], G, 1, D, 16, "f16", seed=35, spread=0.0)
    kc, vc = c["kc"].view(torch.uint8), c["vc"].view(torch.uint8)
    t = c["bt"][0].long()
    kc.zero_()
    one = int(torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8))
    kc[t[0], :, 0] = one
    vc[:] = one
    vc[t[0], :, 0] = 0
    c["ks"].view(torch.uint8).fill_(127)
    c["vs"].view(torch.uint8).fill_(127)
    c["scale"] = 1.0
    c["q"].fill_(gap / D)
    out = check(c, "f16")
    s = (c["q"][0, 0].double().sum()).item()
    want = (n - 1) * math.exp(-s) / (1 + (n - 1) * math.exp(-s))
    # the output's own rounding, the weights' 2^-12 and the sums'
    assert abs(float(out[0, 0, 0]) - want) <= want * (2.0 ** -11 + 2.0 ** -12 + 2 * n * 2.0 ** -24 + 2.0 ** -16) + 2.0 ** -25


@pytest.mark.parametrize("D,G", [(128, 8), (64, 4)])
def test_rising_scores(D, G):
    """Later keys far above earlier ones: the running maximum moves all the way."""
    c = make([900], G, 1, D, 16, "bf16", seed=23, spread=0.0)
    c["q"].fill_(1.0)
    t = c["bt"][0].long()
    for j in range(t.shape[0]):
        codes = torch.full((1, 16, D), 1.0 if j % 2 else -1.0, device=DEV).to(torch.float8_e4m3fn)
        c["kc"].view(torch.uint8)[t[j]] = codes.view(torch.uint8)
        c["ks"].view(torch.uint8)[t[j]] = 127 - 6 + (j * 6) // t.shape[0]
    check(c, "bf16")


def test_no_context_and_tables_that_hold_nothing():
    c = make([0, 0], 4, 2, 128, 16, "bf16", seed=24)
    c["most"] = 40
    assert not bool(decode(c).any())
    for D in (64, 128):
        c = make([40, 700, 20], 4, 2, D, 16, "bf16", seed=25)
        good = check(c, "bf16").clone()
        c["bt"][0] = -5
        c["bt"][1] = 1 << 20
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = decode(c, err)
        torch.cuda.synchronize()
        assert int(err.item()) == pa.capi.DEVERR["block_range"]
        assert not bool(out[:2].any())
        assert bool(((out[2].float() - good[2].float()).abs() <= 2.0 ** -7 * good[2].float().abs() + 2.0 ** -12).all())


@pytest.mark.parametrize("D,G,bs", [(128, 8, 16), (128, 1, 8), (64, 2, 16)])
def test_a_bad_entry_leaves_its_keys_out(D, G, bs):
    c = make([200], G, 1, D, bs, "bf16", seed=26, poison=True)
    j = 3
    keep = torch.ones(200, dtype=torch.bool)
    keep[j * bs:(j + 1) * bs] = False
    kv, vv = (ref8.rows_of(ref8.values(c[a], c[b]), c["bt"][0], 200)[keep] for a, b in (("kc", "ks"), ("vc", "vs")))
    c["bt"][0, j] = c["kc"].shape[0]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = decode(c, err)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.capi.DEVERR["block_range"]
    near(out[0], c["q"][0].cpu().double(), kv, vv, c["scale"], "bf16", 200)


def test_lengths_out_of_range_are_clamped_and_flagged():
    for D in (64, 128):
        c = make([100, 40, 20], 4, 1, D, 16, "bf16", seed=27)
        c["bt"][1:, 3:] = c["bt"][0, 3:].clone()
        want = c["lens"].tolist()
        c["lens"][0] = 10 ** 9
        c["lens"][1] = -4
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = decode(c, err)
        torch.cuda.synchronize()
        assert int(err.item()) == pa.capi.DEVERR["context_range"]
        assert not bool(out[1].any())
        c["lens"] = torch.tensor([100, 0, want[2]], dtype=torch.int32, device=DEV)
        assert torch.equal(out, decode(c))


def test_negative_and_zero_scale():
    c = make([70, 300], 4, 1, 128, 16, "bf16", seed=28)
    for s in (-0.05, 0.0):
        c["scale"] = s
        check(c, "bf16")


def test_nan_in_a_key_or_value_that_is_seen():
    for D, G in ((128, 8), (128, 2), (64, 2)):
        c = make([50, 50], G, 1, D, 16, "bf16", seed=29)
        c["vc"].view(torch.uint8)[c["bt"][0, 1].long(), 0, 3, 7] = 0x7f
        out = decode(c)
        assert bool(torch.isnan(out[0, :, 7]).all())
        others = torch.ones(D, dtype=torch.bool, device=DEV)
        others[7] = False
        assert bool(torch.isfinite(out[0][:, others].float()).all()) and bool(torch.isfinite(out[1].float()).all())
        c["kc"].view(torch.uint8)[c["bt"][1, 0].long(), 0, 3, 7] = 0xff
        out = decode(c)
        assert bool(torch.isnan(out[1]).all())


def test_same_bits_twice_on_another_stream_and_replayed():
    c = make([2000, 5, 700, 64], 16, 2, 128, 16, "bf16", seed=30)
    out = decode(c).clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = torch.zeros_like(out)
    decode(c, out=got, stream=s)
    s.synchronize()
    assert torch.equal(got, out)
    ws = [pa.decode_fp8_workspace(c["q"], 2, 16, c["most"]) for _ in range(2)]
    graphs, outs = [], []
    for w in ws:
        graphs.append(torch.cuda.CUDAGraph())
        outs.append(torch.zeros_like(out))
        with torch.cuda.graph(graphs[-1]):
            decode(c, out=outs[-1], workspace=w)
    for _ in range(2):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)


def test_two_streams_at_once():
    a, b = make([900, 33], 8, 1, 128, 16, "bf16", seed=31), make([1200, 64, 7], 4, 1, 128, 16, "bf16", seed=32)
    wa, wb = decode(a).clone(), decode(b).clone()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        oa, ob = decode(a, stream=sa), decode(b, stream=sb)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)


@pytest.mark.parametrize("D,G", [(128, 8), (128, 4), (64, 1)])
def test_pool_past_32_bits_of_bytes(D, G):
    Hkv, bs = 8, 128
    nb = 2 ** 32 // (Hkv * bs * D) + 40
    lens = [300, 129]
    small = make(lens, G * Hkv, Hkv, D, bs, "bf16", seed=33)
    n = small["kc"].shape[0]
    c = dict(small)
    for x in ("kc", "vc"):
        c[x] = torch.full((nb, Hkv, bs, D), 0x7f, dtype=torch.uint8, device=DEV)
        c[x][nb - n:] = small[x].view(torch.uint8)
        c[x] = c[x].view(torch.float8_e4m3fn)
    for x in ("ks", "vs"):
        c[x] = torch.full((nb, Hkv), 255, dtype=torch.uint8, device=DEV)
        c[x][nb - n:] = small[x].view(torch.uint8)
    c["bt"] = torch.where(small["bt"] >= 0, small["bt"] + (nb - n), small["bt"])
    assert torch.equal(decode(c), decode(small))


def test_wrong_tensors_are_refused():
    c = make([10, 20], 4, 2, 128, 16, "bf16", seed=34)
    a = dict(out=torch.zeros_like(c["q"]), query=c["q"], k_cache=c["kc"], v_cache=c["vc"], k_scales=c["ks"], v_scales=c["vs"],
             block_tables=c["bt"], context_lens=c["lens"], scale=0.1, max_context_len=20)
    pa.pa_decode_fp8(**a)
    for exc, kw in ((TypeError, dict(k_cache=c["kc"].bfloat16())), (TypeError, dict(v_cache=c["vc"].view(torch.uint8))),
                    (TypeError, dict(k_scales=c["ks"].view(torch.uint8).int())), (ValueError, dict(v_scales=c["vs"][:-1])),
                    (TypeError, dict(query=c["q"].float())), (TypeError, dict(out=torch.zeros_like(c["q"]).half())),
                    (TypeError, dict(block_tables=c["bt"].long())), (TypeError, dict(context_lens=c["lens"].long())),
                    (ValueError, dict(context_lens=c["lens"][:1])), (ValueError, dict(block_tables=c["bt"].cpu())),
                    (ValueError, dict(out=torch.zeros_like(c["q"])[:1])), (pa.PAError, dict(scale=float("nan"))),
                    (pa.PAError, dict(max_context_len=100000, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV)))):
        with pytest.raises(exc):
            pa.pa_decode_fp8(**{**a, **kw})
