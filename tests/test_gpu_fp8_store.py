"""Writing an 8-bit cache, against its definition in 64 bits.

Values and unrotated keys are exact until they are rounded to a code, so their
codes and all scales have to be equal.  Rotated and normed keys carry an fp32
error d before that rounding:
  rotation  2^-21 (|a| + |b|) for a pair (the 16-bit call's bound);
  norm      the sum of at most 256 squares is off by (16 + 4 + 2) 2^-24 of itself
            (16 terms a lane, 4 additions across lanes), which its inverse root
            halves; root, two products and eps add 4 * 2^-24: 2^-20 in all.
A code is then off from the exact value by at most half a step at that value plus
d; the scale is the exact one unless the largest magnitude is within d of a limit."""
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


def make_slots(kind, T, bs, rng):
    """(slots, blocks) of T tokens."""
    i = np.arange(T)
    if kind == "run":        # one sequence from its first row on
        nb = -(-T // bs) + 3
        b = rng.permutation(nb)
        return b[i // bs] * bs + i % bs, nb
    if kind == "onward":     # one sequence from the middle of a block on
        nb = -(-T // bs) + 3
        b = rng.permutation(nb)
        j = i + bs // 2
        return b[j // bs] * bs + j % bs, nb
    if kind == "step":       # a token of each of T sequences
        return rng.permutation(T + 2)[:T] * bs + rng.integers(0, bs, size=T), T + 2
    if kind == "scattered":  # any rows, in any order, some twice, some padding
        nb = max(2, T // bs + 1)
        s = rng.integers(0, nb * bs, size=T)
        s[rng.random(T) < 0.2] = -1
        return s, nb
    raise ValueError(kind)


def make(T, Hq, Hkv, D, R, dtype, bs, kind, seed, norm, fused=True, axes=2):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[dtype]
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g).to(dt).to(DEV)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    slots, nb = make_slots(kind, T, bs, rng)
    caches = []
    for _ in range(2):
        # what earlier writes left: of all sizes, so that some scales grow and some stay
        x = torch.randn((nb, Hkv, bs, D), generator=g) * torch.exp2(torch.randint(-6, 3, (nb, Hkv, 1, 1), generator=g).float())
        c, s = ref8.quantise(x)
        caches += [c.to(DEV), s.view(torch.float8_e8m0fnu).to(DEV)]
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt).to(DEV) for _ in range(2)] if norm else [None, None]
    return dict(q=q, k=k, v=v, slots=torch.as_tensor(slots.astype(np.int64), device=DEV),
                pos=torch.as_tensor(rng.integers(-99999, 1 << 20, size=(axes, T)).astype(np.int32), device=DEV),
                inv=torch.as_tensor((1e4 ** (-np.arange(R // 2) / max(1, R // 2))).astype(np.float32), device=DEV),
                ax=rng.integers(0, axes, size=R // 2).astype(np.int32), wq=w[0], wk=w[1], eps=1e-5,
                kc=caches[0], ks=caches[1], vc=caches[2], vs=caches[3])


def keys_of(c, x, w, R, interleaved):
    """Exact normed and rotated rows, and their fp32 error bound."""
    y = x.cpu().double() if w is None else ref8.normed(x, w, c["eps"])
    size = y.abs()
    both = size.clone()
    half = R // 2
    i, j = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, half), slice(half, R))
    both[..., i] = size[..., i] + size[..., j]
    both[..., j] = both[..., i]
    d = both * 2.0 ** -21 if R else torch.zeros_like(y)
    d[..., R:] = 0
    if w is not None:
        d = d + both * 2.0 ** -20
    return ref8.turned(y, c["pos"], c["inv"], c["ax"], interleaved), d


def check(c, R, interleaved, dtype, call=None):
    old = [x.clone() for x in (c["kc"], c["ks"], c["vc"], c["vs"])]
    q0 = c["q"].clone()
    out = torch.full(c["q"].shape, float("nan"), dtype=c["q"].dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    if call is None:
        pa.pa_rotary_and_cache_fp8(out, c["q"], c["k"], c["v"], c["kc"], c["vc"], c["ks"], c["vs"], c["pos"], c["slots"],
                                   c["inv"], c["wq"], c["wk"], c["eps"], c["ax"], interleaved=interleaved, d_err=err)
    else:
        call(err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    f16 = dtype == "f16"
    # values: codes and scales to the bit, all over the pool
    want, e = ref8.store(old[2], old[3], c["v"].cpu().double(), c["slots"].cpu(), f16)
    assert torch.equal(c["vs"].cpu().view(torch.uint8).long() - 127, e)
    got = c["vc"].cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(), want.nan_to_num())
    # keys
    y, d = keys_of(c, c["k"], c["wk"], R, interleaved)
    want, e = ref8.store(old[0], old[1], y, c["slots"].cpu(), f16)
    assert torch.equal(c["ks"].cpu().view(torch.uint8).long() - 127, e)
    got = c["kc"].cpu().double()
    bs = got.shape[2]
    place = {}
    for t, s in enumerate(c["slots"].tolist()):
        if s >= 0:
            place[s] = t
    left = torch.ones(got.shape[0], bs, dtype=torch.bool)
    for s, t in place.items():
        b, r = s // bs, s % bs
        left[b, r] = False
        sc = ref8.pow2(e[b])[:, None]
        x = y[t].clamp(-ref8.F16_TOP, ref8.F16_TOP) if f16 else y[t]
        bound = torch.maximum(x.abs() * 2.0 ** -4, sc * 2.0 ** -10) + d[t] * 2
        lost = ~torch.isfinite(x)
        assert torch.equal(torch.isnan(got[b, :, r]), lost)
        assert bool((((got[b, :, r] * sc - x).abs() <= bound) | lost).all())
        # and the very code wherever the exact value is not within d of a rounding border
        sure = ref8.to_grid((x - d[t]) / sc) == ref8.to_grid((x + d[t]) / sc)
        assert torch.equal(got[b, :, r][sure], want[b, :, r][sure])
    keep = left[:, None].expand(-1, got.shape[1], -1)
    assert torch.equal(got[keep], want[keep])
    if call is None:
        # queries, as the 16-bit calls leave them
        y, d = keys_of(c, q0, c["wq"], R, interleaved)
        bound = y.abs() * half_step(dtype) * (1 + 2.0 ** -10) + d + 2.0 ** -25
        assert bool(((out.cpu().double() - y).abs() <= bound).all())
    return out


CASES = [
    # (T, Hq, Hkv, D, R, bs, dtype, interleaved, norm, kind)
    (1, 8, 2, 128, 128, 16, "bf16", False, True, "run"),
    (1, 8, 2, 128, 128, 16, "f16", False, False, "onward"),
    (40, 4, 2, 64, 64, 16, "f16", True, True, "onward"),
    (37, 32, 8, 128, 128, 16, "bf16", False, True, "step"),
    (70, 5, 5, 96, 48, 8, "bf16", False, True, "scattered"),      # a head's units are not a power of two
    (33, 20, 20, 128, 64, 32, "f16", True, False, "run"),         # more heads than a CTA takes
    (300, 2, 1, 128, 128, 128, "bf16", False, True, "onward"),    # blocks of more rows than are held at a time
    (200, 3, 3, 64, 32, 64, "f16", False, True, "scattered"),
    (90, 1, 1, 256, 256, 16, "bf16", True, True, "run"),
    (50, 2, 2, 16, 16, 16, "f16", False, True, "step"),           # one unit a head
    (64, 4, 1, 128, 0, 16, "bf16", False, True, "scattered"),     # norms alone
    (64, 4, 4, 64, 0, 32, "f16", False, False, "scattered"),      # neither
    (600, 2, 2, 64, 64, 16, "bf16", False, False, "run"),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,R,bs,dtype,interleaved,norm,kind", CASES)
def test_rotary_store(T, Hq, Hkv, D, R, bs, dtype, interleaved, norm, kind):
    c = make(T, Hq, Hkv, D, R, dtype, bs, kind, seed=T + D + R, norm=norm)
    check(c, R, interleaved, dtype)


@pytest.mark.parametrize("kind", ["run", "onward", "step", "scattered"])
@pytest.mark.parametrize("dtype,bs,D,Hkv", [("bf16", 16, 128, 8), ("f16", 8, 64, 3), ("f16", 128, 128, 17)])
def test_plain_store(kind, dtype, bs, D, Hkv):
    c = make(45, 1, Hkv, D, 0, dtype, bs, kind, seed=45 + bs, norm=False, fused=False)
    check(c, 0, False, dtype, call=lambda err: pa.pa_reshape_and_cache_fp8(
        c["k"], c["v"], c["kc"], c["vc"], c["ks"], c["vs"], c["slots"], d_err=err))


def test_a_block_filled_token_by_token_and_at_once_agree_where_nothing_is_subnormal():
    c = make(16, 1, 2, 64, 0, "bf16", 16, "run", seed=3, norm=False, fused=False)
    for x in (c["k"], c["v"]):  # magnitudes within the normal codes of any scale on the way
        x.copy_(torch.where(x < 0, -1.0, 1.0) * (x.float().abs().clamp(0.25, 3.0)))
    kc, ks, vc, vs = (x.clone() for x in (c["kc"], c["ks"], c["vc"], c["vs"]))
    pa.pa_reshape_and_cache_fp8(c["k"], c["v"], kc, vc, ks, vs, c["slots"])
    for t in range(16):
        pa.pa_reshape_and_cache_fp8(c["k"][t:t + 1], c["v"][t:t + 1], c["kc"], c["vc"], c["ks"], c["vs"], c["slots"][t:t + 1])
    for a, b in ((kc, c["kc"]), (ks, c["ks"]), (vc, c["vc"]), (vs, c["vs"])):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_zeros_infinities_nan_and_the_ends_of_the_range(dtype):
    c = make(48, 1, 2, 64, 0, dtype, 16, "run", seed=4, norm=False, fused=False)
    big = 3.0e38 if dtype == "bf16" else 65504.0
    c["v"][:16] = 0
    c["v"][16, 0, 3] = float("inf")
    c["v"][17, 0, 5] = float("nan")
    c["v"][18, 1, 0] = -float("inf")
    c["v"][33, 0, 1] = big
    c["v"][34, 1, 2] = -big
    c["v"][35, 0, 0] = 1e-30 if dtype == "bf16" else 6e-8
    c["k"][:16] = float("nan")          # a block and head without one finite value
    c["k"][32:] = 1e-38 if dtype == "bf16" else 6e-8
    check(c, 0, False, dtype, call=lambda err: pa.pa_reshape_and_cache_fp8(
        c["k"], c["v"], c["kc"], c["vc"], c["ks"], c["vs"], c["slots"], d_err=err))


def test_scales_at_their_limits():
    """amax exactly 448 * 2^e, and the next bf16 value above."""
    c = make(32, 1, 1, 64, 0, "bf16", 16, "run", seed=5, norm=False, fused=False)
    c["v"].clamp_(-1, 1)
    c["v"][3, 0, 0], c["v"][20, 0, 9] = 448.0 / 64, 450.0 / 64
    check(c, 0, False, "bf16", call=lambda err: pa.pa_reshape_and_cache_fp8(
        c["k"], c["v"], c["kc"], c["vc"], c["ks"], c["vs"], c["slots"], d_err=err))
    b = (c["slots"][[0, 16]] // 16).tolist()
    assert [int(x) for x in c["vs"].view(torch.uint8)[b, 0]] == [127 - 6, 127 - 5]


def test_slot_past_the_pool_is_flagged_and_the_rest_written():
    c = make(6, 4, 2, 64, 64, "bf16", 16, "step", seed=9, norm=False)
    nb = c["kc"].shape[0]
    d = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    c["slots"][2], c["slots"][4] = nb * 16, 2 ** 40
    d["slots"][2], d["slots"][4] = -1, -1
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = []
    for x in (c, d):
        outs.append(torch.zeros_like(c["q"]))
        pa.pa_rotary_and_cache_fp8(outs[-1], x["q"], x["k"], x["v"], x["kc"], x["vc"], x["ks"], x["vs"], x["pos"], x["slots"],
                                   x["inv"], pair_axis=x["ax"], d_err=err if x is c else None)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.capi.DEVERR["slot_range"]
    assert torch.equal(outs[0], outs[1])
    for n in ("kc", "vc", "ks", "vs"):
        assert torch.equal(c[n].view(torch.uint8), d[n].view(torch.uint8))


def test_query_in_place_strided_and_one_dimensional_positions():
    c = make(31, 4, 2, 64, 64, "f16", 16, "run", seed=8, norm=True, axes=1)
    c["pos"], c["ax"] = c["pos"][0].contiguous(), None
    want = check(c, 64, True, "f16").clone()
    pa.pa_rotary_and_cache_fp8(c["q"], c["q"], c["k"], c["v"], c["kc"], c["vc"], c["ks"], c["vs"], c["pos"], c["slots"],
                               c["inv"], c["wq"], c["wk"], c["eps"], interleaved=True)
    assert torch.equal(c["q"], want)


@pytest.mark.parametrize("T", [1, 2, 7, 64, 700])
def test_slots_that_begin_between_16_byte_boundaries(T):
    """(as a slice of a step's slot mapping does)"""
    c = make(T, 4, 2, 64, 64, "bf16", 16, "scattered" if T > 2 else "step", seed=12 + T, norm=True)
    home = torch.full((T + 1,), 3, dtype=torch.int64, device=DEV)   # the slot before would clash
    home[1:] = c["slots"]
    c["slots"] = home[1:]
    check(c, 64, True, "bf16")


def test_two_runs_of_one_block_far_apart():
    """Tokens of one block at the call's two ends, and a slot that three of them name."""
    T = 900
    c = make(T, 2, 3, 64, 64, "f16", 16, "run", seed=13, norm=False)
    b = int(c["slots"][0]) // 16
    c["slots"][T - 5:] = torch.tensor([b * 16 + 9, b * 16 + 3, b * 16 + 3, b * 16 + 15, b * 16 + 9], device=DEV)
    c["slots"][450] = b * 16 + 3
    check(c, 64, False, "f16")
    c["slots"][:16] = c["slots"][:16].flip(0)
    check(c, 64, False, "f16")


def test_same_bits_on_another_stream_and_replayed():
    c = make(64, 8, 2, 128, 128, "bf16", 16, "onward", seed=11, norm=True)
    start = [x.clone() for x in (c["kc"], c["vc"], c["ks"], c["vs"])]
    out = check(c, 128, False, "bf16").clone()
    done = [x.clone() for x in (c["kc"], c["vc"], c["ks"], c["vs"])]
    got = torch.zeros_like(out)
    args = (got, c["q"], c["k"], c["v"], c["kc"], c["vc"], c["ks"], c["vs"], c["pos"], c["slots"], c["inv"], c["wq"], c["wk"],
            c["eps"], c["ax"])

    def restart():
        got.zero_()
        for x, y in zip((c["kc"], c["vc"], c["ks"], c["vs"]), start):
            x.copy_(y)

    def same():
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        for x, y in zip((c["kc"], c["vc"], c["ks"], c["vs"]), done):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    s = torch.cuda.Stream()
    restart()
    torch.cuda.synchronize()
    pa.pa_rotary_and_cache_fp8(*args, stream=s)
    s.synchronize()
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_rotary_and_cache_fp8(*args)
    for _ in range(2):
        restart()
        graph.replay()
        same()


def test_pools_past_32_bits_of_bytes():
    Hkv, bs, D = 8, 128, 128
    nb = 2 ** 32 // (Hkv * bs * D) + 40
    kc, vc = (torch.zeros((nb, Hkv, bs, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((nb, Hkv), 100, dtype=torch.uint8, device=DEV) for _ in range(2))
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((4, Hkv, D), generator=g).bfloat16().to(DEV) for _ in range(2))
    far = nb - 2
    slots = torch.tensor([far * bs, far * bs + 1, bs + 1, bs + 2], device=DEV)
    pa.pa_reshape_and_cache_fp8(k, v, kc, vc, ks, vs, slots)
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        small = torch.stack([c[far], c[1]])
        want, e = ref8.store(torch.zeros(2, Hkv, bs, D).to(torch.float8_e4m3fn), torch.full((2, Hkv), 100, dtype=torch.uint8),
                             x.cpu().double(), torch.tensor([0, 1, bs + 1, bs + 2]), False)
        # (the second block gets its second and third rows, so that its old scale counts)
        assert torch.equal(small.cpu().double(), want)
        assert torch.equal(s[[far, 1]].cpu().long() - 127, e)
        assert not bool(c.view(torch.uint8)[2:far].view(torch.int64).any())


def test_no_tokens_and_wrong_tensors_are_refused():
    c = make(4, 4, 2, 64, 64, "bf16", 16, "run", seed=10, norm=False, fused=False)
    pa.pa_reshape_and_cache_fp8(c["k"][:0], c["v"][:0], c["kc"], c["vc"], c["ks"], c["vs"], c["slots"][:0])
    a = dict(key=c["k"], value=c["v"], k_cache=c["kc"], v_cache=c["vc"], k_scales=c["ks"], v_scales=c["vs"],
             slot_mapping=c["slots"])

    def bad(exc, **kw):
        with pytest.raises(exc):
            pa.pa_reshape_and_cache_fp8(**{**a, **kw})
    bad(TypeError, k_cache=c["kc"].float())
    bad(TypeError, k_cache=c["kc"].view(torch.uint8))
    bad(TypeError, k_scales=c["ks"].view(torch.uint8).float())
    bad(TypeError, slot_mapping=c["slots"].int())
    bad(TypeError, value=c["v"].half())
    bad(TypeError, key=c["k"].float(), value=c["v"].float())
    bad(ValueError, k_scales=c["ks"][:, :1].contiguous())
    bad(ValueError, key=c["k"][:3])
    bad(ValueError, key=c["k"].cpu())
    bad(pa.PAError, v_scales=c["ks"])
    bad(pa.PAError, v_cache=c["kc"])
    r = dict(query_out=torch.zeros_like(c["q"]), query=c["q"], key=c["k"], value=c["v"], k_cache=c["kc"], v_cache=c["vc"],
             k_scales=c["ks"], v_scales=c["vs"], positions=c["pos"], slot_mapping=c["slots"], inv_freq=c["inv"])
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    for exc, kw in ((ValueError, dict(query_norm=w)), (TypeError, dict(query_norm=w.float(), key_norm=w.float())),
                    (ValueError, dict(query_norm=w[:32], key_norm=w[:32])), (ValueError, dict(positions=None)),
                    (TypeError, dict(positions=c["pos"].long())), (ValueError, dict(pair_axis=[0])),
                    (pa.PAError, dict(query_norm=w, key_norm=w, eps=-1.0)),
                    (pa.PAError, dict(query_norm=w, key_norm=w, eps=float("nan")))):
        with pytest.raises(exc):
            pa.pa_rotary_and_cache_fp8(**{**r, **kw})
