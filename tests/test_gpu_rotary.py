"""pa_rotary_and_cache against the rotation in 64 bits.

Tolerance, by arithmetic: cosine and sine carry at most 2^-22 each (the angle
is a rounded fp32 fraction of a turn, and sincospi is good to 2 ulp), the two
products and their sum 2^-23 more, so a result is off by at most 2^-21 (|a| +
|b|) before it is rounded once to the element type (2^-25 more where fp16 is
subnormal)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.ref64 import DTYPES, half_step, rotate

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def make(T, Hq, Hkv, D, R, axes, dtype, bs, seed, far=1 << 20, fused=True, pad=0.2):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[dtype]
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g).to(dt).to(DEV)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = -(-T // bs) + 3
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    slots[rng.random(T) < pad] = -1
    pos = rng.integers(-far, far, size=(axes, T)).astype(np.int32)
    inv = (10000.0 ** (-np.arange(R // 2) / max(1, R // 2))).astype(np.float32)
    ax = rng.integers(0, axes, size=R // 2).astype(np.int32)
    return dict(q=q, k=k, v=v, pos=torch.as_tensor(pos, device=DEV), slots=torch.as_tensor(slots, device=DEV),
                inv=torch.as_tensor(inv, device=DEV), ax=ax,
                kc=torch.randn((nb, Hkv, bs, D), generator=g).to(dt).to(DEV),
                vc=torch.randn((nb, Hkv, bs, D), generator=g).to(dt).to(DEV))


def want(c, interleaved):
    pos, inv = c["pos"].cpu().numpy().astype(np.float64), c["inv"].cpu().numpy().astype(np.float64)
    ax = c["ax"] if c["ax"] is not None else np.zeros(len(inv), int)
    angle = torch.as_tensor((pos.reshape(-1, pos.shape[-1])[ax] if len(ax) else np.zeros((0, pos.shape[-1]))).T * inv)
    q, k = c["q"].cpu().double(), c["k"].cpu().double()
    return rotate(q, angle, interleaved), rotate(k, angle, interleaved)


def near(got, ref, src, R, interleaved, dtype):
    """|got - ref| within the bound; ``src`` holds the unrotated values."""
    a = src.cpu().double().abs()
    size = a.clone()
    half = R // 2
    i, j = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, half), slice(half, R))
    size[..., i] = a[..., i] + a[..., j]
    size[..., j] = a[..., i] + a[..., j]
    bound = ref.abs() * half_step(dtype) * (1 + 2.0 ** -10) + size * 2.0 ** -21 + 2.0 ** -25
    bound[..., R:] = 0.0  # passes unchanged
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


def check(c, R, interleaved, dtype, query_out=None):
    kc0, vc0 = c["kc"].clone(), c["vc"].clone()
    qsrc, ksrc = c["q"].clone(), c["k"].clone()
    wq, wk = want(c, interleaved)
    out = torch.full(c["q"].shape, float("nan"), dtype=c["q"].dtype, device=DEV) if query_out is None else query_out
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_rotary_and_cache(out, c["q"], c["k"], c["v"], c["kc"], c["vc"], c["pos"], c["slots"], c["inv"], c["ax"],
                           interleaved=interleaved, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    near(out, wq, qsrc, R, interleaved, dtype)
    bs = kc0.shape[2]
    slots = c["slots"].cpu()
    t = torch.nonzero(slots >= 0)[:, 0]
    b, r = slots[t] // bs, slots[t] % bs
    if len(t):
        near(c["kc"].cpu()[b, :, r], wk[t], ksrc.cpu()[t], R, interleaved, dtype)
    # values to the bit, and every other slot as it was
    vc0[b.to(DEV), :, r.to(DEV)] = c["v"][t.to(DEV)]
    assert torch.equal(vc0, c["vc"])
    kc0[b.to(DEV), :, r.to(DEV)] = c["kc"][b.to(DEV), :, r.to(DEV)]
    assert torch.equal(kc0, c["kc"])
    return out


CASES = [
    # (T, Hq, Hkv, D, R, axes, bs, dtype, interleaved, fused)
    (1, 32, 8, 128, 128, 3, 16, "bf16", False, True),
    (1, 1, 1, 64, 64, 1, 8, "f16", True, False),
    (33, 8, 2, 128, 128, 3, 16, "f16", True, True),
    (65, 4, 4, 128, 64, 2, 32, "bf16", True, True),      # half of the head unrotated
    (17, 4, 1, 128, 32, 4, 128, "f16", False, False),
    (129, 5, 5, 96, 48, 8, 64, "bf16", False, True),     # units of a head not a power of two
    (40, 3, 1, 256, 256, 1, 16, "f16", False, True),
    (7, 64, 8, 16, 16, 3, 16, "bf16", True, True),       # one unit a head
    (300, 40, 40, 128, 128, 1, 16, "f16", False, True),  # more units than threads
    (9, 8, 8, 64, 0, 1, 16, "bf16", False, True),        # nothing rotated: a plain cache write
    (45, 4, 2, 64, 32, 2, 5, "f16", False, True),        # any block size
    (2100, 2, 1, 64, 64, 3, 16, "bf16", False, True),    # more tokens than CTAs: each walks several
    (1300, 1, 1, 256, 256, 2, 32, "f16", True, False),   # more pairs than threads
]


@pytest.mark.parametrize("T,Hq,Hkv,D,R,axes,bs,dtype,interleaved,fused", CASES)
def test_rotation_and_cache_write(T, Hq, Hkv, D, R, axes, bs, dtype, interleaved, fused):
    c = make(T, Hq, Hkv, D, R, axes, dtype, bs, seed=T + R + axes, fused=fused)
    check(c, R, interleaved, dtype)


def test_positions_to_the_ends_of_their_range():
    c = make(24, 4, 2, 128, 128, 1, "f16", 16, seed=5)
    ends = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 10 ** 9 + 7, 131071]
    c["pos"] = torch.as_tensor(np.resize(np.array(ends, np.int64), 24).astype(np.int32)[None], device=DEV)
    check(c, 128, False, "f16")


def test_position_zero_changes_nothing_and_pads_are_not_written():
    c = make(50, 8, 2, 128, 128, 1, "bf16", 16, seed=6, pad=1.1)
    c["pos"].zero_()
    out = check(c, 128, True, "bf16")
    assert torch.equal(out, c["q"])


def test_in_place_and_one_dimensional_positions():
    c = make(70, 8, 2, 128, 128, 1, "bf16", 16, seed=7)
    c["pos"], c["ax"] = c["pos"][0].contiguous(), None
    check(c, 128, False, "bf16", query_out=c["q"])


def test_odd_strides_and_a_strided_output():
    c = make(31, 4, 2, 64, 64, 2, "f16", 16, seed=8)
    wide = torch.randn((31, 17, 64), device=DEV).half()
    c["q"] = wide[:, 3:7]
    home = torch.zeros((31, 9, 64), dtype=torch.float16, device=DEV)
    check(c, 64, True, "f16", query_out=home[:, 5:9])
    assert not bool(home[:, :5].any())


def test_slot_past_the_pool_is_flagged_and_the_rest_written():
    c = make(6, 4, 2, 64, 64, 1, "bf16", 16, seed=9, pad=0.0)
    nb, bs = c["kc"].shape[0], 16
    c["slots"][2] = nb * bs
    c["slots"][4] = 2 ** 40
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(c["q"])
    v0 = c["vc"].clone()
    pa.pa_rotary_and_cache(out, c["q"], c["k"], c["v"], c["kc"], c["vc"], c["pos"], c["slots"], c["inv"], c["ax"], d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.capi.DEVERR["slot_range"]
    ok = [0, 1, 3, 5]
    s = c["slots"][ok]
    v0[s // bs, :, s % bs] = c["v"][ok]
    assert torch.equal(v0, c["vc"])
    near(out, want(c, False)[0], c["q"], 64, False, "bf16")   # their queries are rotated all the same


def test_no_tokens_is_a_no_op_and_wrong_tensors_are_refused():
    c = make(4, 4, 2, 64, 64, 1, "bf16", 16, seed=10)
    e = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    z = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    pa.pa_rotary_and_cache(e, e, z, z, c["kc"], c["vc"], c["pos"][:, :0].contiguous(), c["slots"][:0], c["inv"])
    a = (torch.zeros_like(c["q"]), c["q"], c["k"], c["v"], c["kc"], c["vc"], c["pos"], c["slots"], c["inv"])

    def bad(i, x, exc):
        b = list(a)
        b[i] = x
        with pytest.raises(exc):
            pa.pa_rotary_and_cache(*b)
    bad(6, c["pos"].long(), TypeError)
    bad(7, c["slots"].int(), TypeError)
    bad(8, c["inv"].double(), TypeError)
    bad(1, c["q"].half(), TypeError)
    bad(1, c["q"].cpu(), ValueError)
    bad(2, c["k"][:3], ValueError)
    bad(1, c["q"].transpose(1, 2).contiguous().transpose(1, 2), ValueError)   # heads not contiguous
    with pytest.raises(ValueError):
        pa.pa_rotary_and_cache(*a, pair_axis=[0])
    with pytest.raises(pa.PAError) as e3:
        pa.pa_rotary_and_cache(*a, pair_axis=[1] * 32)
    assert e3.value.status == -3


def test_captured_and_replayed_and_on_another_stream():
    c = make(20, 8, 2, 128, 128, 3, "bf16", 16, seed=11)
    out = check(c, 128, False, "bf16").clone()
    kc, vc = c["kc"].clone(), c["vc"].clone()
    got = torch.zeros_like(out)
    s = torch.cuda.Stream()
    args = (got, c["q"], c["k"], c["v"], c["kc"], c["vc"], c["pos"], c["slots"], c["inv"], c["ax"])
    torch.cuda.synchronize()
    pa.pa_rotary_and_cache(*args, stream=s)
    s.synchronize()
    assert torch.equal(got, out)
    got.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_rotary_and_cache(*args)
    for _ in range(2):
        got.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, out) and torch.equal(kc, c["kc"]) and torch.equal(vc, c["vc"])
