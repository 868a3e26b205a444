"""Head norms with the rotation and the 16-bit cache write, against 64 bits.

Error before the one rounding: 2^-21 (|a| + |b|) from the rotation of a pair (the
rotary call's bound) and, from the norm, 2^-20 of either: the sum of at most 256
squares is off by (16 + 4 + 2) 2^-24 of itself, which its inverse root halves; root,
two products and eps add 4 * 2^-24."""
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


def make(T, Hq, Hkv, D, R, axes, bs, dtype, seed, pad=0.2):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[dtype]
    # heads of very different sizes: what a norm is for
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g) * torch.exp2(4 * torch.randn((T, Hq + 2 * Hkv, 1), generator=g))
    qkv = qkv.clamp(-3e4, 3e4).to(dt).to(DEV)
    nb = -(-T // bs) + 3
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    slots[rng.random(T) < pad] = -1
    return dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], slots=torch.as_tensor(slots, device=DEV),
                pos=torch.as_tensor(rng.integers(-99999, 1 << 20, size=(axes, T)).astype(np.int32), device=DEV),
                inv=torch.as_tensor((1e4 ** (-np.arange(R // 2) / max(1, R // 2))).astype(np.float32), device=DEV),
                ax=rng.integers(0, axes, size=R // 2).astype(np.int32),
                wq=(1 + 0.3 * torch.randn(D, generator=g)).to(dt).to(DEV),
                wk=(1 + 0.3 * torch.randn(D, generator=g)).to(dt).to(DEV),
                kc=torch.randn((nb, Hkv, bs, D), generator=g).to(dt).to(DEV),
                vc=torch.randn((nb, Hkv, bs, D), generator=g).to(dt).to(DEV))


def want(c, x, w, R, interleaved, eps, dtype):
    y = ref8.normed(x, w, eps)
    a = y.abs()
    both = a.clone()
    i, j = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    both[..., i] = a[..., i] + a[..., j]
    both[..., j] = both[..., i]
    y = ref8.turned(y, c["pos"], c["inv"], c["ax"], interleaved)
    return y, y.abs() * half_step(dtype) * (1 + 2.0 ** -10) + both * (2.0 ** -20 + 2.0 ** -21) + 2.0 ** -25


def check(c, R, interleaved, dtype, eps=1e-6, out=None):
    kc0, vc0 = c["kc"].clone(), c["vc"].clone()
    wq, bq = want(c, c["q"], c["wq"], R, interleaved, eps, dtype)
    wk, bk = want(c, c["k"], c["wk"], R, interleaved, eps, dtype)
    out = torch.full(c["q"].shape, float("nan"), dtype=c["q"].dtype, device=DEV) if out is None else out
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_norm_rotary_and_cache(out, c["q"], c["k"], c["v"], c["kc"], c["vc"], c["pos"], c["slots"], c["inv"], c["wq"],
                                c["wk"], eps, c["ax"], interleaved=interleaved, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert bool(((out.cpu().double() - wq).abs() <= bq).all())
    bs = kc0.shape[2]
    t = torch.nonzero(c["slots"].cpu() >= 0)[:, 0]
    s = c["slots"].cpu()[t]
    b, r = s // bs, s % bs
    assert bool(((c["kc"].cpu().double()[b, :, r] - wk[t]).abs() <= bk[t]).all())
    vc0[b.to(DEV), :, r.to(DEV)] = c["v"][t.to(DEV)]
    assert torch.equal(vc0, c["vc"])
    kc0[b.to(DEV), :, r.to(DEV)] = c["kc"][b.to(DEV), :, r.to(DEV)]
    assert torch.equal(kc0, c["kc"])
    return out


CASES = [
    # (T, Hq, Hkv, D, R, axes, bs, dtype, interleaved)
    (1, 32, 8, 128, 128, 1, 16, "bf16", False),
    (33, 8, 2, 128, 128, 3, 16, "f16", True),
    (65, 4, 4, 128, 64, 2, 32, "bf16", True),       # half of the head unrotated
    (129, 5, 5, 96, 48, 8, 64, "bf16", False),      # lanes without a unit
    (50, 3, 2, 80, 80, 1, 16, "f16", True),
    (40, 3, 1, 256, 256, 1, 16, "f16", False),
    (7, 64, 8, 16, 16, 3, 16, "bf16", True),        # one unit a head
    (300, 40, 40, 128, 128, 1, 16, "f16", False),   # more units than threads
    (9, 8, 8, 64, 0, 1, 16, "bf16", False),         # norms alone
    (45, 4, 2, 64, 32, 2, 5, "f16", False),         # any block size
    (2100, 2, 1, 64, 64, 3, 16, "bf16", False),     # more tokens than CTAs
    (1300, 1, 1, 256, 256, 2, 32, "f16", True),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,R,axes,bs,dtype,interleaved", CASES)
def test_norm_rotation_and_cache_write(T, Hq, Hkv, D, R, axes, bs, dtype, interleaved):
    check(make(T, Hq, Hkv, D, R, axes, bs, dtype, seed=T + R + axes), R, interleaved, dtype)


def test_heads_of_zeros_and_a_large_eps():
    c = make(20, 4, 2, 128, 128, 1, 16, "bf16", seed=5)
    c["q"][3:7] = 0
    c["k"][5] = 0
    check(c, 128, False, "bf16", eps=1e-3)
    check(c, 128, False, "bf16", eps=4.0)


def test_in_place_and_replayed_on_another_stream():
    c = make(70, 8, 2, 128, 128, 2, 16, "f16", seed=7)
    out = check(c, 128, True, "f16").clone()
    got = torch.zeros_like(out)
    args = (got, c["q"], c["k"], c["v"], c["kc"], c["vc"], c["pos"], c["slots"], c["inv"], c["wq"], c["wk"], 1e-6, c["ax"], True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pa.pa_norm_rotary_and_cache(*args, stream=s)
    s.synchronize()
    assert torch.equal(got, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_norm_rotary_and_cache(*args)
    for _ in range(2):
        got.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, out)
    check(c, 128, True, "f16", out=c["q"])


def test_the_plain_call_is_unchanged_by_unit_norms_of_unit_rows():
    """A row whose mean square is 1 with eps 0 and weights 1 turns as pa_rotary_and_cache turns it."""
    c = make(16, 4, 2, 64, 64, 1, 16, "bf16", seed=8, pad=0.0)
    for n in ("q", "k"):
        c[n].copy_(torch.where(c[n] < 0, -1.0, 1.0))
    c["wq"].fill_(1)
    c["wk"].fill_(1)
    a, b = torch.zeros_like(c["q"]), torch.zeros_like(c["q"])
    kc, vc = c["kc"].clone(), c["vc"].clone()
    pa.pa_norm_rotary_and_cache(a, c["q"], c["k"], c["v"], c["kc"], c["vc"], c["pos"], c["slots"], c["inv"], c["wq"], c["wk"], 0.0)
    pa.pa_rotary_and_cache(b, c["q"], c["k"], c["v"], kc, vc, c["pos"], c["slots"], c["inv"])
    assert torch.equal(a, b) and torch.equal(kc, c["kc"]) and torch.equal(vc, c["vc"])


def test_wrong_tensors_are_refused():
    c = make(4, 4, 2, 64, 64, 1, 16, "bf16", seed=10)
    a = dict(query_out=torch.zeros_like(c["q"]), query=c["q"], key=c["k"], value=c["v"], k_cache=c["kc"], v_cache=c["vc"],
             positions=c["pos"], slot_mapping=c["slots"], inv_freq=c["inv"], query_norm=c["wq"], key_norm=c["wk"], eps=1e-6)
    for exc, kw in ((ValueError, dict(query_norm=None)), (ValueError, dict(query_norm=None, key_norm=None)),
                    (TypeError, dict(query_norm=c["wq"].float())), (ValueError, dict(key_norm=c["wk"][:32])),
                    (ValueError, dict(key_norm=c["wk"].cpu())), (TypeError, dict(v_cache=c["vc"].half())),
                    (ValueError, dict(positions=None)), (pa.PAError, dict(eps=-1e-9)), (pa.PAError, dict(eps=float("inf"))),
                    (ValueError, dict(query=c["q"][:2])), (TypeError, dict(key=c["k"].half()))):
        with pytest.raises(exc):
            pa.pa_norm_rotary_and_cache(**{**a, **kw})
