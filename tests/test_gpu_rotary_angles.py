"""pa_rotary_and_cache at frequencies of more than one radian a position and at the
farthest positions, against angles in exact rational arithmetic.  Tolerance: the
angle is off by |position| * 2^-64 turns, at most 2^-33; with that cosine and sine still carry at most 2^-22 each, and a result is off by at
most 2^-21 (|a| + |b|) before it is rounded once (2^-25 more where fp16 is subnormal)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.ref64 import DTYPES, half_step, rotate

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
# 1 / (2 pi) to 80 digits
TURN = Fraction("0.15915494309189533576888376337251436203445964574045644874766734405889679763422654")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def exact_angle(pos, f):
    t = Fraction(int(pos)) * Fraction(float(f)) * TURN
    t -= round(t)
    return float(t) * (2 * np.pi)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_large_frequencies_and_far_positions(interleaved, dtype):
    T, Hq, Hkv, D, bs = 64, 2, 1, 64, 16
    g = torch.Generator().manual_seed(1)
    rng = np.random.default_rng(2)
    dt = DTYPES[dtype]
    q, k, v = (torch.randn((T, h, D), generator=g).to(dt).to(DEV) for h in (Hq, Hkv, Hkv))
    pos = np.concatenate([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1], rng.integers(-2 ** 31, 2 ** 31, T - 6)]).astype(np.int32)
    inv = np.array([1.0, 2 * np.pi, np.pi, 100.0, 12345.678, 3.0e6, 2.0 ** 20, 1e9, -100.0, -7.5, 0.7, 1e-3, 2.0 ** -40, 0.0,
                    6.25, 1 / 3, 3.4e38, -1e-40, 1e20, 2.0 ** 104] + list(10.0 ** rng.uniform(-6, 9, 12)), dtype=np.float32)
    nb = T // bs
    kc, vc = (torch.zeros((nb, Hkv, bs, D), dtype=dt, device=DEV) for _ in range(2))
    out = torch.empty_like(q)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_rotary_and_cache(out, q, k, v, kc, vc, torch.as_tensor(pos, device=DEV), torch.arange(T, device=DEV),
                           torch.as_tensor(inv, device=DEV), interleaved=interleaved, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    angle = torch.tensor([[exact_angle(p, f) for f in inv] for p in pos], dtype=torch.float64)
    half = D // 2
    i, j = (slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, half), slice(half, D))
    keys = kc.permute(0, 2, 1, 3).reshape(T, Hkv, D)
    for got, src in ((out, q), (keys, k)):
        x = src.cpu().double()
        ref = rotate(x, angle, interleaved)
        size = torch.empty_like(x)
        size[..., i] = x[..., i].abs() + x[..., j].abs()
        size[..., j] = size[..., i]
        bound = ref.abs() * half_step(dtype) * (1 + 2.0 ** -10) + size * 2.0 ** -21 + 2.0 ** -25
        off = (got.cpu().double() - ref).abs() - bound
        assert bool((off <= 0).all()), float(off.max())
