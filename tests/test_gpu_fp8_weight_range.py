"""Decode over an 8-bit cache: many small softmax weights beside a large one, in rows
that a CTA has as a whole (every row of the batch attends the same blocks, so that there
are many of them at no cost), and in rows that are cut.

Tolerance, by arithmetic.  A weight w = 2^(z - M + 11), M a running maximum that lags
behind by less than 2^4, enters as four e5m2 rows, each the residual of those before
times 2^3.  A row keeps three bits, so that four are off by at most 2^-12 of the weight;
the last row's half step is 2^-17 2^-9, 2^-37 beside a weight at the maximum.  All small
weights are rounded alike, so that nothing averages.  The rest as in the decode's test."""
import math

import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.ref64 import DTYPES, half_step
from tests.test_gpu_fp8_decode import DEV, _built  # noqa: F401

pytestmark = pytest.mark.gpu


def code(x):
    return int(torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("D,G", [(128, 1), (128, 4), (128, 8), (64, 2), (64, 8)])
@pytest.mark.parametrize("gap", [9.0, 14.0, 18.0, 22.0])
@pytest.mark.parametrize("at", [0, 1023, 700])
@pytest.mark.parametrize("dtype,B", [("f16", 1400), ("bf16", 3)])
def test_a_tail_beside_one_key(D, G, gap, at, dtype, B):
    n, bs = 1024, 16
    nb = n // bs
    kc = torch.zeros((nb, 1, bs, D), dtype=torch.uint8, device=DEV)
    vc = torch.full((nb, 1, bs, D), code(256.0), dtype=torch.uint8, device=DEV)
    kc[at // bs, 0, at % bs] = code(1.0)
    vc[at // bs, 0, at % bs] = 0
    ks, vs = (torch.full((nb, 1), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    q = torch.full((B, G, D), gap / D, device=DEV).to(DTYPES[dtype])
    bt = torch.arange(nb, dtype=torch.int32, device=DEV).repeat(B, 1)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, float("nan"))
    pa.pa_decode_fp8(out, q, kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), ks, vs, bt, lens, 1.0, n)
    s = float(q[0, 0].double().sum())
    want = 256.0 * (n - 1) * math.exp(-s) / (1 + (n - 1) * math.exp(-s))
    size = 2 * (D + 8) * 2.0 ** -24 * s
    rel = 2.0 ** -12 + 2.0 ** -37 * math.exp(s) + 2 * (size + 2.0 ** -22) + 2 * n * 2.0 ** -24 + 2.0 ** -20
    bound = want * (half_step(dtype) * (1 + 2.0 ** -10) + rel) + 2.0 ** -25
    err = float((out.double() - want).abs().max())
    assert err <= bound, (err / want, bound / want)
