"""Prompt chunks over an 8-bit cache: softmax weights reach the tensor cores with more bits
than the model's type has, so that over short contexts, where few weights share the sum,
outputs stay within one rounding of the exact ones.

Tolerance, by arithmetic.  u = half a step of the type, relative.  In f16 a weight P goes in
as hi + lo, hi = rn(P), lo = rn(P - hi): off by p = u^2, relative, or by 2^-25 where lo is
below f16's normal range (the sum of the weights is 1 at least).  In bf16 it goes in as one
f16 value, the cached values in f16 too: off by p = 2^-12, u / 16, or 2^-32.  A score is off
by D 2^-23 A, A the largest scaled sum of |q_i k_i| (the tensor cores may truncate), a weight
by twice that relatively, plus 2^-19 for the exponentials, sums and division, plus 2^-23 a
key for the product with V.  With W = sum w |v|:
  delta = W (p + 4 D 2^-23 A + 2^-19 + n 2^-22) + n 2^-25 max |v|,
and the result is rounded once: |got - ref| <= delta + u (|ref| + delta).  Queries are
small, so that A is: one 16-bit value for a weight would be off by u W / 2, above that."""
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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 2), (4, 1), (8, 1)])
def test_outputs_within_one_rounding(G, Hkv, bs, dtype):
    prefixes, chunks = [0, 1, 2, 15, 16, 40, 129, 130, 250], [4, 1, 3, 2, 33, 5, 2, 1, 20]
    kc, ks, vc, vs, bt = ref8.make_pool([a + b for a, b in zip(prefixes, chunks)], Hkv, 128, bs, DEV, 81 + G, spread=0.0,
                                        poison=True)
    g = torch.Generator().manual_seed(82)
    q = (torch.randn((sum(chunks), G * Hkv, 128), generator=g) / 16).to(DTYPES[dtype]).to(DEV)
    out, err = torch.full_like(q, float("nan")), torch.zeros(1, dtype=torch.int32, device=DEV)
    scale = 1 / math.sqrt(128)
    pa.pa_prefill_batch_fp8(out, q, kc, vc, ks, vs, bt, prefixes, chunks, scale, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    kv, vv = ref8.values(kc, ks), ref8.values(vc, vs)
    u, at, over, worst = half_step(dtype), 0, 0, 0.0
    p16 = u * u if dtype == "f16" else 2.0 ** -12
    for i, (p, n) in enumerate(zip(prefixes, chunks)):
        K, V = ref8.rows_of(kv, bt[i], p + n), ref8.rows_of(vv, bt[i], p + n)
        for r in range(n):
            m = p + r + 1
            ref, W, A = ref8.attend_sizes(q[at + r].cpu().double(), K[:m], V[:m], scale)
            delta = W * (p16 + 4 * 128 * 2.0 ** -23 * A[:, None] + 2.0 ** -19 + m * 2.0 ** -22) + \
                m * 2.0 ** -25 * float(V[:m].abs().max())
            e = (out[at + r].cpu().double() - ref).abs() / (delta + u * (ref.abs() + delta))
            over += int((e > 1).sum())
            worst = max(worst, float(e.max()))
        at += n
    assert over == 0, (over, worst)
