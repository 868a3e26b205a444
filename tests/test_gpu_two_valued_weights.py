"""Softmax weights that reach the tensor cores as two 16-bit values: over short
contexts, where few weights share the sum, outputs stay within one rounding.

Tolerance, by arithmetic.  u = half a step of the type, relative.  A weight goes in
as hi + lo, hi = rn(P), lo = rn(P - hi): off by u^2 P, or by 2^-25 where lo is below
f16's normal range (P is 1 at least for the largest, and their sum l too).  A score
is off by D 2^-23 A, A the largest scaled sum of |q_i k_i| (the tensor cores may
truncate), and a weight by twice that relatively, plus 2^-19 for the exponentials,
sums and division, plus 2^-23 a key for the product with V.  With W = sum w |v|:
delta = W (u^2 + 4 D 2^-23 A + 2^-19 + n 2^-22) + n 2^-25 max |v|, and the result is
rounded once: |got - ref| <= delta + u (|ref| + delta).  Queries are small, so that A
is: one 16-bit value for a weight would be off by u W / 2, above that, in thousands
of the outputs.  (That is what a common prefix of more than 128 query rows does, by
its contract: there delta takes u W more, half a step of each weight.)"""
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.ref64 import DTYPES, half_step, make_pool

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def check(out, q, kc, vc, table, n, scale, dtype, once=False):
    """out, q [rows][per row][Hq][D] over the first n keys of each table row."""
    bs, u = kc.shape[2], half_step(dtype)
    j = torch.arange(n, device=DEV)
    t = table.long()[:, j // bs]
    K, V = (c[t, :, j % bs].double() for c in (kc, vc))                 # [rows][n][Hkv][D]
    Hkv, D = K.shape[2], K.shape[3]
    R, P, Hq, _ = q.shape
    qd = q.double().view(R, P, Hkv, Hq // Hkv, D)
    s = torch.einsum("rpkgd,rnkd->rpkgn", qd, K) * scale
    A = float((torch.einsum("rpkgd,rnkd->rpkgn", qd.abs(), K.abs()) * scale).max())
    w = torch.softmax(s, -1)
    ref = torch.einsum("rpkgn,rnkd->rpkgd", w, V).reshape(out.shape)
    W = torch.einsum("rpkgn,rnkd->rpkgd", w, V.abs()).reshape(out.shape)
    delta = W * (u * u + 4 * D * 2.0 ** -23 * A + 2.0 ** -19 + n * 2.0 ** -22) + n * 2.0 ** -25 * float(V.abs().max())
    if once:
        delta = delta + W * u
    err = (out.double() - ref).abs()
    over = err > delta + u * (ref.abs() + delta)
    assert not bool(over.any()), (int(over.sum()), float(err.max()), A)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 7, 17, 130])
@pytest.mark.parametrize("w,G", [(4, 8), (16, 2), (40, 8)])     # 32 query rows each, and 320: a second row tile
def test_positions_attended_together(n, w, G, dtype):
    R, Hkv, D, bs = (70 if w < 40 else 9), 2, 128, 16
    kc, vc, table, _ = make_pool([n] * R, Hkv, D, bs, dtype, DEV, n + w)
    g = torch.Generator(device=DEV).manual_seed(n)
    q = torch.randn((R * w, Hkv * G, D), device=DEV, generator=g).to(DTYPES[dtype])
    lens = torch.full((R * w,), n, dtype=torch.int32, device=DEV)
    out, tot = torch.empty_like(q), torch.zeros((R, Hkv, n), device=DEV)
    scale = D ** -0.5 / 16
    pa.pa_decode_weights(out, q, kc, vc, table.repeat_interleave(w, 0).contiguous(), lens, scale, n, tot, queries_per_row=w)
    torch.cuda.synchronize()
    check(out.view(R, w, Hkv * G, D), q.view(R, w, Hkv * G, D), kc, vc, table, n, scale, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size,G", [(3, 4), (16, 8), (33, 4), (80, 4)])   # 12, 128, 132 and 320 query rows
@pytest.mark.parametrize("blocks", [1, 9])
def test_a_common_prefix(blocks, size, G, dtype):
    groups, Hkv, D, bs = 8, 2, 128, 16
    n = blocks * bs
    kc, vc, table, _ = make_pool([n] * groups, Hkv, D, bs, dtype, DEV, n + size)
    g = torch.Generator(device=DEV).manual_seed(size)
    q = torch.randn((groups * size, Hkv * G, D), device=DEV, generator=g).to(DTYPES[dtype])
    lens = torch.full((groups * size,), n, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    scale = D ** -0.5 / 16
    pa.pa_decode_common_prefix(out, q, kc, vc, table.repeat_interleave(size, 0).contiguous(), lens, scale, n, size, blocks)
    torch.cuda.synchronize()
    check(out.view(groups, size, Hkv * G, D), q.view(groups, size, Hkv * G, D), kc, vc, table, n, scale, dtype, size * G > 128)
