"""Prompt chunks over an 8-bit cache whose value blocks have scales far apart, up to all that
the write leaves: a key in a block of small values, or of zeros, counts for the sum of
weights as any other does, whether a unit is one CTA's or merged of several.  Tolerances:
the prompt chunks' test (weights rounded once to the type, which is more than they are),
and 2 ln(2) 2^-17 < 2^-16 for scores and exponents added up in fp32."""
import pytest
import torch

from tests import ref8
from tests.ref64 import half_step
from tests.test_gpu_fp8_prefill import DEV, _built, attend, make  # noqa: F401

pytestmark = pytest.mark.gpu


def check(c, rows):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = attend(c, err).cpu().double()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    kv, vv = ref8.values(c["kc"], c["ks"]), ref8.values(c["vc"], c["vs"])
    at, h = 0, half_step("bf16")
    for i, (p, n) in enumerate(zip(c["prefixes"], c["chunks"])):
        K, V = ref8.rows_of(kv, c["bt"][i], p + n), ref8.rows_of(vv, c["bt"][i], p + n)
        for r in sorted({x % n for x in rows}):
            m = p + r + 1
            want, mean, size = ref8.attend_sizes(c["q"][at + r].cpu().double(), K[:m], V[:m], c["scale"])
            rel = h + 2 * (2 * (128 + 8) * 2.0 ** -24 * size + 2.0 ** -22) + 2.0 ** -16 + 2 * m * 2.0 ** -24 + 2.0 ** -20
            bound = want.abs() * h * (1 + 2.0 ** -10) + mean * rel[:, None] + 2.0 ** -25
            assert bool(torch.isfinite(out[at + r]).all())
            e = (out[at + r] - want).abs() / bound
            assert bool((e <= 1).all()), (i, r, float(e.max()))
        at += n


def exponents(kind, blocks):
    j = torch.arange(blocks, device=DEV)
    e = j * 183 // max(1, blocks - 1) - 64
    if kind == "falling":
        e = e.flip(0)
    if kind == "mixed":
        e = torch.where(j % 3 == 0, -64, torch.where(j % 3 == 1, 119, j % 40))
    return (127 + e).to(torch.uint8)


@pytest.mark.parametrize("G,bs", [(1, 16), (8, 32), (4, 128)])
@pytest.mark.parametrize("kind", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("prefix,chunk", [(2300, 3), (0, 1500), (700, 200)])
def test_scales_over_their_whole_range(G, bs, kind, prefix, chunk):
    c = make([prefix], [chunk], G, 1, bs, "bf16", seed=83, spread=0.0, poison=True)
    t = c["bt"][0].long()
    c["vs"].view(torch.uint8)[t, 0] = exponents(kind, t.shape[0])
    check(c, (0, 1, 15, 16, 17, 31, 127, 128, 200, 511, 900, -1))


@pytest.mark.parametrize("high", [40, 60, 75, 100, 119])
@pytest.mark.parametrize("zeros_first", [True, False])
def test_a_block_of_zeros_beside_one_of_large_values(high, zeros_first):
    c = make([30, 0], [10, 32], 2, 1, 16, "bf16", seed=84, spread=0.0)
    c["kc"].view(torch.uint8).zero_()                       # every key alike
    t = c["bt"].long()
    vb, vc = c["vs"].view(torch.uint8), c["vc"].view(torch.uint8)
    vb[:] = 127 + high
    a = 0 if zeros_first else 1
    vb[t[:, a]] = 63
    vc[t[:, a]] = 0
    check(c, range(32))


def test_nan_in_a_value_that_is_seen():
    c = make([20], [40], 2, 1, 16, "bf16", seed=85)
    c["vc"].view(torch.uint8)[c["bt"][0, 2].long(), 0, 8, 7] = 0x7f        # key 40, first seen by row 20
    out = attend(c)
    nan = torch.isnan(out.float())
    # (rows of one unit share the tile's product, and a weight of 0 times NaN is NaN)
    assert bool(nan[20:, :, 7].all())
    nan[:, :, 7] = False
    assert not bool(nan.any())
    c["vs"].view(torch.uint8)[c["bt"][0, 2].long()] = 255
    assert bool(torch.isnan(attend(c)[20:].float()).all())


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("apart", [22, 9])
def test_small_values_beside_large_ones_of_their_tile(bs, apart):
    """Exact down to 2^-22 of the greatest scale among 128 keys, whoever sees those; off by 2^-32 of it below."""
    c = make([0, 128], [128, 128], 2, 1, bs, "bf16", seed=86, spread=0.0)
    t = c["bt"].long()
    vb = c["vs"].view(torch.uint8)
    vb[:] = 127 + 100
    vb[t[0, 0]] = vb[t[1, 128 // bs]] = 127 + 100 - apart
    check(c, range(0, 128, 5))
    vb[t[0, 0]] = 127 + 100 - 40
    out = attend(c)[:bs].double().cpu()
    kv, vv = ref8.values(c["kc"], c["ks"]), ref8.values(c["vc"], c["vs"])
    for r in range(0, bs, 3):
        K, V = ref8.rows_of(kv, c["bt"][0], r + 1), ref8.rows_of(vv, c["bt"][0], r + 1)
        want, mean, _ = ref8.attend_sizes(c["q"][r].cpu().double(), K, V, c["scale"])
        assert bool(((out[r] - want).abs() <= 2.0 ** 68 + (mean + 2.0 ** 68) * (2 * half_step("bf16"))).all())
