"""Decode over an 8-bit cache whose value blocks have scales far apart, up to all that the
write leaves (2^-64 to 2^120).  A key in a block of small values, or of zeros, counts for
the sum of weights as any other does.  Tolerances: the decode's test; scores and exponents
of scales are added up in fp32, off by up to 2^-17 where they reach 2^7, which enters as
2 ln(2) 2^-17 < 2^-16."""
import pytest
import torch

from tests import ref8
from tests.ref64 import half_step
from tests.test_gpu_fp8_decode import DEV, _built, decode, make  # noqa: F401

pytestmark = pytest.mark.gpu


def check(c, rows=None):
    out = decode(c).cpu().double()
    kv, vv = ref8.values(c["kc"], c["ks"]), ref8.values(c["vc"], c["vs"])
    for i, n in enumerate(c["lens"].tolist()):
        if rows is not None and i not in rows:
            continue
        want, mean, size = ref8.attend_sizes(c["q"][i].cpu().double(), ref8.rows_of(kv, c["bt"][i], n),
                                             ref8.rows_of(vv, c["bt"][i], n), c["scale"])
        D = want.shape[1]
        rel = 2 * (2 * (D + 8) * 2.0 ** -24 * size + 2.0 ** -22) + 2.0 ** -16 + 2.0 ** -12 + 2 * n * 2.0 ** -24 + 2.0 ** -20
        bound = want.abs() * half_step("bf16") * (1 + 2.0 ** -10) + mean * rel[:, None] + 2.0 ** -25
        assert bool(torch.isfinite(out[i]).all())
        assert bool(((out[i] - want).abs() <= bound).all()), (i, float(((out[i] - want).abs() / bound).max()))


@pytest.mark.parametrize("D,G", [(128, 1), (128, 8), (64, 4)])
@pytest.mark.parametrize("high", [40, 60, 75, 100, 119])
@pytest.mark.parametrize("zeros_first", [True, False])
def test_a_block_of_zeros_beside_one_of_large_values(D, G, high, zeros_first):
    c = make([32, 20], G, 1, D, 16, "bf16", seed=71, spread=0.0)
    c["kc"].view(torch.uint8).zero_()                       # every key alike
    t = c["bt"].long()
    vb, vc = c["vs"].view(torch.uint8), c["vc"].view(torch.uint8)
    vb[:] = 127 + high
    a = 0 if zeros_first else 1
    vb[t[:, a]] = 63
    vc[t[:, a]] = 0
    check(c)


@pytest.mark.parametrize("D,G", [(128, 2), (128, 8), (64, 1), (64, 8)])
@pytest.mark.parametrize("kind", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("copies", [1, 400])
def test_scales_over_their_whole_range(D, G, kind, copies):
    """Alone, where every piece is a CTA's and they are merged, and as many times as CTAs have whole rows."""
    n = 1400
    c = make([n], G, 1, D, 16, "bf16", seed=73, spread=0.0)
    t = c["bt"][0].long()
    j = torch.arange(t.shape[0], device=DEV)
    e = j * 183 // (t.shape[0] - 1) - 64
    if kind == "falling":
        e = e.flip(0)
    if kind == "mixed":
        e = torch.where(j % 3 == 0, -64, torch.where(j % 3 == 1, 119, j % 40))
    c["vs"].view(torch.uint8)[t, 0] = (127 + e).to(torch.uint8)
    if copies > 1:
        c["q"] = c["q"].repeat(copies, 1, 1)
        c["bt"] = c["bt"].repeat(copies, 1)
        c["lens"] = c["lens"].repeat(copies)
    check(c, rows=(0, 1, copies // 2, copies - 1))
