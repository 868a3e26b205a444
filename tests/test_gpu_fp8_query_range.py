"""Decode over an 8-bit cache: queries whose elements are of very different sizes.

Tolerance, by arithmetic: that of the decode's test, and what the query loses.  With
2^E <= the head's largest magnitude < 2^(E+1), each element enters as four e4m3 rows,
each the residual of those before times 2^5, over a power of two that brings the largest
to 2^7 .. 2^8.  An element is exact where its last bit is not below the last row's step,
2^-9 2^-15 2^(E-7) = 2^(E-31): from 2^(E-21) on in fp16 (10 bits after the first), from
2^(E-24) in bf16 (7 bits).  Below that it is off by half a step, 2^(E-32).  A score is
then off by at most scale 2^(E-32) sum |k_i| over the inexact elements, an output by twice
that times the weighted mean of |v|."""
import pytest
import torch

from tests import ref8
from tests.ref64 import half_step
from tests.test_gpu_fp8_decode import DEV, _built, decode, make  # noqa: F401

pytestmark = pytest.mark.gpu


def check(c, dtype):
    out = decode(c).cpu().double()
    kv, vv = ref8.values(c["kc"], c["ks"]), ref8.values(c["vc"], c["vs"])
    worst = 0.0
    for i, n in enumerate(c["lens"].tolist()):
        q = c["q"][i].cpu().double()
        K, V = ref8.rows_of(kv, c["bt"][i], n), ref8.rows_of(vv, c["bt"][i], n)
        want, mean, size = ref8.attend_sizes(q, K, V, c["scale"])
        _, e = torch.frexp(q.abs().amax(1))
        top = e - 1                                                      # E of each head
        lost = torch.zeros_like(size)
        for h in range(q.shape[0]):
            inexact = (q[h].abs() < 2.0 ** float(top[h] - (21 if dtype == "f16" else 24))).double()
            k = K[:, h // (q.shape[0] // K.shape[1])]
            lost[h] = float((k.abs() @ inexact).max()) * c["scale"] * 2.0 ** float(top[h] - 32)
        D = q.shape[1]
        rel = 2 * (2 * (D + 8) * 2.0 ** -24 * size + 2.0 ** -22 + lost) + 2.0 ** -12 + 2 * n * 2.0 ** -24 + 2.0 ** -20
        bound = want.abs() * half_step(dtype) * (1 + 2.0 ** -10) + mean * rel[:, None] + 2.0 ** -25
        worst = max(worst, float(((out[i] - want).abs() / bound).max()))
    assert worst <= 1, worst


@pytest.mark.parametrize("D,G", [(128, 1), (128, 4), (128, 8), (64, 2), (64, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("big", [100.0, 1000.0, 10000.0, -60000.0])
def test_one_large_element_beside_small_ones(D, G, dtype, big):
    """The large element meets zeros: the scores are what the small ones make of them."""
    c = make([2, 3, 17, 130, 700], 2 * G, 2, D, 16, dtype, seed=51 + D + G, qsize=0.02)
    c["q"][:, :, 5] = big
    c["q"][1, 0] *= 2.0 ** -6                # another head, another power of two
    c["kc"].view(torch.uint8)[..., 5] = 0
    c["scale"] = 8.0
    check(c, dtype)


@pytest.mark.parametrize("D,G", [(128, 4), (64, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_elements_of_all_sizes(D, G, dtype):
    """Elements over 14 octaves, keys as much the other way round: every dimension counts alike."""
    c = make([2, 40, 300], G, 1, D, 16, dtype, seed=61, qsize=4.0, spread=0.0)
    e = torch.arange(D, device=DEV) % 15
    c["q"] *= torch.exp2(-e.float()).to(c["q"].dtype)
    c["kc"].view(torch.uint8)[:] = (c["kc"].float() * torch.exp2(e.float() - 7)).to(torch.float8_e4m3fn).view(torch.uint8)
    check(c, dtype)
