"""Head norms at the ends of the range that they are stated for: root mean squares just
below 2^59, and just above 2^-50 or anything beside an eps of 2^-80 and more.  Tolerances:
those of the head norms' and the 8-bit write's tests."""
import pytest
import torch

from tests import test_gpu_fp8_store as store
from tests import test_gpu_norm_rotary as norm
from tests.test_gpu_norm_rotary import _built  # noqa: F401

pytestmark = pytest.mark.gpu
RANGES = [(1e-6, [58, 40, 0, -20, -100]), (0.0, [58, 0, -30, -49]), (2.0 ** -80, [58, -39, -41, -60, -120])]


def spread(x, exponents):
    """Heads of N(0, 1) times powers of two in turn."""
    g = torch.Generator().manual_seed(3)
    e = torch.tensor(exponents, dtype=torch.float64)[torch.arange(x.shape[0] * x.shape[1]) % len(exponents)]
    y = torch.randn(x.shape, generator=g).double().clamp(-3.5, 3.5) * torch.exp2(e.view(x.shape[0], x.shape[1], 1))
    x.copy_(y.to(torch.bfloat16))


@pytest.mark.parametrize("D,R,interleaved", [(128, 128, False), (64, 32, True), (256, 0, False)])
@pytest.mark.parametrize("eps,exponents", RANGES)
def test_heads_of_all_sizes(D, R, interleaved, eps, exponents):
    c = norm.make(37, 5, 3, D, R, 2, 16, "bf16", seed=D + R)
    spread(c["q"], exponents)
    spread(c["k"], exponents[::-1])
    norm.check(c, R, interleaved, "bf16", eps=eps)


@pytest.mark.parametrize("T,kind", [(40, "run"), (3, "step")])
@pytest.mark.parametrize("eps,exponents", RANGES)
def test_in_the_8_bit_write(T, kind, eps, exponents):
    c = store.make(T, 4, 3, 128, 128, "bf16", 16, kind, seed=7, norm=True)
    c["eps"] = eps
    spread(c["q"], exponents)
    spread(c["k"], exponents[::-1])
    store.check(c, 128, False, "bf16")
