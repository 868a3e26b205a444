"""Calls on two streams at once, with every round's outputs kept and compared: outputs
are made and filled before the streams start, and live until both have ended."""
import pytest
import torch

from tests import test_gpu_fp8_decode as dec
from tests import test_gpu_fp8_prefill as pre
from tests.test_gpu_fp8_decode import _built  # noqa: F401

pytestmark = pytest.mark.gpu


def both(a, b, run_a, run_b, rounds=20):
    """Outputs of ``rounds`` calls of either kind, on a stream each."""
    outs = [(torch.full_like(a["q"], float("nan")), torch.full_like(b["q"], float("nan"))) for _ in range(rounds)]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for oa, ob in outs:
        run_a(a, out=oa, stream=sa)
        run_b(b, out=ob, stream=sb)
    torch.cuda.synchronize()
    return outs


def test_two_decodes():
    a = dec.make([900, 33], 8, 1, 128, 16, "bf16", seed=31)
    b = dec.make([1200, 64, 7], 4, 1, 128, 16, "bf16", seed=32)
    wa, wb = dec.decode(a).clone(), dec.decode(b).clone()
    for oa, ob in both(a, b, dec.decode, dec.decode):
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_a_decode_beside_a_prompt_chunk():
    a = dec.make([900, 33], 8, 1, 128, 16, "bf16", seed=31)
    b = pre.make([300, 20], [64, 30], 8, 2, 16, "bf16", seed=11)
    wa, wb = dec.decode(a).clone(), pre.attend(b).clone()
    for oa, ob in both(a, b, dec.decode, pre.attend):
        assert torch.equal(oa, wa)
        # (merged in the order of the keys, whoever merges: the same bits)
        assert torch.equal(ob, wb)
