"""Host lengths of prompt chunks that are no 32-bit whole numbers are refused, whatever they
come in; none is cut down to one that is."""
import numpy as np
import pytest
import torch

from paged_kv_cache_224_gb300 import capi


def test_lengths_past_32_bits():
    for bad in ([2 ** 31], np.asarray([2 ** 32 + 5]), torch.tensor([2 ** 32]), [-2 ** 31 - 1], np.asarray([2 ** 63], np.uint64),
                [1.5], np.asarray([0.5])):
        for a, b in ((bad, [1]), ([1], bad)):
            with pytest.raises((ValueError, OverflowError, TypeError)):
                capi._lens32(a, b)
    pl, cl = capi._lens32(torch.tensor([5, 2 ** 31 - 1]), np.asarray([7, 0], np.int64))
    assert pl.dtype == np.int32 and pl.tolist() == [5, 2 ** 31 - 1] and cl.tolist() == [7, 0]
    pl, cl = capi._lens32([], [])
    assert pl.dtype == np.int32 and pl.size == 0 == cl.size
