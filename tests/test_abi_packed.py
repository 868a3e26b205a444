"""Arguments of the packed calls that do not fit their types are refused: cut down to 32
bits, 2^32 tokens would be none.  Nothing is launched, so no GPU is needed."""
import struct

import pytest

BUF = 1 << 20
# (call, layout, good arguments, positions of the ints); good arguments describe a call
# without work, which returns 0
CALLS = {
    "norm": (0, "=19qd9q", [BUF, 1024, BUF, 1024, BUF, 256, BUF, 256, BUF, 2 * BUF, BUF, BUF, BUF, 0, 1, 128, 0, BUF, BUF, 1e-6,
                            0, 8, 2, 128, 16, 64, 1, 0, 0], [14, 15, 16, 20, 21, 22, 23, 24, 25, 26]),
    "rotary8": (1, "=21qd9q", [BUF, 1024, BUF, 1024, BUF, 256, BUF, 256, BUF, 2 * BUF, BUF, 2 * BUF, BUF, BUF, BUF, 0, 1, 128, 0,
                               BUF, BUF, 1e-6, 0, 8, 2, 128, 16, 64, 1, 0, 0], [16, 17, 18, 22, 23, 24, 25, 26, 27, 28]),
    "reshape8": (2, "=15q", [BUF, BUF, BUF, 2 * BUF, BUF, 2 * BUF, BUF, 0, 2, 128, 16, 64, 1, 0, 0], [7, 8, 9, 10, 11, 12]),
    "decode8": (3, "=16qd5q", [BUF] * 7 + [8, BUF, 0, 8, 2, 128, 16, 64, 100, 0.1, 1, BUF, 1 << 30, 0, 0],
                [7, 9, 10, 11, 12, 13, 14, 15, 17]),
    "prefill8": (4, "=16qd5q", [BUF] * 7 + [8, BUF, BUF, 0, 8, 2, 128, 16, 64, 0.1, 1, BUF, 1 << 30, 0, 0],
                 [7, 10, 11, 12, 13, 14, 15, 17]),
    "copy8": (5, "=14q", [BUF] * 5 + [0, 2, 128, 16, 64, BUF, 1 << 30, 0, 0], [5, 6, 7, 8, 9]),
}


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_224_gb300 import build
    build.build()
    import paged_kv_cache_224_gb300 as pa
    return pa.lib()


@pytest.mark.parametrize("name", list(CALLS))
def test_numbers_past_32_bits(lib, name):
    number, layout, args, ints = CALLS[name]

    def call(a):
        return lib.pa_call_packed(number, struct.pack(layout, *a))
    assert call(args) == 0
    for i in ints:
        for past in (1 << 32, -(1 << 32), 1 << 40):
            a = list(args)
            a[i] += past
            assert call(a) == -3, (i, past)


def test_unknown_calls(lib):
    assert lib.pa_call_packed(6, b"\0" * 256) == -1 and lib.pa_call_packed(-1, b"\0" * 256) == -1
    assert lib.pa_call_packed(0, None) == -1
