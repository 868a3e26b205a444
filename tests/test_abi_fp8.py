"""Refusals of the head-norm and 8-bit-cache entry points: every check happens on the
host before anything is launched, so no GPU is needed."""
import ctypes

import numpy as np
import pytest

P = ctypes.c_void_p
BUF = 1 << 20
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_224_gb300 import build
    build.build()
    import paged_kv_cache_224_gb300 as pa
    return pa.lib()


ROTARY = dict(qo=BUF, qos=1024, q=BUF, qs=1024, k=BUF, ks=256, v=BUF, vs=256, kc=BUF, vc=2 * BUF, ksc=BUF, vsc=2 * BUF, pos=BUF,
              slot=BUF, inv=BUF, axis=None, A=1, R=128, qn=BUF, kn=BUF, eps=1e-6, T=4, Hq=8, Hkv=2, D=128, bs=16, NB=64, dt=1)


def norm(lib, **kw):
    a = {**ROTARY, **kw}
    ax = None if a["axis"] is None else np.asarray(a["axis"], np.int32).ctypes.data_as(P)
    return lib.pa_norm_rotary_and_cache(
        P(a["qo"]), a["qos"], P(a["q"]), a["qs"], P(a["k"]), a["ks"], P(a["v"]), a["vs"], P(a["kc"]), P(a["vc"]), P(a["pos"]),
        P(a["slot"]), P(a["inv"]), ax, a["A"], a["R"], 0, P(a["qn"]), P(a["kn"]), F(a["eps"]), a["T"], a["Hq"], a["Hkv"], a["D"],
        a["bs"], a["NB"], a["dt"], None, None)


def rotary8(lib, **kw):
    a = {**ROTARY, **kw}
    ax = None if a["axis"] is None else np.asarray(a["axis"], np.int32).ctypes.data_as(P)
    return lib.pa_rotary_and_cache_fp8(
        P(a["qo"]), a["qos"], P(a["q"]), a["qs"], P(a["k"]), a["ks"], P(a["v"]), a["vs"], P(a["kc"]), P(a["vc"]), P(a["ksc"]),
        P(a["vsc"]), P(a["pos"]), P(a["slot"]), P(a["inv"]), ax, a["A"], a["R"], 0, P(a["qn"]), P(a["kn"]), F(a["eps"]), a["T"],
        a["Hq"], a["Hkv"], a["D"], a["bs"], a["NB"], a["dt"], None, None)


@pytest.mark.parametrize("call", [norm, rotary8])
def test_rotary_refusals(lib, call):
    assert call(lib, T=0) == 0
    assert call(lib, T=-1) == -1 and call(lib, Hq=0) == -1 and call(lib, A=0) == -1 and call(lib, dt=5) == -1
    for name in ("qo", "q", "k", "v", "kc", "vc", "pos", "slot", "inv"):
        assert call(lib, **{name: 0}) == -1, name
    assert call(lib, qn=0) == -1 and call(lib, kn=0) == -1      # one norm without the other
    assert call(lib, eps=-1e-9) == -3 and call(lib, eps=float("nan")) == -3 and call(lib, eps=float("inf")) == -3
    assert call(lib, D=120, R=112) == -2                        # heads in units of 16 values
    assert call(lib, R=24) == -2 and call(lib, A=9) == -2
    assert call(lib, D=272, R=128, qs=8192, qos=8192, ks=1024, vs=1024) == -2
    assert call(lib, D=64, R=128) == -3
    assert call(lib, axis=[0] * 63 + [1]) == -3
    assert call(lib, qs=1016) == -3 and call(lib, ks=0) == -3
    assert call(lib, qs=1028) == -6 and call(lib, v=BUF + 8) == -6 and call(lib, kn=BUF + 2) == -6


def test_norms_are_required_where_they_are_the_point(lib):
    assert norm(lib, qn=0, kn=0) == -1


def test_store_refusals(lib):
    assert rotary8(lib, bs=5) == -2 and rotary8(lib, bs=256) == -2
    assert rotary8(lib, Hkv=65536, D=16, R=16, ks=1 << 20, vs=1 << 20) == -2
    assert rotary8(lib, ksc=0) == -1 and rotary8(lib, vsc=0) == -1
    assert rotary8(lib, vsc=BUF) == -1 and rotary8(lib, vc=BUF) == -1     # one buffer for both

    def plain(k=BUF, v=BUF, kc=BUF, vc=2 * BUF, ks=BUF, vs=2 * BUF, slot=BUF, T=4, H=2, D=128, bs=16, NB=64, dt=1):
        return lib.pa_reshape_and_cache_fp8(P(k), P(v), P(kc), P(vc), P(ks), P(vs), P(slot), T, H, D, bs, NB, dt, None, None)
    assert plain(T=0) == 0 and plain(T=-1) == -1 and plain(H=0) == -1 and plain(D=0) == -1 and plain(NB=0) == -1
    for name in ("k", "v", "kc", "vc", "ks", "vs", "slot"):
        assert plain(**{name: 0}) == -1, name
    assert plain(D=24) == -2 and plain(bs=12) == -2 and plain(dt=2) == -1 and plain(k=BUF + 2) == -6 and plain(vs=BUF) == -1


def decode(lib, out=BUF, q=BUF, kc=BUF, vc=BUF, ks=BUF, vs=BUF, bt=BUF, mb=8, lens=BUF, B=4, Hq=8, Hkv=2, D=128, bs=16, NB=64,
           ml=100, scale=0.1, dt=1, ws=BUF, wsb=1 << 30):
    return lib.pa_decode_fp8(P(out), P(q), P(kc), P(vc), P(ks), P(vs), P(bt), mb, P(lens), B, Hq, Hkv, D, bs, NB, ml, F(scale),
                             dt, P(ws), wsb, None, None)


def test_decode_refusals(lib):
    assert decode(lib, B=0) == 0 and decode(lib, B=-1) == -1
    for name in ("out", "q", "kc", "vc", "ks", "vs", "bt", "lens"):
        assert decode(lib, **{name: 0}) == -1, name
    assert decode(lib, Hq=7) == -1 and decode(lib, dt=9) == -1 and decode(lib, mb=0) == -1 and decode(lib, ml=-1) == -1
    assert decode(lib, D=96) == -2 and decode(lib, bs=24) == -2 and decode(lib, Hq=32) == -2 and decode(lib, Hq=6) == -2
    assert decode(lib, mb=1 << 28) == -2                    # a table of 2^32 tokens
    assert decode(lib, NB=1 << 27) == -2                    # a pool of 2^32 rows
    assert decode(lib, B=1 << 29) == -2
    assert decode(lib, scale=float("inf")) == -3
    assert decode(lib, q=BUF + 2) == -6 and decode(lib, kc=BUF + 8) == -6
    # contexts of a single tile are never cut
    assert lib.pa_decode_fp8_workspace_bytes(4, 8, 2, 128, 16, 128) == 0
    # 4 sequences of 2 tiles, 2 kv heads: 16 CTAs, two partials each of 4 heads
    need = lib.pa_decode_fp8_workspace_bytes(4, 8, 2, 128, 16, 200)
    assert need == 4096 + 2 * 16 * 4 * (128 + 2) * 4
    assert decode(lib, ml=200, ws=0) == -5 and decode(lib, ml=200, wsb=need - 1) == -5
    assert decode(lib, ml=200, ws=BUF + 16) == -6
    # two CTAs to each of (without a device) 152 SMs, however large the batch
    assert lib.pa_decode_fp8_workspace_bytes(256, 32, 8, 128, 16, 4096) == 4096 + 2 * 304 * 4 * (128 + 2) * 4
    assert lib.pa_decode_fp8_workspace_bytes(4, 7, 2, 128, 16, 200) == 0
    assert lib.pa_decode_fp8_workspace_bytes(4, 8, 2, 128, 24, 200) == 0


def prefill(lib, out=BUF, q=BUF, kc=BUF, vc=BUF, ks=BUF, vs=BUF, bt=BUF, mb=8, prefix=(64, 0), chunk=(20, 30), Hq=8, Hkv=2, D=128,
            bs=16, NB=64, scale=0.1, dt=1, ws=BUF, wsb=1 << 40):
    a, b = (np.asarray(x, np.int32) for x in (prefix, chunk))
    return lib.pa_prefill_batch_fp8(P(out), P(q), P(kc), P(vc), P(ks), P(vs), P(bt), mb, a.ctypes.data, b.ctypes.data, a.size, Hq,
                                    Hkv, D, bs, NB, F(scale), dt, P(ws), wsb, None, None)


def prefill_bytes(lib, prefix, chunk, Hq=8, Hkv=2, D=128, bs=16):
    a, b = (np.asarray(x, np.int32) for x in (prefix, chunk))
    return lib.pa_prefill_batch_fp8_workspace_bytes(a.ctypes.data, b.ctypes.data, a.size, Hq, Hkv, D, bs)


def test_prefill_refusals(lib):
    assert prefill(lib, prefix=(), chunk=()) == 0 and prefill(lib, chunk=(0, 0)) == 0
    for name in ("out", "q", "kc", "vc", "ks", "vs", "bt"):
        assert prefill(lib, **{name: 0}) == -1, name
    assert prefill(lib, chunk=(-1, 3)) == -1 and prefill(lib, prefix=(-1, 3)) == -1 and prefill(lib, Hq=7) == -1
    assert prefill(lib, chunk=(65, 1)) == -3                # past the table
    assert prefill(lib, prefix=(2 ** 31 - 1, 0)) == -3
    assert prefill(lib, scale=0.0) == -3 and prefill(lib, scale=-0.1) == -3
    assert prefill(lib, D=64) == -2 and prefill(lib, bs=8, mb=16) == -2 and prefill(lib, Hq=32) == -2
    need = prefill_bytes(lib, (64, 0), (20, 30))
    pre = lib.pa_prefill_workspace_bytes(2, 50, 8, 2, 128)
    assert need == pre + 256 + 2 * 8 * 2 * 16 * 128 * 2     # 6 + 2 blocks, K and V
    assert prefill(lib, ws=0) == -5 and prefill(lib, wsb=need - 1) == -5 and prefill(lib, ws=BUF + 64) == -6
    assert prefill(lib, kc=BUF + 4) == -6
    assert prefill_bytes(lib, (64, 0), (20, -1)) == 0 and prefill_bytes(lib, (64, 0), (20, 1), Hq=7) == 0


def test_copy_refusals(lib):
    ws = lib.pa_copy_blocks_workspace_bytes(3)

    def copy(kc=BUF, vc=BUF, ks=BUF, vs=BUF, pairs=BUF, n=3, H=2, D=128, bs=16, NB=64, w=BUF, wb=ws):
        return lib.pa_copy_blocks_fp8(P(kc), P(vc), P(ks), P(vs), P(pairs), n, H, D, bs, NB, P(w), wb, None, None)
    assert copy(n=0) == 0 and copy(n=-1) == -1 and copy(n=(1 << 26) + 1, wb=1 << 40) == -3
    for name in ("kc", "vc", "ks", "vs", "pairs"):
        assert copy(**{name: 0}) == -1, name
    assert copy(H=1, D=3, bs=2) == -2 and copy(w=0) == -5 and copy(wb=ws - 1) == -5 and copy(w=BUF + 8) == -6
    assert copy(kc=BUF + 8) == -6
