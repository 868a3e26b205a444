"""Refusals of the bounded- and shared-cache entry points: every check happens
on the host before anything is launched, so no GPU is needed."""
import ctypes

import numpy as np
import pytest
import torch

P = ctypes.c_void_p
BUF = 1 << 20
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_224_gb300 import build
    build.build()
    import paged_kv_cache_224_gb300 as pa
    return pa.lib()


def rotary(lib, qo=BUF, qos=1024, q=BUF, qs=1024, k=BUF, ks=256, v=BUF, vs=256, kc=BUF, vc=BUF, pos=BUF, slot=BUF,
           inv=BUF, axis=None, A=1, R=128, T=4, Hq=8, Hkv=2, D=128, bs=16, NB=64, dt=1):
    ax = None if axis is None else np.asarray(axis, np.int32).ctypes.data_as(P)
    return lib.pa_rotary_and_cache(P(qo), qos, P(q), qs, P(k), ks, P(v), vs, P(kc), P(vc), P(pos), P(slot), P(inv), ax,
                                   A, R, 0, T, Hq, Hkv, D, bs, NB, dt, None, None)


def test_rotary_refusals(lib):
    assert rotary(lib, T=0) == 0
    assert rotary(lib, T=-1) == -1 and rotary(lib, Hq=0) == -1 and rotary(lib, A=0) == -1 and rotary(lib, dt=5) == -1
    for name in ("qo", "q", "k", "v", "kc", "vc", "pos", "slot", "inv"):
        assert rotary(lib, **{name: 0}) == -1, name
    assert rotary(lib, D=120, R=112) == -2          # heads in units of 16 values
    assert rotary(lib, R=24) == -2
    assert rotary(lib, D=272, R=128, qs=8192, qos=8192, ks=1024, vs=1024) == -2
    assert rotary(lib, A=9) == -2
    assert rotary(lib, D=64, R=128) == -3           # more rotated dimensions than the head has
    assert rotary(lib, axis=[0] * 63 + [1]) == -3   # an axis that positions does not have
    assert rotary(lib, axis=[-1] + [0] * 63, A=2) == -3
    assert rotary(lib, qs=1016) == -3               # rows that overlap
    assert rotary(lib, ks=0) == -3
    assert rotary(lib, qs=1028) == -6 and rotary(lib, v=BUF + 8) == -6


def weights(lib, out=BUF, q=BUF, k=BUF, v=BUF, bt=BUF, mb=8, lens=BUF, B=4, Hq=8, Hkv=2, D=128, bs=16, NB=64, ml=100,
            scale=0.1, pt=0, w=BUF, wo=BUF, W=100, qpr=1, dt=1, ws=BUF, wsb=1 << 30):
    return lib.pa_decode_weights(P(out), P(q), P(k), P(v), P(bt), mb, P(lens), B, Hq, Hkv, D, bs, NB, ml, F(scale), pt,
                                 P(w), P(wo), W, qpr, dt, P(ws), wsb, None, None)


def test_decode_weights_refusals(lib):
    assert weights(lib, B=0) == 0
    for name in ("out", "q", "k", "v", "bt", "lens", "w", "wo"):
        assert weights(lib, **{name: 0}) == -1, name
    assert weights(lib, Hq=7) == -1 and weights(lib, qpr=0) == -1 and weights(lib, qpr=3) == -1
    assert weights(lib, W=99) == -3                  # a row of totals shorter than the contexts
    assert weights(lib, scale=float("nan")) == -3 and weights(lib, pt=24) == -3 and weights(lib, pt=-16) == -3
    assert weights(lib, D=96) == -2 and weights(lib, bs=24) == -2 and weights(lib, Hq=32) == -2
    assert weights(lib, q=BUF + 2) == -6
    assert weights(lib, wo=BUF + 4) == -1            # overlapping, but not the same
    need = lib.pa_decode_weights_workspace_bytes(4, 8, 2, 128, 16, 100, 1, 0)
    # (max, sum) pairs of 32 (sequence, head)s, then 100 scores each
    assert need == 256 + 4 * 8 * 100 * 4
    assert weights(lib, ws=0) == -5 and weights(lib, wsb=need - 1) == -5
    assert weights(lib, ws=BUF + 16) == -6
    assert lib.pa_decode_weights_workspace_bytes(4, 7, 2, 128, 16, 100, 1, 0) == 0
    assert lib.pa_decode_weights_workspace_bytes(4, 8, 2, 128, 16, 100, 1, 24) == 0
    assert lib.pa_decode_weights_workspace_bytes(4, 8, 2, 128, 16, 100, 3, 0) == 0
    # four positions of four heads are attended together: one piece of 128 values and (max, sum) each, and
    # 128 scores for each of two kv heads' 16 query rows, rounded up to 32
    assert lib.pa_decode_weights_workspace_bytes(4, 8, 2, 128, 16, 100, 4, 0) == 4 * 8 * (128 + 2) * 4 + 2 * 32 * 128 * 4
    assert weights(lib, qpr=4, scale=-0.1) == -3 and weights(lib, qpr=4, pt=24) == -3


def evict(lib, k=BUF, v=BUF, w=BUF, nw=2 * BUF, W=100, bt=BUF, mb=8, lens=BUF, nbt=BUF, nmb=4, nl=2 * BUF, kept=BUF, B=2,
          Hkv=2, D=128, bs=16, NB=64, ml=100, keep=48, sink=4, recent=8, dt=1, ws=BUF, wsb=1 << 20):
    return lib.pa_evict(P(k), P(v), P(w), P(nw), W, P(bt), mb, P(lens), P(nbt), nmb, P(nl), P(kept), B, Hkv, D, bs, NB,
                        ml, keep, sink, recent, dt, P(ws), wsb, None, None)


def test_evict_refusals(lib):
    assert evict(lib, B=0) == 0
    for name in ("k", "v", "w", "nw", "bt", "lens", "nbt", "nl", "kept"):
        assert evict(lib, **{name: 0}) == -1, name
    assert evict(lib, keep=0) == -1 and evict(lib, sink=-1) == -1 and evict(lib, recent=-1) == -1
    assert evict(lib, sink=40, recent=9) == -3       # more protected tokens than are kept
    assert evict(lib, W=99) == -3
    assert evict(lib, nmb=2) == -3                   # 32 rows cannot hold 48
    assert evict(lib, D=96) == -2 and evict(lib, bs=24, nmb=8) == -2
    assert evict(lib, k=BUF + 8) == -6
    assert evict(lib, nw=BUF) == -1 and evict(lib, nw=BUF + 4) == -1   # the totals cannot be moved in place
    assert evict(lib, nl=BUF) == -1
    assert lib.pa_evict_workspace_bytes(64) == 256 and lib.pa_evict_workspace_bytes(0) == 0
    assert evict(lib, ws=0) == -5 and evict(lib, wsb=255) == -5 and evict(lib, ws=BUF + 4) == -6


def prefix(lib, out=BUF, q=BUF, k=BUF, v=BUF, bt=BUF, mb=8, lens=BUF, B=12, size=6, pb=2, Hq=8, Hkv=2, D=128, bs=16,
           NB=64, ml=100, scale=0.1, pt=0, dt=1, ws=BUF, wsb=1 << 30):
    return lib.pa_decode_common_prefix(P(out), P(q), P(k), P(v), P(bt), mb, P(lens), B, size, pb, Hq, Hkv, D, bs, NB, ml,
                                       F(scale), pt, dt, P(ws), wsb, None, None)


def test_common_prefix_refusals(lib):
    assert prefix(lib, B=0) == 0
    for name in ("out", "q", "k", "v", "bt", "lens"):
        assert prefix(lib, **{name: 0}) == -1, name
    assert prefix(lib, size=5) == -1 and prefix(lib, size=0) == -1 and prefix(lib, pb=0) == -1 and prefix(lib, Hq=7) == -1
    assert prefix(lib, pb=7) == -3 and prefix(lib, pb=9, ml=1000) == -3     # longer than the contexts, than the table
    assert prefix(lib, scale=0.0) == -3 and prefix(lib, scale=-1.0) == -3 and prefix(lib, pt=24) == -3
    assert prefix(lib, D=64) == -2 and prefix(lib, bs=8) == -2 and prefix(lib, Hq=32) == -2
    assert prefix(lib, k=BUF + 8) == -6
    need = lib.pa_decode_common_prefix_workspace_bytes(12, 8, 2, 128, 16, 100, 6, 2, 0)
    # 2 groups x 2 kv heads x one row tile of one key tile: one piece each, and one partition of own tokens;
    # before them the queue's counter
    assert need == 12 * 8 * 2 * (128 + 2) * 4 + 256
    assert prefix(lib, ws=0) == -5 and prefix(lib, wsb=need - 1) == -5 and prefix(lib, ws=BUF + 16) == -6
    assert lib.pa_decode_common_prefix_workspace_bytes(12, 8, 2, 128, 16, 100, 5, 2, 0) == 0
    assert lib.pa_decode_common_prefix_workspace_bytes(12, 8, 2, 128, 16, 100, 6, 7, 0) == 0


def test_python_checks_come_before_the_library():
    import paged_kv_cache_224_gb300 as pa
    t = torch.zeros(4)
    with pytest.raises(ValueError):
        pa.pa_rotary_and_cache(t, t, t, t, t, t, t, t, t)      # not on a CUDA device
    with pytest.raises(ValueError):
        pa.pa_decode_weights(t, t, t, t, t, t, 1.0, 4, t)
    with pytest.raises(ValueError):
        pa.pa_evict(t, t, t, t, t, t, t, t, t, 4, 0, 0, 4)
    with pytest.raises(ValueError):
        pa.pa_decode_common_prefix(t, t, t, t, t, t, 1.0, 4, 1, 1)


# ---- the block manager's side of an eviction ----------------------------------

def test_evicted_sequence_moves_to_fresh_private_blocks(lib):
    import paged_kv_cache_224_gb300 as pa
    m = pa.BlockManager(16, 4)
    m.add_sequence(1, list(range(18)))               # 5 blocks, 4 of them full: in the prefix tree
    m.fork(1, 2)
    old = m.block_table(1)
    m.evict_sequence(1, 7)
    new = m.block_table(1)
    assert m.seq_len(1) == 7 and len(new) == 2 and not set(new) & set(old)
    assert list(m.block_table(2)) == list(old)       # the sibling's table is as it was
    assert all(m.refcount(int(b)) == 1 for b in list(new) + list(old))
    # it goes on growing, in its own block, and its blocks never join the prefix tree
    slots = [m.append_token(1, 100 + i) for i in range(9)]
    assert slots[0][0] == int(new[1]) * 4 + 3 and all(pair is None for _, pair in slots)
    m.free_sequence(1)
    s = m.stats()
    assert s["cached_free_blocks"] == 0 and s["used_blocks"] == 5
    # a prompt equal to the tokens it was given finds nothing of it
    _, cached = m.add_sequence(3, [0, 1, 2, 3] + [100, 101])
    assert cached == 4                               # the shared prefix of sequence 2 alone


def test_evict_sequence_refusals_change_nothing(lib):
    import paged_kv_cache_224_gb300 as pa
    m = pa.BlockManager(6, 4, prefix_cache=False)
    m.add_sequence(1, list(range(16)))               # 4 of 6 blocks
    table = list(m.block_table(1))
    for bad, status in ((17, -3), (-1, -3), (12, -8)):   # longer than it is, negative, no three free blocks
        with pytest.raises(pa.PAError) as e:
            m.evict_sequence(1, bad)
        assert e.value.status == status
        assert list(m.block_table(1)) == table and m.seq_len(1) == 16 and m.stats()["free_blocks"] == 2
    with pytest.raises(pa.PAError):
        m.evict_sequence(9, 0)
    m.evict_sequence(1, 8)
    assert m.seq_len(1) == 8 and m.stats()["free_blocks"] == 4
    m.evict_sequence(1, 0)
    assert m.seq_len(1) == 0 and m.stats()["free_blocks"] == 6 and len(m.block_table(1)) == 0
