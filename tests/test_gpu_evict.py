"""pa_evict against a plain selection on the host: which tokens stay, where
their rows and totals go, and everything else left as it was.  All of it is
exact: rows and totals move, nothing is computed."""
import numpy as np
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.ref64 import evict_choice, make_pool

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def setup(lens, keep, sink, recent, Hkv, D, bs, dtype, seed, width=None, values="ties"):
    kc, vc, old, new = make_pool(lens, Hkv, D, bs, dtype, DEV, seed, extra=[min(n, keep) for n in lens])
    rng = np.random.default_rng(seed)
    W = width or max(max(lens), 1)
    shape = (len(lens), Hkv, W)
    if values == "ties":
        w = rng.integers(0, 7, size=shape).astype(np.float32) / 4
    elif values == "equal":
        w = np.full(shape, 0.125, np.float32)
    elif values == "odd":   # negatives, both zeros, infinities, subnormals, NaN of either sign
        pick = np.array([-1.5, -0.0, 0.0, np.inf, -np.inf, 1e-40, -1e-40, np.nan, -np.nan, 2.0], np.float32)
        w = pick[rng.integers(0, len(pick), size=shape)]
    else:
        w = rng.random(shape).astype(np.float32) ** 8
    return dict(kc=kc, vc=vc, old=old, new=new, lens=lens, keep=keep, sink=sink, recent=recent, w=w, W=W, bs=bs, Hkv=Hkv)


def call(c, **kw):
    B = len(c["lens"])
    w = torch.as_tensor(c["w"], device=DEV)
    kept = torch.full((B, c["Hkv"], c["keep"]), 123, dtype=torch.int32, device=DEV)
    nl = torch.full((B,), 123, dtype=torch.int32, device=DEV)
    nw = torch.full_like(w, -7.0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_evict(c["kc"], c["vc"], w, c["old"], torch.as_tensor(c["lens"], dtype=torch.int32, device=DEV), c["new"], nl,
                nw, kept, c["keep"], c["sink"], c["recent"], c["W"], d_err=err, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(w.cpu().numpy(), c["w"], equal_nan=True)
    return kept.cpu().numpy(), nl.cpu().numpy(), nw.cpu().numpy(), int(err.item())


def check(c, skip=()):
    """Everything as the plain selection says; sequences in ``skip`` write nothing."""
    k0, v0 = c["kc"].clone(), c["vc"].clone()
    kept, nl, nw, err = call(c)
    bs = c["bs"]
    old, new = c["old"].cpu().numpy(), c["new"].cpu().numpy()
    for s, n in enumerate(c["lens"]):
        m = min(n, c["keep"])
        assert nl[s] == m
        for h in range(c["Hkv"]):
            idx = evict_choice(c["w"][s, h], n, c["keep"], c["sink"], c["recent"])
            assert list(kept[s, h, :m]) == idx, (s, h)
            assert (kept[s, h, m:] == -1).all()
            assert np.array_equal(nw[s, h, :m], c["w"][s, h, idx], equal_nan=True) and (nw[s, h, m:] == 0).all()
            if s in skip or not m:
                continue
            j = np.asarray(idx)
            src = torch.as_tensor(old[s, j // bs].astype(np.int64), device=DEV), torch.as_tensor(j % bs, device=DEV)
            i = np.arange(m)
            dst = torch.as_tensor(new[s, i // bs].astype(np.int64), device=DEV), torch.as_tensor(i % bs, device=DEV)
            k0[dst[0], h, dst[1]] = k0[src[0], h, src[1]]
            v0[dst[0], h, dst[1]] = v0[src[0], h, src[1]]
    assert torch.equal(k0.view(torch.int16), c["kc"].view(torch.int16))
    assert torch.equal(v0.view(torch.int16), c["vc"].view(torch.int16))
    return err


CASES = [
    ([90, 17, 64, 200, 33, 5, 0, 120], 40, 2, 9, 2, 64, 16, "bf16", "random"),
    # (lens, keep, sink, recent, Hkv, D, bs, dtype, values)
    ([40, 200, 48, 49, 0, 1], 48, 4, 16, 4, 64, 16, "f16", "ties"),
    ([1], 1, 0, 0, 1, 128, 16, "bf16", "ties"),
    ([2, 3], 1, 0, 1, 2, 128, 8, "bf16", "random"),            # the newest alone
    ([100, 7], 5, 5, 0, 1, 64, 16, "f16", "random"),           # the first ones alone: nothing is ranked
    ([100, 31], 30, 10, 20, 2, 128, 32, "bf16", "random"),     # sink + recent == keep
    ([300, 257, 17], 64, 0, 0, 3, 128, 64, "f16", "equal"),    # every total equal: the lowest indices
    ([500, 123], 100, 3, 17, 2, 64, 128, "bf16", "odd"),
    ([2500, 2048, 2049, 4100], 1024, 4, 256, 2, 128, 16, "bf16", "random"),
    ([2500, 4097], 2047, 0, 1, 1, 64, 16, "f16", "ties"),
    ([9000], 8999, 1, 1, 1, 64, 32, "f16", "ties"),            # one token goes
    ([9000, 20000], 70, 4, 32, 1, 64, 8, "bf16", "odd"),
    ([20000], 20001, 0, 0, 1, 64, 16, "bf16", "random"),       # nothing goes: moved as it is
    ([33000, 5], 15000, 7, 900, 1, 64, 64, "f16", "ties"),     # rows spread over eight CTAs, one of them all but empty
    ([65537], 30000, 7, 900, 1, 64, 128, "bf16", "equal"),     # one token more than eight CTAs hold at once
    ([150001], 70001, 0, 33, 1, 64, 128, "f16", "odd"),
]


@pytest.mark.parametrize("lens,keep,sink,recent,Hkv,D,bs,dtype,values", CASES)
def test_selection_and_move(lens, keep, sink, recent, Hkv, D, bs, dtype, values):
    c = setup(lens, keep, sink, recent, Hkv, D, bs, dtype, seed=len(lens) + keep, values=values)
    assert check(c) == 0


def test_totals_that_differ_in_their_last_bit():
    c = setup([3000], 1000, 2, 10, 2, 64, 16, "f16", seed=3)
    base = np.float32(0.3).view(np.uint32)
    rng = np.random.default_rng(0)
    c["w"] = (base + rng.integers(0, 300, size=c["w"].shape).astype(np.uint32)).view(np.float32)
    assert check(c) == 0


def test_rows_wider_than_the_contexts_and_special_values_in_the_cache():
    c = setup([90, 130], 64, 4, 8, 2, 64, 16, "f16", seed=4, width=333)
    c["kc"][:, :, ::3] = float("nan")
    c["vc"][:, :, ::5] = float("-inf")
    assert check(c) == 0


def test_old_blocks_may_be_shared_between_sequences():
    c = setup([100, 100, 64], 48, 4, 8, 2, 64, 16, "bf16", seed=5)
    c["old"][1] = c["old"][0]
    assert check(c) == 0


def test_a_new_block_named_twice_is_written_by_nobody():
    c = setup([100, 120, 90], 64, 4, 8, 1, 64, 16, "bf16", seed=6)
    # the third sequence's blocks are the first's, all four of them
    c["new"][2] = c["new"][0]
    assert check(c, skip=(0, 2)) == pa.capi.DEVERR["copy_pair"]


def test_conflicts_among_many_sequences():
    # more than one CTA marks and checks: a block named twice, one still read, one of its own
    c = setup([100 + i for i in range(9)], 64, 4, 8, 2, 64, 16, "bf16", seed=16)
    c["new"][7] = c["new"][3]
    c["new"][5] = c["old"][8, :4]
    c["new"][0] = c["old"][0, 2:6]
    assert check(c, skip=(0, 3, 5, 7)) == pa.capi.DEVERR["copy_pair"]


def test_a_new_block_that_is_still_read_is_not_written():
    c = setup([100, 120], 64, 4, 8, 1, 64, 16, "bf16", seed=7)
    before = c["kc"].clone()
    c["new"][0] = c["old"][1, :4]      # another sequence's blocks
    assert check(c, skip=(0,)) == pa.capi.DEVERR["copy_pair"]
    c["new"][0] = c["old"][0, :4]      # its own
    c["kc"].copy_(before)
    assert check(c, skip=(0,)) == pa.capi.DEVERR["copy_pair"]


def test_what_a_stale_workspace_says_is_ignored():
    c = setup([100, 120, 30], 64, 4, 8, 1, 64, 16, "bf16", seed=8)
    ws = pa.evict_workspace(c["kc"])
    nb = c["kc"].shape[0]
    for fill in (0, -1, 5, 2 ** 30):
        ws[:4 * nb].view(torch.int32).fill_(fill)
        assert call(c, workspace=ws)[3] == 0
    # left from a call whose new blocks are this call's old ones
    a = dict(c)
    call(a, workspace=ws)
    b = dict(c, old=c["new"].clone(), new=c["old"][:, :4].contiguous(), lens=[64, 64, 30])
    assert call(b, workspace=ws)[3] == 0


def test_entries_out_of_the_pool_are_flagged_and_the_rest_moves():
    c = setup([96, 100], 64, 4, 8, 1, 64, 16, "f16", seed=9, values="random")
    k0 = c["kc"].clone()
    good_old, good_new = c["old"].clone(), c["new"].clone()
    c["old"][0, 2] = 10 ** 6
    c["new"][1, 1] = -4
    kept, nl, nw, err = call(c)
    assert err == pa.capi.DEVERR["block_range"]
    for s in range(2):
        for i, j in enumerate(kept[s, 0, :64]):
            dst = k0[int(good_new[s, i // 16]), 0, i % 16]
            src = k0[int(good_old[s, j // 16]), 0, j % 16]
            lost = (s == 0 and j // 16 == 2) or (s == 1 and i // 16 == 1)
            got = c["kc"][int(good_new[s, i // 16]), 0, i % 16]
            assert torch.equal(got, dst if lost else src), (s, i)


def test_lengths_out_of_range_are_clamped_and_flagged():
    c = setup([64, 30], 32, 4, 8, 1, 64, 16, "f16", seed=10)
    real = c["lens"]
    c["lens"] = [1000, -2]
    kept, nl, nw, err = call(c)
    assert err == pa.capi.DEVERR["context_range"]
    assert list(nl) == [32, 0] and (kept[1] == -1).all()
    assert list(kept[0, 0]) == evict_choice(c["w"][0, 0], 64, 32, 4, 8)
    c["lens"] = real


def test_capture_replay_and_another_stream():
    c = setup([500, 900], 256, 4, 32, 2, 128, 16, "bf16", seed=11, values="random")
    check(c)
    kc, vc = c["kc"].clone(), c["vc"].clone()
    B = 2
    w, lens = torch.as_tensor(c["w"], device=DEV), torch.as_tensor(c["lens"], dtype=torch.int32, device=DEV)
    kept = torch.zeros((B, 2, 256), dtype=torch.int32, device=DEV)
    nl, nw = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros_like(w)
    ws = pa.evict_workspace(c["kc"])
    args = (c["kc"], c["vc"], w, c["old"], lens, c["new"], nl, nw, kept, 256, 4, 32, c["W"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pa.pa_evict(*args, workspace=ws, stream=s)
    s.synchronize()
    first = kept.clone(), nw.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_evict(*args, workspace=ws)
    new = c["new"].long().flatten()
    for _ in range(2):
        c["kc"][new] = 0
        c["vc"][new] = 0
        kept.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept, first[0]) and torch.equal(nw, first[1])
    assert torch.equal(kc, c["kc"]) and torch.equal(vc, c["vc"])


def test_wrong_tensors_are_refused():
    c = setup([40, 60], 32, 4, 8, 2, 64, 16, "f16", seed=12)
    w = torch.as_tensor(c["w"], device=DEV)
    lens = torch.as_tensor(c["lens"], dtype=torch.int32, device=DEV)
    a = [c["kc"], c["vc"], w, c["old"], lens, c["new"], torch.empty_like(lens), torch.empty_like(w),
         torch.empty((2, 2, 32), dtype=torch.int32, device=DEV), 32, 4, 8, 60]
    for i, x, exc in ((2, w.double(), TypeError), (3, c["old"].long(), TypeError), (8, a[8][:, :, :31], ValueError),
                      (7, w[:, :, :5], ValueError), (5, c["new"][:1], ValueError), (1, c["vc"].cpu(), ValueError),
                      (1, c["vc"].bfloat16(), TypeError)):
        b = list(a)
        b[i] = x
        with pytest.raises(exc):
            pa.pa_evict(*b)
    for i, x, status in ((10, 30, -3), (12, 61, -3), (7, w, -1), (6, lens, -1)):
        b = list(a)
        b[i] = x
        with pytest.raises(pa.PAError) as e:
            pa.pa_evict(*b)
        assert e.value.status == status
