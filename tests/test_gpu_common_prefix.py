"""pa_decode_common_prefix against attention in 64 bits over every sequence's
whole context, which knows nothing of sharing, within the attention bounds."""
import numpy as np
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.helpers import check_attention, scale_for, to_f64
from tests.ref64 import DTYPES, attend, gather, make_pool

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def setup(groups, size, pre, tails, Hq, Hkv, bs, dtype, seed, nan=False):
    """``tails``: own tokens of every sequence."""
    B, D = groups * size, 128
    kc, vc, own, shared = make_pool(tails, Hkv, D, bs, dtype, DEV, seed, extra=[pre * bs] * groups)
    bt = torch.full((B, pre + own.shape[1]), -1, dtype=torch.int32, device=DEV)
    bt[:, :pre] = shared.repeat_interleave(size, 0)
    bt[:, pre:] = own
    lens = [pre * bs + int(t) for t in tails]
    if nan:   # whatever no sequence holds
        used = torch.zeros(kc.shape[:1] + (bs,), dtype=torch.bool)
        for s, n in enumerate(lens):
            j = torch.arange(n)
            used[bt[s].cpu().long()[j // bs], j % bs] = True
        gap = (~used).to(DEV)[:, None, :, None]
        kc = torch.where(gap, torch.full_like(kc, float("nan")), kc)
        vc = torch.where(gap, torch.full_like(vc, float("inf")), vc)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn((B, Hq, D), generator=g).to(DTYPES[dtype]).to(DEV)
    return dict(kc=kc, vc=vc, bt=bt, lens=lens, q=q, size=size, pre=pre, ml=max(lens), scale=scale_for(D), dtype=dtype)


def call(c, lens=None, bt=None, **kw):
    out = torch.full(c["q"].shape, float("nan"), dtype=c["q"].dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_decode_common_prefix(out, c["q"], c["kc"], c["vc"], c["bt"] if bt is None else bt,
                               torch.as_tensor(lens or c["lens"], dtype=torch.int32, device=DEV), c["scale"], c["ml"],
                               c["size"], c["pre"], d_err=err, **kw)
    torch.cuda.synchronize()
    return out, int(err.item())


def check(c, seqs=None, **kw):
    out, err = call(c, **kw)
    assert err == 0, hex(err)
    seqs = range(len(c["lens"])) if seqs is None else seqs
    ref = [attend(c["q"][s].cpu().double(), gather(c["kc"], c["bt"][s], c["lens"][s]),
                  gather(c["vc"], c["bt"][s], c["lens"][s]), c["scale"])[0] for s in seqs]
    assert torch.isfinite(out.float()).all()
    check_attention(to_f64(out[list(seqs)]), torch.stack(ref).numpy(), c["dtype"], "common prefix")
    return out


CASES = [
    # (groups, size, prefix blocks, most own tokens, Hq, Hkv, bs, dtype)
    (1, 1, 1, 5, 1, 1, 16, "bf16"),
    (1, 2, 8, 20, 2, 2, 16, "f16"),        # one key tile exactly
    (1, 12, 62, 40, 4, 4, 16, "bf16"),     # more rows than the narrow form takes
    (2, 20, 9, 40, 8, 4, 16, "f16"),       # a ragged last key tile, two groups
    (3, 7, 5, 300, 8, 2, 32, "bf16"),
    (1, 33, 3, 10, 8, 1, 64, "f16"),       # 264 rows: a second row tile of 8
    (1, 70, 2, 3, 16, 2, 128, "bf16"),     # 560 rows
    (1, 300, 1, 1, 1, 1, 16, "bf16"),      # many rows, 16 keys
    (2, 3, 130, 600, 8, 8, 16, "bf16"),    # 17 key tiles, few rows: units cut in pieces
    (1, 5, 200, 0, 8, 1, 32, "f16"),       # no own tokens at all: 50 key tiles over as many CTAs
    (70, 2, 2, 9, 2, 1, 16, "bf16"),       # more groups than one launch takes
    (1, 9, 2, 700, 4, 4, 16, "f16"),       # own tokens in several partitions
]


@pytest.mark.parametrize("groups,size,pre,most,Hq,Hkv,bs,dtype", CASES)
def test_shapes(groups, size, pre, most, Hq, Hkv, bs, dtype):
    rng = np.random.default_rng(groups * 100 + size)
    tails = rng.integers(0, most + 1, size=groups * size)
    c = setup(groups, size, pre, tails, Hq, Hkv, bs, dtype, seed=size + pre)
    check(c, seqs=None if len(tails) <= 40 else sorted(set(rng.integers(0, len(tails), size=24)) | {0, len(tails) - 1}))


@pytest.mark.parametrize("pt", [16, 64, 4096])
def test_partitions_of_the_own_tokens(pt):
    c = setup(1, 10, 20, [0, 1, 15, 16, 17, 64, 65, 200, 333, 500], 8, 2, 16, "bf16", seed=pt)
    check(c, partition_tokens=pt)


def test_a_partition_longer_than_any_context():
    c = setup(1, 10, 20, [0, 1, 15, 16, 17, 64, 65, 200, 333, 500], 8, 2, 16, "bf16", seed=31)
    check(c, partition_tokens=2 ** 31 - 16)


def test_garbage_outside_the_contexts_stays_outside():
    check(setup(2, 10, 9, [3, 0, 17, 40, 5, 1, 2, 16, 31, 100] * 2, 8, 2, 16, "f16", seed=21, nan=True))


def test_agrees_with_the_narrow_form_and_with_plain_decode():
    c = setup(2, 4, 30, [10, 0, 55, 300, 7, 8, 9, 100], 4, 2, 16, "f16", seed=22)
    out = check(c)
    lens = torch.as_tensor(c["lens"], dtype=torch.int32, device=DEV)
    a, b = torch.empty_like(out), torch.empty_like(out)
    pa.pa_decode_shared_prefix(a, c["q"], c["kc"], c["vc"], c["bt"], lens, c["scale"], c["ml"], 4, 30)
    pa.pa_decode(b, c["q"], c["kc"], c["vc"], c["bt"], lens, c["scale"], c["ml"])
    torch.cuda.synchronize()
    assert (out.float() - a.float()).abs().max() <= 4e-3 and (out.float() - b.float()).abs().max() <= 4e-3


def test_scores_that_grow_along_the_prefix_and_lie_far_apart():
    # every later key tile raises the maxima past the rescale threshold, and the own tokens raise them once more
    c = setup(1, 40, 40, [30] * 40, 8, 2, 16, "bf16", seed=23)
    n = 40 * 16
    j = torch.arange(n)
    tb = c["bt"][0].cpu().long()
    ramp = (1 + (j // 64).float() * 0.8).to(DEV)
    blk, r = tb[j // 16].to(DEV), (j % 16).to(DEV)
    c["kc"][blk, :, r] = (c["kc"][blk, :, r].float() * ramp[:, None, None]).to(torch.bfloat16)
    check(c)


def test_one_long_prefix_behind_a_large_batch():
    rng = np.random.default_rng(5)
    c = setup(1, 150, 256, rng.integers(1, 40, size=150), 16, 2, 16, "bf16", seed=24)
    check(c, seqs=[0, 1, 31, 32, 63, 64, 100, 148, 149])


def test_broken_promises_are_flagged():
    c = setup(2, 10, 4, [20] * 20, 4, 2, 16, "bf16", seed=25)
    bad = c["bt"].clone()
    bad[13, 2] = c["bt"][0, 0]
    _, err = call(c, bt=bad)
    assert err == pa.capi.DEVERR["prefix"]
    lens = list(c["lens"])
    lens[7] = 63
    out, err = call(c, lens=lens)
    assert err & pa.capi.DEVERR["context_range"]
    lens[7] = c["ml"] + 1
    _, err = call(c, lens=lens)
    assert err & pa.capi.DEVERR["context_range"]
    bad = c["bt"].clone()
    bad[:10, 1] = 10 ** 6
    out, err = call(c, bt=bad)
    assert err == pa.capi.DEVERR["block_range"]
    # the other group's outputs are right all the same
    good, _ = call(c)
    assert torch.equal(out[10:], good[10:])


@pytest.mark.parametrize("length", [0, 63, 65, 200])
def test_wrong_lengths_are_flagged_where_the_prefix_is_the_whole_context(length):
    c = setup(2, 3, 4, [0] * 6, 4, 2, 16, "bf16", seed=32)
    good = check(c)
    lens = list(c["lens"])
    lens[4] = length
    out, err = call(c, lens=lens)
    assert err == pa.capi.DEVERR["context_range"]
    assert torch.equal(out[:4], good[:4]) and torch.equal(out[5:], good[5:])


def test_results_repeat_bit_for_bit_whatever_the_workspace_holds_captured_and_on_another_stream():
    c = setup(1, 24, 70, list(range(24)), 8, 2, 16, "bf16", seed=26)
    ref, _ = call(c)
    ws = pa.decode_common_prefix_workspace(c["q"], 2, 16, c["ml"], 24, 70)
    ws[256:].fill_(255)    # past the counter its content is ignored
    out = torch.zeros_like(ref)
    lens = torch.as_tensor(c["lens"], dtype=torch.int32, device=DEV)
    args = (out, c["q"], c["kc"], c["vc"], c["bt"], lens, c["scale"], c["ml"], 24, 70)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pa.pa_decode_common_prefix(*args, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_common_prefix(*args, workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


def test_one_workspace_serves_calls_of_other_sizes():
    big = setup(2, 40, 30, list(range(80)), 8, 2, 16, "f16", seed=28)
    small = setup(1, 3, 2, [5, 0, 40], 8, 2, 16, "f16", seed=29)
    none = setup(1, 4, 3, [0] * 4, 8, 2, 16, "f16", seed=30)
    ws = pa.decode_common_prefix_workspace(big["q"], 2, 16, big["ml"], 40, 30)
    want = [call(c)[0] for c in (big, small, none)]
    for _ in range(2):
        for c, w in zip((big, small, none), want):
            out, err = call(c, workspace=ws)
            assert err == 0 and torch.equal(out, w)


def test_wrong_tensors_are_refused():
    c = setup(1, 10, 2, [4] * 10, 4, 2, 16, "f16", seed=27)
    lens = torch.as_tensor(c["lens"], dtype=torch.int32, device=DEV)
    a = [torch.empty_like(c["q"]), c["q"], c["kc"], c["vc"], c["bt"], lens, c["scale"], c["ml"], 10, 2]
    for i, x, exc in ((4, c["bt"].long(), TypeError), (1, c["q"].bfloat16(), TypeError), (5, lens[:3], ValueError),
                      (3, c["vc"][:2], ValueError), (0, a[0].cpu(), ValueError)):
        b = list(a)
        b[i] = x
        with pytest.raises(exc):
            pa.pa_decode_common_prefix(*b)
    for i, x, status in ((8, 3, -1), (9, 0, -1), (9, 50, -3), (6, 0.0, -3)):
        b = list(a)
        b[i] = x
        with pytest.raises(pa.PAError) as e:
            pa.pa_decode_common_prefix(*b, workspace=torch.empty(1 << 22, dtype=torch.uint8, device=DEV))
        assert e.value.status == status
