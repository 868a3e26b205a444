"""pa_decode_weights against attention in 64 bits, token by token.

Tolerance of a weight, by arithmetic: a score is a sum of D products, each
exact in fp32, added up in fp32: off by at most D 2^-23 A, A = the largest sum
of |q_i k_i| times the scale (2^-23: the tensor cores may truncate).  A weight
exp(s - M) / l moves by that much relatively, twice (its own score, and the
sum's), plus 2^-19 for the scaling by log2 e, the exponentials, the sums and
the division.  A total adds its own roundings, 2^-23 of its size per query.
Outputs have the bounds of every attention here."""
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


def setup(rows, w, Hq, Hkv, D, bs, dtype, seed, width=None):
    """rows: cache lengths; w query positions observe each, the last ones of the sequence."""
    kc, vc, table, _ = make_pool(rows, Hkv, D, bs, dtype, DEV, seed)
    ctx = [max(0, n - (w - 1 - i)) for n in rows for i in range(w)]
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn((len(ctx), Hq, D), generator=g).to(DTYPES[dtype]).to(DEV)
    ml = max(max(rows), 1)
    tot = torch.rand((len(rows), Hkv, width or ml), generator=g).to(DEV)
    return dict(kc=kc, vc=vc, bt=table.repeat_interleave(w, 0).contiguous(), ctx=ctx, q=q, ml=ml, tot=tot, w=w,
                lens=torch.as_tensor(ctx, dtype=torch.int32, device=DEV), scale=scale_for(D), dtype=dtype)


def reference(c):
    outs, tot = [], c["tot"].cpu().double().clone()
    tol = torch.zeros_like(tot)
    for i, n in enumerate(c["ctx"]):
        K, V = gather(c["kc"], c["bt"][i], n), gather(c["vc"], c["bt"][i], n)
        o, p, size = attend(c["q"][i].cpu().double(), K, V, c["scale"])
        outs.append(o)
        r = i // c["w"]
        tot[r, :, :n] += p
        D = c["q"].shape[2]
        tol[r, :, :n] += p * (2 * D * 2.0 ** -23 * size + 2.0 ** -19)
        tol[r, :, :n] += tot[r, :, :n] * 2.0 ** -23
    return torch.stack(outs), tot, tol


def call(c, in_place=False, **kw):
    out = torch.full(c["q"].shape, float("nan"), dtype=c["q"].dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tot = c["tot"].clone()
    new = tot if in_place else torch.full_like(tot, -7.0)
    pa.pa_decode_weights(out, c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["scale"], c["ml"], tot,
                         None if in_place else new, queries_per_row=c["w"], d_err=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0, hex(int(err.item()))
    if not in_place:
        assert torch.equal(tot, c["tot"])
    return out, new


def check(c, in_place=False, **kw):
    ref, tot, tol = reference(c)
    out, new = call(c, in_place, **kw)
    check_attention(to_f64(out), ref.numpy(), c["dtype"], "outputs")
    new = new.cpu().double()
    rows = [max(c["ctx"][r * c["w"]:(r + 1) * c["w"]]) for r in range(len(c["ctx"]) // c["w"])]
    for r, n in enumerate(rows):
        err = (new[r, :, :n] - tot[r, :, :n]).abs()
        assert bool((err <= tol[r, :, :n]).all()), (r, float((err - tol[r, :, :n]).max()))
        # entries past the contexts are left as they were
        left = c["tot"].cpu().double()[r, :, n:] if in_place else torch.full_like(new[r, :, n:], -7.0)
        assert torch.equal(new[r, :, n:], left)


SHAPES = [
    # (D, bs, G, Hkv, dtype)
    (128, 16, 4, 2, "bf16"), (128, 16, 1, 3, "f16"), (128, 16, 8, 1, "bf16"), (128, 16, 2, 2, "f16"),
    (128, 8, 4, 1, "bf16"), (128, 8, 8, 1, "f16"), (128, 32, 8, 2, "f16"), (128, 64, 1, 2, "bf16"),
    (128, 128, 8, 1, "bf16"), (128, 128, 2, 1, "f16"), (64, 16, 1, 4, "f16"), (64, 8, 8, 1, "bf16"),
    (64, 16, 4, 2, "bf16"), (64, 32, 2, 2, "f16"), (64, 64, 8, 1, "f16"), (64, 128, 1, 1, "bf16"),
]


@pytest.mark.parametrize("D,bs,G,Hkv,dtype", SHAPES)
def test_shapes_and_ragged_lengths(D, bs, G, Hkv, dtype):
    check(setup([1, bs - 1, bs, bs + 1, 0, 3 * bs + 5, 255, 257, 530], 1, G * Hkv, Hkv, D, bs, dtype, seed=D + bs + G))


@pytest.mark.parametrize("G,D", [(1, 128), (4, 128), (8, 128), (8, 64)])
@pytest.mark.parametrize("pt", [16, 64, 256, 4096])
def test_partitions(G, D, pt):
    check(setup([1, 16, 17, 300, 1025], 1, G, 1, D, 16, "bf16", seed=pt + G), partition_tokens=pt)


@pytest.mark.parametrize("G,D,w", [(4, 128, 1), (1, 64, 1), (2, 128, 3)])
def test_a_partition_longer_than_any_context(G, D, w):
    check(setup([1, 16, 17, 300, 1025], w, G, 1, D, 16, "bf16", seed=D + G), partition_tokens=2 ** 31 - 16)


@pytest.mark.parametrize("w", [2, 5, 16])
@pytest.mark.parametrize("G", [4, 8])
def test_several_queries_add_to_one_row_in_place(w, G):
    # contexts shorter than the window among them: their first queries see nothing
    check(setup([3, 700, 0, 64], w, 2 * G, 2, 128, 16, "f16", seed=w), in_place=True)


@pytest.mark.parametrize("D,bs,G,dtype", [(64, 16, 4, "bf16"), (64, 128, 8, "f16"), (128, 8, 8, "bf16"), (128, 16, 1, "f16")])
def test_several_queries_one_after_the_other(D, bs, G, dtype):
    # shapes that are not attended together; more positions than are summed at once
    check(setup([600, 37], 20 if G * 20 < 16 or D == 64 or bs == 8 else 3, G, 1, D, bs, dtype, seed=D + G))


WINDOWS = [
    # (cache lengths, positions, G, Hkv, bs, dtype): attended together on the tensor cores
    ([300], 16, 1, 1, 16, "bf16"),
    ([2000, 3, 640], 8, 4, 2, 16, "f16"),          # lengths far apart: CTAs with nothing to do
    ([129, 128, 127], 4, 8, 1, 64, "bf16"),
    ([900], 70, 4, 1, 32, "f16"),                  # 280 query rows: a second row tile of 24
    ([40, 0, 1], 33, 8, 1, 128, "bf16"),           # more positions than tokens, no tokens, one token
    ([700, 1500], 20, 2, 3, 16, "bf16"),
    ([33] * 70, 16, 1, 1, 16, "f16"),              # more rows than one launch takes
    ([1, 400], 9, 8, 2, 16, "f16"),
]


@pytest.mark.parametrize("rows,w,G,Hkv,bs,dtype", WINDOWS)
@pytest.mark.parametrize("in_place", [False, True])
def test_windows(rows, w, G, Hkv, bs, dtype, in_place):
    check(setup(rows, w, G * Hkv, Hkv, 128, bs, dtype, seed=w + G), in_place=in_place)


def test_window_positions_in_any_order_and_apart():
    c = setup([700, 500], 6, 8, 2, 128, 16, "bf16", seed=31)
    c["ctx"] = [700, 1, 350, 0, 129, 128, 20, 500, 499, 17, 16, 256]
    c["lens"] = torch.as_tensor(c["ctx"], dtype=torch.int32, device=DEV)
    check(c)


def test_window_garbage_past_the_contexts_does_not_reach_anything():
    c = setup([300, 45], 8, 4, 1, 128, 16, "f16", seed=32)
    a, wa = call(c)
    for r, n in enumerate((300, 45)):
        b = int(c["bt"][r * 8, (n - 1) // 16])
        c["kc"][b, :, n % 16:] = float("nan")
        c["vc"][b, :, n % 16:] = float("inf")
    b, wb = call(c)
    assert torch.equal(a, b) and torch.equal(wa, wb)


def test_window_bad_entries_weigh_nothing_and_broken_promises_are_flagged():
    c = setup([300], 5, 8, 2, 128, 32, "bf16", seed=33)
    bad = c["bt"].clone()
    bad[:, 3] = 10 ** 6
    bad[:, 5] = -9

    def run(bt, lens):
        out, new = torch.empty_like(c["q"]), torch.full_like(c["tot"], -7.0)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        pa.pa_decode_weights(out, c["q"], c["kc"], c["vc"], bt, lens, c["scale"], c["ml"], c["tot"], new,
                             queries_per_row=5, d_err=err)
        torch.cuda.synchronize()
        return out, new, int(err.item())
    out, new, err = run(bad, c["lens"])
    assert err == pa.capi.DEVERR["block_range"]
    tot, tol, ref = c["tot"][0].cpu().double().clone(), torch.zeros_like(c["tot"][0].cpu().double()), []
    for i, n in enumerate(c["ctx"]):
        keep = [j for j in range(n) if j // 32 not in (3, 5)]
        K, V = gather(c["kc"], c["bt"][i], n)[keep], gather(c["vc"], c["bt"][i], n)[keep]
        o, p, size = attend(c["q"][i].cpu().double(), K, V, c["scale"])
        ref.append(o)
        tot[:, keep] += p
        tol[:, keep] += p * (2 * 128 * 2.0 ** -23 * size + 2.0 ** -19) + tot[:, keep] * 2.0 ** -23
    check_attention(to_f64(out), torch.stack(ref).numpy(), "bf16", "kept keys")
    assert bool(((new[0].cpu().double() - tot).abs() <= tol).all())
    # a position whose table row is another's
    odd = c["bt"].clone()
    odd[2, 1] = c["bt"][0, 0]
    assert run(odd, c["lens"])[2] == pa.capi.DEVERR["prefix"]
    # lengths out of range are clamped
    lens = c["lens"].clone()
    lens[4], lens[1] = 10000, -1
    out2, _, err = run(c["bt"], lens)
    assert err == pa.capi.DEVERR["context_range"]
    good, _, _ = run(c["bt"], c["lens"])
    assert torch.equal(out2[4], good[4]) and not bool(out2[1].any())


def test_window_workspace_content_capture_and_another_stream():
    c = setup([900, 77], 16, 4, 1, 128, 16, "bf16", seed=34)
    ref, wref = call(c)
    ws = pa.decode_weights_workspace(c["q"], 1, 16, c["ml"], queries_per_row=16)
    ws.fill_(255)
    out, new = torch.zeros_like(ref), torch.full_like(wref, -7.0)
    args = (out, c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["scale"], c["ml"], c["tot"], new)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pa.pa_decode_weights(*args, queries_per_row=16, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(new, wref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_weights(*args, queries_per_row=16, workspace=ws)
    for _ in range(2):
        out.zero_()
        new.fill_(-7.0)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(new, wref)


def test_a_row_of_totals_wider_than_the_contexts():
    check(setup([40, 5], 1, 4, 2, 64, 16, "bf16", seed=3, width=77))


def test_no_tokens_at_all():
    c = setup([0, 0], 1, 4, 2, 128, 16, "bf16", seed=4)
    out, new = call(c)
    assert not bool(out.any()) and bool((new == -7.0).all())


def test_agrees_with_plain_decode_to_the_bit_in_one_partition_and_across():
    for lens in ([30, 200, 250], [30, 900, 2000]):
        c = setup(lens, 1, 8, 2, 128, 16, "bf16", seed=12)
        out, _ = call(c)
        plain = torch.empty_like(out)
        pa.pa_decode(plain, c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["scale"], c["ml"])
        torch.cuda.synchronize()
        assert torch.equal(out, plain)


def test_repeated_calls_are_bit_identical_and_totals_accumulate():
    c = setup([513, 1300, 64], 2, 16, 2, 128, 16, "bf16", seed=13)
    a, wa = call(c)
    b, wb = call(c)
    assert torch.equal(a, b) and torch.equal(wa, wb)
    # twice in place: two steps' weights (a query's weights of a kv head sum to its G heads)
    t = torch.zeros_like(c["tot"])
    for _ in range(2):
        pa.pa_decode_weights(torch.empty_like(a), c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["scale"], c["ml"], t,
                             queries_per_row=2)
    torch.cuda.synchronize()
    assert torch.allclose(t.sum(-1), torch.full_like(t.sum(-1), 2 * 2 * 8.0), rtol=1e-4)


@pytest.mark.parametrize("G,D,bs", [(4, 128, 16), (8, 128, 16), (2, 64, 32), (4, 128, 8)])
def test_bad_table_entries_weigh_nothing_and_are_flagged(G, D, bs):
    # 16-key groups, so that at block size 8 the tile that is left out is the two bad blocks
    c = setup([160, 48], 1, G, 1, D, bs, "bf16", seed=14)
    bad = c["bt"].clone()
    per = max(1, 16 // bs)
    bad[0, 2 * per:3 * per] = 10 ** 6
    bad[1] = torch.where(bad[1] >= 0, torch.full_like(bad[1], -5), bad[1])   # every key left out
    out, new = torch.empty_like(c["q"]), torch.full_like(c["tot"], -7.0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_decode_weights(out, c["q"], c["kc"], c["vc"], bad, c["lens"], c["scale"], c["ml"], c["tot"], new, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.capi.DEVERR["block_range"]
    gone = list(range(2 * per * bs, 3 * per * bs))
    keep = [j for j in range(160) if j not in gone]
    good = c["bt"][0]
    K, V = gather(c["kc"], good, 160)[keep], gather(c["vc"], good, 160)[keep]
    o, p, size = attend(c["q"][0].cpu().double(), K, V, c["scale"])
    check_attention(to_f64(out[:1]), o[None].numpy(), "bf16", "kept keys")
    got, base = new[0].cpu().double(), c["tot"][0].cpu().double()
    assert torch.equal(got[:, gone], base[:, gone])
    tol = p * (2 * D * 2.0 ** -23 * size + 2.0 ** -19) + (base[:, keep] + p) * 2.0 ** -23
    assert bool(((got[:, keep] - base[:, keep] - p).abs() <= tol).all())
    # nothing to attend: zeros, and the totals as they were
    assert not bool(out[1].any()) and torch.equal(new[1, :, :48], c["tot"][1, :, :48])


def test_lengths_out_of_range_are_clamped_and_flagged():
    c = setup([64, 30], 1, 4, 1, 128, 16, "f16", seed=15)
    lens = c["lens"].clone()
    lens[0], lens[1] = 1000, -3
    out, new = torch.empty_like(c["q"]), torch.full_like(c["tot"], -7.0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_decode_weights(out, c["q"], c["kc"], c["vc"], c["bt"], lens, c["scale"], c["ml"], c["tot"], new, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.capi.DEVERR["context_range"]
    full, tot = call(c)
    assert torch.equal(out[0], full[0]) and torch.equal(new[0], tot[0])
    assert not bool(out[1].any()) and bool((new[1] == -7.0).all())


def test_garbage_past_the_contexts_does_not_reach_anything():
    c = setup([5, 33, 300], 1, 8, 1, 128, 16, "f16", seed=16)
    a, wa = call(c)
    for i, n in enumerate(c["ctx"]):
        b = int(c["bt"][i, (n - 1) // 16])
        if n % 16:
            c["kc"][b, :, n % 16:] = float("nan")
            c["vc"][b, :, n % 16:] = float("inf")
    b, wb = call(c)
    assert torch.equal(a, b) and torch.equal(wa, wb)


def test_workspace_reuse_capture_and_another_stream():
    c = setup([900, 40, 1500], 1, 8, 2, 128, 16, "bf16", seed=17)
    ref, wref = call(c)
    ws = pa.decode_weights_workspace(c["q"], 2, 16, c["ml"])
    ws.fill_(255)          # its content on entry is ignored
    out, new = torch.zeros_like(ref), torch.full_like(wref, -7.0)
    args = (out, c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["scale"], c["ml"], c["tot"], new)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pa.pa_decode_weights(*args, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(new, wref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_weights(*args, workspace=ws)
    for _ in range(2):
        out.zero_()
        new.fill_(-7.0)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(new, wref)


def test_wrong_tensors_are_refused():
    c = setup([20, 40], 1, 4, 2, 64, 16, "f16", seed=18)
    a = [torch.empty_like(c["q"]), c["q"], c["kc"], c["vc"], c["bt"], c["lens"], c["scale"], c["ml"], c["tot"]]
    for i, x, exc in ((4, c["bt"].long(), TypeError), (5, c["lens"].long(), TypeError), (8, c["tot"].half(), TypeError),
                      (8, c["tot"][:1], ValueError), (8, c["tot"].cpu(), ValueError), (1, c["q"].bfloat16(), TypeError),
                      (1, c["q"][:, :, :32], ValueError), (3, c["vc"][:1], ValueError)):
        b = list(a)
        b[i] = x
        with pytest.raises(exc):
            pa.pa_decode_weights(*b)
    with pytest.raises(ValueError):
        pa.pa_decode_weights(*a, queries_per_row=3)
    with pytest.raises(pa.PAError) as e:
        b = list(a)
        b[7] = 41     # contexts longer than a row of totals
        pa.pa_decode_weights(*b)
    assert e.value.status == -3
    with pytest.raises(pa.PAError) as e:
        pa.pa_decode_weights(*a, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == -5
    pa.pa_decode_weights(a[0][:0], c["q"][:0], c["kc"], c["vc"], c["bt"][:0], c["lens"][:0], c["scale"], c["ml"], c["tot"][:0])
