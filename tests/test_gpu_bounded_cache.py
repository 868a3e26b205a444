"""The bounded-cache calls together, as an engine makes them, against a 64-bit
replay on the host: a prompt enters through pa_rotary_and_cache, its last
positions observe it through pa_decode_weights, pa_evict cuts it down, and
decode steps go on at the true positions with further evictions, while a fork
taken before the first eviction keeps decoding over the whole prompt.  The
block manager supplies every table, slot and copy pair.

What is computed is held to the operators' bounds; which tokens are kept is
checked exactly, as the plain choice on the totals the GPU holds at that
moment, and the replay then drops the same tokens."""
import numpy as np
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests.helpers import check_attention, to_f64
from tests.ref64 import DTYPES, attend, evict_choice, gather, half_step, make_pool, rotate

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
AXES, W = 3, 300     # position axes, width of a row of totals


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


class Engine:
    def __init__(self, Hq, Hkv, D, bs, dtype, seed):
        self.Hq, self.Hkv, self.D, self.bs, self.dtype = Hq, Hkv, D, bs, dtype
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator().manual_seed(seed)
        self.bm = pa.BlockManager(96, bs)
        dt = DTYPES[dtype]
        self.kc = torch.randn((96, Hkv, bs, D), generator=self.gen).to(dt).to(DEV)
        self.vc = torch.randn((96, Hkv, bs, D), generator=self.gen).to(dt).to(DEV)
        self.inv = (1e4 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
        self.axis = (np.arange(D // 2) % AXES).astype(np.int32)
        self.inv_d = torch.as_tensor(self.inv, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.scale = D ** -0.5
        self.pairs = None

    def enter(self, pos, slots):
        """Tokens at ``pos`` [axes][T] into ``slots``; their rotated queries."""
        T = pos.shape[1]
        qkv = torch.randn((T, self.Hq + 2 * self.Hkv, self.D), generator=self.gen).to(DTYPES[self.dtype]).to(DEV)
        q, k, v = qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hkv], qkv[:, self.Hq + self.Hkv:]
        out = torch.empty((T, self.Hq, self.D), dtype=qkv.dtype, device=DEV)
        pa.pa_rotary_and_cache(out, q, k, v, self.kc, self.vc, torch.as_tensor(pos, device=DEV),
                               torch.as_tensor(slots, device=DEV), self.inv_d, self.axis, d_err=self.err)
        angle = torch.as_tensor(pos[self.axis].T.astype(np.float64) * self.inv.astype(np.float64))
        rk = rotate(k.cpu().double(), angle, False)
        return out, rk, v.cpu().double()

    def table(self, seq):
        return torch.as_tensor(self.bm.tables([seq]), device=DEV)

    def check_cache(self, seq, K, V):
        """The cached rows are the replay's, K within one rounding of it, V to the bit."""
        n = self.bm.seq_len(seq)
        t = self.table(seq)[0]
        gk, gv = gather(self.kc, t, n), gather(self.vc, t, n)
        for h in range(self.Hkv):
            assert torch.equal(gv[:, h], torch.stack(V[h])), h
            # (the rotation in fp32: 2^-21 of |a| + |b|, which is below 8 here)
            assert bool(((gk[:, h] - torch.stack(K[h])).abs() <=
                         torch.stack(K[h]).abs() * half_step(self.dtype) * 1.01 + 2.0 ** -18).all())
        return gk, gv


@pytest.mark.parametrize("Hq,Hkv,D,bs,dtype", [(8, 2, 128, 16, "bf16"), (8, 1, 128, 32, "f16"), (4, 2, 64, 8, "f16")])
def test_prompt_observation_eviction_and_decode(Hq, Hkv, D, bs, dtype):
    e = Engine(Hq, Hkv, D, bs, dtype, seed=D + bs)
    N, keep, sink, recent, w = 150, 64, 4, 16, 8
    tokens = e.rng.integers(0, 1000, size=N)
    slots, cached = e.bm.add_sequence(1, tokens)
    assert cached == 0
    pos = np.stack([np.arange(N), np.arange(N) // 7, np.arange(N) % 7]).astype(np.int32) + 40000
    q, rk, v = e.enter(pos, slots)
    K = [[rk[t, h] for t in range(N)] for h in range(Hkv)]
    V = [[v[t, h] for t in range(N)] for h in range(Hkv)]
    gk, gv = e.check_cache(1, K, V)
    e.bm.fork(1, 2)
    full = gk.clone(), gv.clone()

    # the last w positions observe the prompt
    tot = torch.zeros((1, Hkv, W), dtype=torch.float32, device=DEV)
    ctx = np.arange(N - w + 1, N + 1)
    out = torch.empty((w, Hq, D), dtype=q.dtype, device=DEV)
    pa.pa_decode_weights(out, q[N - w:].contiguous(), e.kc, e.vc, e.table(1).repeat(w, 1).contiguous(),
                         torch.as_tensor(ctx.astype(np.int32), device=DEV), e.scale, N, tot, queries_per_row=w, d_err=e.err)
    ref_tot = torch.zeros((Hkv, W), dtype=torch.float64)
    ref = []
    for i, n in enumerate(ctx):
        o, p, size = attend(q[N - w + i].cpu().double(), gk[:n], gv[:n], e.scale)
        ref.append(o)
        ref_tot[:, :n] += p
    check_attention(to_f64(out), torch.stack(ref).numpy(), dtype, "observation")
    # 2 D 2^-23 A + 2^-19 < 2^-11 for A < 12 and D <= 128 (A: the largest scaled sum of |q_i k_i|)
    near = lambda a, b: bool(((a - b).abs() <= b * 2.0 ** -11).all())
    assert size < 12 and near(tot[0].cpu().double(), ref_tot)

    def cut(seq, tot):
        n = e.bm.seq_len(seq)
        old = e.table(seq)
        e.bm.evict_sequence(seq, min(n, keep))
        new = e.table(seq)
        kept = torch.empty((1, Hkv, keep), dtype=torch.int32, device=DEV)
        nl, nt = torch.zeros(1, dtype=torch.int32, device=DEV), torch.empty_like(tot)
        pa.pa_evict(e.kc, e.vc, tot, old, torch.tensor([n], dtype=torch.int32, device=DEV), new, nl, nt, kept, keep, sink,
                    recent, n, d_err=e.err)
        host = tot[0].cpu().numpy()
        for h in range(Hkv):
            idx = evict_choice(host[h], n, keep, sink, recent)
            assert list(kept[0, h].cpu().numpy()) == idx
            K[h][:], V[h][:] = [K[h][j] for j in idx], [V[h][j] for j in idx]
            ref_tot[h, :keep] = ref_tot[h, idx].clone()
            ref_tot[h, keep:] = 0
        assert int(nl.item()) == keep == e.bm.seq_len(seq)
        return nt

    tot = cut(1, tot)
    evictions = 1
    for step in range(60):
        # one token for the bounded sequence and one for its fork, whose cache is whole
        new_slots, pairs = [], []
        for s in (1, 2):
            slot, pair = e.bm.append_token(s, 2000 + step)
            new_slots.append(slot)
            if pair:
                pairs.append(pair)
        if pairs:
            pa.pa_copy_blocks(e.kc, e.vc, torch.tensor(pairs, dtype=torch.int64, device=DEV), d_err=e.err)
        p = np.full((AXES, 2), 40000 + N + step, np.int32)
        q, rk, v = e.enter(p, np.array(new_slots, np.int64))
        for h in range(Hkv):
            K[h].append(rk[0, h])
            V[h].append(v[0, h])
        n = e.bm.seq_len(1)
        gk, gv = e.check_cache(1, K, V)
        out = torch.empty((1, Hq, D), dtype=q.dtype, device=DEV)
        pa.pa_decode_weights(out, q[:1].contiguous(), e.kc, e.vc, e.table(1),
                             torch.tensor([n], dtype=torch.int32, device=DEV), e.scale, n, tot, d_err=e.err)
        o, pr, size = attend(q[0].cpu().double(), gk, gv, e.scale)
        assert size < 12
        ref_tot[:, :n] += pr
        check_attention(to_f64(out), o[None].numpy(), dtype, f"step {step}")
        assert near(tot[0].cpu().double(), ref_tot), step
        if step in (0, 31, 59):   # the fork: the whole prompt, and what followed it
            n2 = e.bm.seq_len(2)
            assert n2 == N + step + 1
            t2 = e.table(2)[0]
            fk, fv = gather(e.kc, t2, n2), gather(e.vc, t2, n2)
            assert torch.equal(fk[:N], full[0]) and torch.equal(fv[:N], full[1])
            out2 = torch.empty_like(out)
            pa.pa_decode(out2, q[1:].contiguous(), e.kc, e.vc, e.table(2), torch.tensor([n2], dtype=torch.int32, device=DEV),
                         e.scale, n2, d_err=e.err)
            check_attention(to_f64(out2), attend(q[1].cpu().double(), fk, fv, e.scale)[0][None].numpy(), dtype, "fork")
        if n >= keep + 24:
            tot = cut(1, tot)
            evictions += 1
    torch.cuda.synchronize()
    assert int(e.err.item()) == 0 and evictions == 3
    e.bm.free_sequence(1)
    e.bm.free_sequence(2)
    assert e.bm.stats()["used_blocks"] == 0


def test_a_batch_behind_a_system_prompt_step_by_step():
    """Rotary write, then the shared-prefix decode, for a few steps of a batch whose
    sequences were forked from one prompt."""
    e = Engine(8, 2, 128, 16, "bf16", seed=9)
    N, B = 64, 11
    slots, _ = e.bm.add_sequence(0, np.arange(N))
    pos = np.tile(np.arange(N, dtype=np.int32), (AXES, 1))
    e.enter(pos, slots)
    for s in range(1, B):
        e.bm.fork(0, s)
    # (N is whole blocks: every sequence goes on in blocks of its own)
    ws = pa.decode_common_prefix_workspace(torch.empty((B, 8, 128), dtype=torch.bfloat16, device=DEV), 2, 16, N + 20, B, N // 16)
    for step in range(20):
        new = [e.bm.append_token(s, step) for s in range(B)]
        assert all(p is None for _, p in new)
        q, _, _ = e.enter(np.full((AXES, B), N + step, np.int32), np.array([s for s, _ in new], np.int64))
        bt = torch.as_tensor(e.bm.tables(range(B)), device=DEV)
        lens = torch.full((B,), N + step + 1, dtype=torch.int32, device=DEV)
        out = torch.empty_like(q)
        pa.pa_decode_common_prefix(out, q, e.kc, e.vc, bt, lens, e.scale, N + 20 if bt.shape[1] * 16 >= N + 20 else N + step + 1,
                                   B, N // 16, workspace=ws, d_err=e.err)
        if step % 6 == 0 or step == 19:
            ref = [attend(q[s].cpu().double(), gather(e.kc, bt[s], N + step + 1), gather(e.vc, bt[s], N + step + 1), e.scale)[0]
                   for s in range(B)]
            check_attention(to_f64(out), torch.stack(ref).numpy(), "bf16", f"step {step}")
    torch.cuda.synchronize()
    assert int(e.err.item()) == 0


def test_pools_of_more_than_two_to_the_32_elements():
    """Blocks past element 2^32 of a pool (8.6 GB a cache) against the same blocks
    in a small one: every call gives the same bits."""
    Hkv, Hq, bs, D, n = 8, 32, 16, 128, 40
    far = (1 << 32) // (Hkv * bs * D)
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    g = torch.Generator(device=DEV).manual_seed(1)
    small = [torch.randn((n, Hkv, bs, D), device=DEV, generator=g).half() for _ in range(2)]
    big = [torch.empty((far + n, Hkv, bs, D), dtype=torch.float16, device=DEV) for _ in range(2)]
    for b, c in zip(big, small):
        b[far:] = c
    q = torch.randn((2, Hq, D), device=DEV, generator=g).half()
    k, v = (torch.randn((2, Hkv, D), device=DEV, generator=g).half() for _ in range(2))
    tot = torch.rand((2, Hkv, 200), device=DEV, generator=g)
    lens = torch.tensor([160, 131], dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(kc, vc, off):
        old = torch.arange(20, dtype=torch.int32, device=DEV).view(2, 10) + off
        new = torch.arange(20, 28, dtype=torch.int32, device=DEV).view(2, 4) + off
        slots = torch.tensor([9 * bs + 15, 18 * bs + 2], device=DEV) + off * bs
        qr = torch.empty_like(q)
        pa.pa_rotary_and_cache(qr, q, k, v, kc, vc, torch.tensor([7, 99], dtype=torch.int32, device=DEV), slots,
                               torch.ones(64, device=DEV), d_err=err)
        out, t = torch.empty_like(q), tot.clone()
        pa.pa_decode_weights(out, qr, kc, vc, old, lens, 0.09, 160, t, d_err=err)
        four = [x.repeat_interleave(4, 0).contiguous() for x in (qr, old, lens)]   # attended together
        wout, wt = torch.empty_like(four[0]), tot.clone()
        pa.pa_decode_weights(wout, four[0], kc, vc, four[1], four[2], 0.09, 160, wt, queries_per_row=4, d_err=err)
        kept = torch.empty((2, Hkv, 64), dtype=torch.int32, device=DEV)
        nl, nt = torch.empty_like(lens), torch.empty_like(tot)
        pa.pa_evict(kc, vc, t, old, lens, new, nl, nt, kept, 64, 4, 8, 160, d_err=err)
        shared = torch.cat((old[:1, :4].repeat(2, 1), old[:, 4:]), 1).contiguous()
        pout = torch.empty_like(q)
        pa.pa_decode_common_prefix(pout, qr, kc, vc, shared, lens, 0.09, 160, 2, 4, d_err=err)
        torch.cuda.synchronize()
        return qr, out, t, wout, wt, kept, nl, nt, pout, kc[off:off + n], vc[off:off + n]
    for i, (x, y) in enumerate(zip(run(*small, 0), run(*big, far))):
        assert torch.equal(x, y), i
    assert int(err.item()) == 0


def test_two_streams_at_once():
    """The same calls from two streams, with workspaces of their own, side by side."""
    jobs = []
    for i, lens in enumerate(([900, 300, 77], [1200, 64, 500])):
        kc, vc, old, new = make_pool(lens, 2, 128, 16, "bf16", DEV, 50 + i, extra=[64] * 3)
        g = torch.Generator().manual_seed(i)
        q, tot = torch.randn((3, 16, 128), generator=g).bfloat16().to(DEV), torch.rand((3, 2, 1200), generator=g).to(DEV)
        n, ml = torch.tensor(lens, dtype=torch.int32, device=DEV), max(lens)
        one = old[:1].repeat(3, 1).contiguous()       # three samples of the first sequence
        same = torch.full_like(n, lens[0])
        res = dict(out=torch.empty_like(q), t=torch.zeros_like(tot), kept=torch.empty((3, 2, 64), dtype=torch.int32, device=DEV),
                   nl=torch.empty_like(n), nt=torch.empty_like(tot), pout=torch.empty_like(q))
        ws = (pa.decode_weights_workspace(q, 2, 16, ml), pa.evict_workspace(kc),
              pa.decode_common_prefix_workspace(q, 2, 16, ml, 3, 20))

        def job(stream, kc=kc, vc=vc, old=old, new=new, q=q, tot=tot, n=n, ml=ml, one=one, same=same, r=res, ws=ws):
            pa.pa_decode_weights(r["out"], q, kc, vc, old, n, 0.09, ml, tot, r["t"], workspace=ws[0], stream=stream)
            pa.pa_evict(kc, vc, r["t"], old, n, new, r["nl"], r["nt"], r["kept"], 64, 4, 16, ml, workspace=ws[1], stream=stream)
            pa.pa_decode_common_prefix(r["pout"], q, kc, vc, one, same, 0.09, ml, 3, 20, workspace=ws[2], stream=stream)
        job(None)
        torch.cuda.synchronize()
        jobs.append((job, res, {k: x.clone() for k, x in res.items()}))
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(8):
        for (job, _, _), s in zip(jobs, streams):
            job(s)
    torch.cuda.synchronize()
    for _, res, want in jobs:
        for name, x in want.items():
            assert torch.equal(res[name], x), name
