"""The 8-bit cache as an engine uses it: prompts normed, rotated and written chunk by
chunk with attention after each chunk, a sample forked off (blocks shared, copied on its
first token), then decode steps of all sequences.  The block manager gives slots, tables
and copy pairs.

At every step the attention has to be that of the cached values in 64 bits (the
decode's and the prefill's own bounds), and every cached row within the codes' rounding
of the exact key or value: half a step of it, 2^-4 |x|, and half of the smallest code
step, 2^-10 of the block's scale, for itself and for each time that its scale grew (a
scale that ends at 2^e grew from at least 2^-64 in powers of two: those roundings add up
to less than 2^-10 (1 + 1/2 + 1/4 + ...) 2^e = 2^-9 2^e)."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_224_gb300 as pa
from tests import ref8

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
D = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


class Engine:
    def __init__(self, Hq, Hkv, bs, dtype, graph, seed):
        self.Hq, self.Hkv, self.bs, self.dt = Hq, Hkv, bs, dtype
        self.g = torch.Generator().manual_seed(seed)
        nb = 64
        self.bm = pa.BlockManager(nb, bs)
        # what earlier owners of the blocks left: NaN, under large scales
        self.kc, self.vc = (torch.full((nb, Hkv, bs, D), 0x7f, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
                            for _ in range(2))
        self.ks, self.vs = (torch.full((nb, Hkv), 200, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu) for _ in range(2))
        self.inv = torch.as_tensor((1e4 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32), device=DEV)
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=self.g)).to(dtype).to(DEV) for _ in range(2))
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.rows = {}  # sequence -> [(exact key, its fp32 error, value)] by position
        self.graph = graph

    def qkv(self, n):
        # tokens of very different sizes: scales have to grow
        x = torch.randn((n, self.Hq + 2 * self.Hkv, D), generator=self.g) * torch.exp2(3 * torch.rand((n, 1, 1), generator=self.g))
        return x.to(self.dt).to(DEV)

    def write(self, seqs, positions, slots, x):
        """Norm, rotate and write rows x of these sequences' tokens; the rotated queries."""
        q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]
        out = torch.empty(q.shape, dtype=self.dt, device=DEV)
        pos = torch.tensor(positions, dtype=torch.int32, device=DEV)
        pa.pa_rotary_and_cache_fp8(out, q, k, v, self.kc, self.vc, self.ks, self.vs, pos, torch.tensor(slots, device=DEV), self.inv,
                                   self.wq, self.wk, 1e-6, d_err=self.err)
        y = ref8.normed(k, self.wk, 1e-6)
        exact = ref8.turned(y, pos, self.inv, None, False)
        half = D // 2
        both = y.abs() + torch.cat((y[..., half:], y[..., :half]), -1).abs()
        for i, s in enumerate(seqs):
            assert len(self.rows.setdefault(s, [])) == positions[i]
            self.rows[s].append((exact[i], both[i] * (2.0 ** -20 + 2.0 ** -21), v[i].cpu().double()))
        return out

    def cached(self, s, n):
        """The sequence's cached values, checked against its exact rows."""
        t = torch.as_tensor(self.bm.tables([s]))[0].long()
        j = torch.arange(n)
        b, r = t[j // self.bs], j % self.bs
        got = []
        for cache, scales, which in ((self.kc, self.ks, 0), (self.vc, self.vs, 2)):
            x = ref8.values(cache, scales)[b, :, r]
            sc = ref8.scale_values(scales)[b][..., None]
            want = torch.stack([row[which] for row in self.rows[s][:n]])
            slack = torch.stack([row[1] for row in self.rows[s][:n]]) if which == 0 else torch.zeros_like(want)
            assert bool(((x - want).abs() <= want.abs() * 2.0 ** -4 * 1.001 + sc * 2.0 ** -9 + 2 * slack).all())
            got.append(x)
        return got

    def near(self, got, q, K, V, weight):
        want, mean, size = ref8.attend_sizes(q.cpu().double(), K, V, self.scale)
        h = torch.finfo(self.dt).eps / 2
        n = K.shape[0]
        rel = weight + 2 * (2 * (D + 8) * 2.0 ** -24 * size + 2.0 ** -22) + 2 * n * 2.0 ** -24 + 2.0 ** -20
        bound = want.abs() * h * (1 + 2.0 ** -10) + mean * rel[:, None] + 2.0 ** -25
        if self.dt == torch.float16:
            bound += 2.0 ** -25 * V.abs().sum(0).repeat_interleave(self.Hq // self.Hkv, 0)
        assert bool(((got.cpu().double() - want).abs() <= bound).all())

    scale = 1 / math.sqrt(D)


@pytest.mark.parametrize("Hq,Hkv,bs,dtype,graph", [(8, 1, 16, torch.bfloat16, False), (8, 2, 32, torch.float16, True),
                                                   (4, 4, 16, torch.bfloat16, True)])
def test_prompts_chunks_a_fork_and_decode_steps(Hq, Hkv, bs, dtype, graph):
    e = Engine(Hq, Hkv, bs, dtype, graph, seed=Hq + bs)
    prompts = {0: 75, 1: 33}
    slots = {s: e.bm.add_sequence(s, np.arange(1000 * s, 1000 * s + n))[0] for s, n in prompts.items()}
    done = {s: 0 for s in prompts}
    while any(done[s] < prompts[s] for s in prompts):
        take = {s: min(29, prompts[s] - done[s]) for s in prompts}          # chunks that end inside blocks
        order = [(s, done[s] + i) for s in prompts for i in range(take[s])]
        x = e.qkv(len(order))
        q = e.write([s for s, _ in order], [p for _, p in order], [int(slots[s][p]) for s, p in order], x)
        out = torch.full_like(q, float("nan"))
        pa.pa_prefill_batch_fp8(out, q, e.kc, e.vc, e.ks, e.vs, torch.as_tensor(e.bm.tables(list(prompts)), device=DEV),
                                [done[s] for s in prompts], [take[s] for s in prompts], e.scale, d_err=e.err)
        torch.cuda.synchronize()
        assert int(e.err.item()) == 0
        at = 0
        for s in prompts:
            if take[s]:
                K, V = e.cached(s, done[s] + take[s])
            for i in range(take[s]):
                m = done[s] + i + 1
                e.near(out[at + i], q[at + i], K[:m], V[:m], torch.finfo(dtype).eps / 2)
            at += take[s]
            done[s] += take[s]
    e.bm.fork(0, 2)
    e.rows[2] = list(e.rows[0])
    seqs = [0, 1, 2]
    for step in range(bs + 4):
        pairs, slot, pos = [], [], []
        for s in seqs:
            pos.append(e.bm.seq_len(s))
            at, pair = e.bm.append_token(s, 5000 + 10 * step + s)
            slot.append(at)
            if pair:
                pairs.append(pair)
        assert bool(pairs) == (step == 0)  # the shared, partly filled block is copied once
        if pairs:
            pa.pa_copy_blocks_fp8(e.kc, e.vc, e.ks, e.vs, torch.tensor(pairs, device=DEV), d_err=e.err)
        q = e.write(seqs, pos, slot, e.qkv(len(seqs)))
        out = torch.full_like(q, float("nan"))
        most = max(pos) + 1
        args = (out, q, e.kc, e.vc, e.ks, e.vs, torch.as_tensor(e.bm.tables(seqs), device=DEV),
                torch.tensor([p + 1 for p in pos], dtype=torch.int32, device=DEV), e.scale, most)
        if graph:
            ws = pa.decode_fp8_workspace(q, Hkv, bs, most)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                pa.pa_decode_fp8(*args, workspace=ws, d_err=e.err)
            g.replay()
        else:
            pa.pa_decode_fp8(*args, d_err=e.err)
        torch.cuda.synchronize()
        assert int(e.err.item()) == 0
        for i, s in enumerate(seqs):
            K, V = e.cached(s, pos[i] + 1)
            e.near(out[i], q[i], K, V, 2.0 ** -12)
    for s in seqs:
        e.bm.free_sequence(s)


def test_more_copies_than_one_launch_looks_through():
    """Beyond 1024 pairs the conflicts are found through the workspace's table."""
    n, nb = 1500, 3100
    g = torch.Generator().manual_seed(3)
    kc, vc = (torch.randint(0, 256, (nb, 1, 8, 16), generator=g, dtype=torch.uint8).to(DEV) for _ in range(2))
    ks, vs = (torch.randint(0, 256, (nb, 1), generator=g, dtype=torch.uint8).to(DEV) for _ in range(2))
    perm = torch.randperm(nb, generator=g)
    pairs = torch.stack((perm[:n], perm[n:2 * n]), 1).to(DEV)
    want = []
    for x in (kc, vc, ks, vs):
        y = x.clone()
        y[pairs[:, 1]] = y[pairs[:, 0]]
        want.append(y)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_copy_blocks_fp8(kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), ks, vs, pairs, d_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for x, y in zip((kc, vc, ks, vs), want):
        assert torch.equal(x, y)
