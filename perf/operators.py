"""Cases of the operators of a decode step over a bounded or shared paged cache.

Four operators, each in its plain form (elementary torch operations) and as a
call of the library:

  rotary    rotate queries and keys by positions with several axes and write
            the keys and values into their cache slots;
  weights   single-query attention that also adds each cached token's
            attention weight to a running total;
  evict     keep the tokens with the largest totals and move them, in order,
            into fresh blocks;
  prefix    single-query attention for a batch that shares a long prefix.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one new token of one image-and-text conversation: latency alone
        dict(name="rotary_one_token", op="rotary", tokens=1, heads=32, kv_heads=8, head_dim=128, rot_dim=128, axes=3,
             style="halves", dtype="bf16", block_size=16, padded=False, shape_seed=1),
        # an odd chunk whose head keeps half of its dimensions unrotated, with padding rows (slot -1)
        dict(name="rotary_pairs_1021", op="rotary", tokens=1021, heads=40, kv_heads=40, head_dim=128, rot_dim=64, axes=2,
             style="pairs", dtype="f16", block_size=16, padded=True, shape_seed=2),
        # a long prompt of text and image patches, time / height / width positions
        dict(name="rotary_prompt_8192", op="rotary", tokens=8192, heads=64, kv_heads=8, head_dim=128, rot_dim=128, axes=3,
             style="halves", dtype="bf16", block_size=16, padded=False, shape_seed=3),
        # four short chats: latency alone
        dict(name="weights_4_short", op="weights", seqs=4, queries=1, low=17, high=64, heads=4, kv_heads=4, head_dim=64,
             block_size=16, dtype="f16", shape_seed=4),
        # an ordinary serving step of many sequences
        dict(name="weights_gqa_b256", op="weights", seqs=256, queries=1, low=1, high=4096, heads=32, kv_heads=8,
             head_dim=128, block_size=16, dtype="bf16", shape_seed=5),
        # the last 16 positions of one prompt observe its whole cache before it is cut down
        dict(name="weights_window_16", op="weights", seqs=1, queries=16, low=8191, high=8191, heads=32, kv_heads=8,
             head_dim=128, block_size=16, dtype="f16", shape_seed=6),
        # few long sequences, eight query heads to a kv head
        dict(name="weights_long_b8", op="weights", seqs=8, queries=1, low=16384, high=65536, heads=64, kv_heads=8,
             head_dim=128, block_size=32, dtype="bf16", shape_seed=7),
        # three short chats cut down to 48 tokens: latency alone; one of them is shorter than that already
        dict(name="evict_3_short", op="evict", seqs=3, low=40, high=200, keep=48, sink=4, recent=16, kv_heads=4,
             head_dim=64, block_size=16, dtype="f16", shape_seed=8),
        # a serving batch cut back to 1024 tokens each
        dict(name="evict_b64_1024", op="evict", seqs=64, low=1025, high=4096, keep=1024, sink=4, recent=256, kv_heads=8,
             head_dim=128, block_size=16, dtype="bf16", shape_seed=9),
        # two long prompts cut to a quarter
        dict(name="evict_long_16384", op="evict", seqs=2, low=65000, high=65536, keep=16384, sink=16, recent=1024,
             kv_heads=8, head_dim=128, block_size=32, dtype="bf16", shape_seed=10),
        # two prompts of twelve samples each, one head to a kv head
        dict(name="prefix_2x12", op="prefix", groups=2, size=12, prefix=992, low=0, high=200, heads=16, kv_heads=16,
             head_dim=128, block_size=16, dtype="f16", shape_seed=11),
        # a whole batch behind one long system prompt
        dict(name="prefix_256_8192", op="prefix", groups=1, size=256, prefix=8192, low=1, high=512, heads=64, kv_heads=8,
             head_dim=128, block_size=16, dtype="bf16", shape_seed=12),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rotary", "weights", "evict", "prefix"])
    seed = rng.randrange(1 << 30)
    dtype = rng.choice(["f16", "bf16"])
    if op == "rotary":
        dim = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8, 16, 40])
        group = rng.choice([1, 2, 4, 8])
        if kv * group > 64:
            group = 1
        return dict(op=op, tokens=_log_int(rng, 1, 8192), heads=kv * group, kv_heads=kv, head_dim=dim,
                    rot_dim=rng.choice([dim, dim, dim // 2]), axes=rng.choice([1, 2, 3]),
                    style=rng.choice(["halves", "pairs"]), dtype=dtype, block_size=rng.choice([8, 16, 32, 64, 128]),
                    padded=rng.random() < 0.5, shape_seed=seed)
    if op == "weights":
        kv = rng.choice([1, 2, 4, 8])
        queries = rng.choice([1, 1, 1, 2, 5, 16])
        seqs = _log_int(rng, 1, 256 // queries)
        # seqs * high stays under half of the long case's tokens
        high = _log_int(rng, 16, min(65536, max(64, 131072 // (seqs * queries))))
        return dict(op=op, seqs=seqs, queries=queries, low=max(1, high // rng.choice([1, 2, 64])), high=high,
                    heads=kv * rng.choice([1, 2, 4, 8]), kv_heads=kv, head_dim=rng.choice([64, 128, 128]),
                    block_size=rng.choice([8, 16, 32, 64, 128]), dtype=dtype, shape_seed=seed)
    if op == "evict":
        seqs = _log_int(rng, 1, 64)
        high = _log_int(rng, 32, 131072 // seqs)
        keep = _log_int(rng, 8, max(8, high))
        sink = rng.randrange(0, keep // 4 + 1)
        return dict(op=op, seqs=seqs, low=max(1, high // rng.choice([1, 2, 8])), high=high, keep=keep, sink=sink,
                    recent=rng.randrange(0, (keep - sink) // 2 + 1), kv_heads=rng.choice([1, 2, 4, 8]),
                    head_dim=rng.choice([64, 128]), block_size=rng.choice([8, 16, 32, 64, 128]), dtype=dtype,
                    shape_seed=seed)
    bs = rng.choice([16, 32, 64, 128])
    size = _log_int(rng, 2, 256)
    kv = rng.choice([1, 2, 4, 8])
    return dict(op=op, groups=rng.choice([1, 1, 2, 3]) if size <= 64 else 1, size=size,
                prefix=bs * _log_int(rng, 1, 8192 // bs), low=0, high=_log_int(rng, 1, 512),
                heads=kv * rng.choice([1, 2, 4, 8]), kv_heads=kv, head_dim=128, block_size=bs, dtype=dtype, shape_seed=seed)


# ---------------------------------------------------------------- inputs

def _shape_rng(case):
    return np.random.Generator(np.random.PCG64(case["shape_seed"]))


def _lens(case):
    """Context lengths: part of the case, the same for every seed."""
    n = case["groups"] * case["size"] if case["op"] == "prefix" else case["seqs"]
    return _shape_rng(case).integers(case["low"], case["high"] + 1, size=n).astype(np.int64)


def _blocks(n, bs):
    return -(-n // bs)


def _randn(shape, dtype, gen):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen)


def _deal(counts, perm):
    """Block-table rows (int32, -1 past each row's count) with ids dealt out of perm."""
    width = max(1, max(counts))
    table = np.full((len(counts), width), -1, np.int32)
    at = 0
    for i, n in enumerate(counts):
        table[i, :n] = perm[at:at + n]
        at += n
    return table


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.Generator(np.random.PCG64(seed))
    return {"rotary": _prepare_rotary, "weights": _prepare_weights, "evict": _prepare_evict,
            "prefix": _prepare_prefix}[case["op"]](case, gen, rng)


def _prepare_rotary(case, gen, rng):
    T, A, D, bs = case["tokens"], case["axes"], case["head_dim"], case["block_size"]
    hq, hk = case["heads"], case["kv_heads"]
    dt = DTYPES[case["dtype"]]
    # the rows of one fused projection: queries, keys and values side by side
    qkv = _randn((T, hq + 2 * hk, D), dt, gen)
    # a conversation some way in: text runs (all axes alike), images (a frame number, then row and column)
    pos = np.zeros((A, T), np.int32)
    at, p = 0, int(rng.integers(0, 200000))
    while at < T:
        n = min(T - at, int(rng.integers(1, 400)))
        if A > 1 and rng.random() < 0.6:
            side = int(rng.integers(2, 40))
            i = np.arange(n)
            grid = [p + 0 * i, p + (i // side), p + (i % side)]
            pos[:, at:at + n] = np.stack(grid[3 - A:])
        else:
            pos[:, at:at + n] = p + np.arange(n)
        p = int(pos[:, at:at + n].max()) + 1
        at += n
    nb = _blocks(T + bs, bs) + 3
    slots = rng.permutation(nb)[np.arange(T) // bs] * bs + np.arange(T) % bs
    if case["padded"]:
        slots = np.where(rng.random(T) < 0.1, -1, slots)
    half = case["rot_dim"] // 2
    inv_freq = (1.0e6 ** (-np.arange(half) / half)).astype(np.float32)
    # contiguous sections of the frequencies, one per axis
    pair_axis = np.minimum(np.arange(half) * A // half, A - 1).astype(np.int32)
    return dict(case=case, query=qkv[:, :hq], key=qkv[:, hq:hq + hk], value=qkv[:, hq + hk:],
                query_out=torch.zeros((T, hq, D), dtype=dt, device="cuda"),
                k_cache=_randn((nb, hk, bs, D), dt, gen), v_cache=_randn((nb, hk, bs, D), dt, gen),
                positions=torch.as_tensor(pos).cuda(), slot_mapping=torch.as_tensor(slots.astype(np.int64)).cuda(),
                inv_freq=torch.as_tensor(inv_freq).cuda(), pair_axis=pair_axis)


def _pool(case, table_counts, gen, rng):
    bs, hk, D = case["block_size"], case["kv_heads"], case["head_dim"]
    nb = sum(table_counts) + 8
    dt = DTYPES[case["dtype"]]
    table = _deal(table_counts, rng.permutation(nb))
    return _randn((nb, hk, bs, D), dt, gen), _randn((nb, hk, bs, D), dt, gen), table


def _prepare_weights(case, gen, rng):
    n, w, bs = case["seqs"], case["queries"], case["block_size"]
    lens = _lens(case)
    kc, vc, table = _pool(case, [_blocks(int(x), bs) for x in lens], gen, rng)
    # row r's w queries are its last w positions (fewer in a shorter context): each sees the tokens up to its own
    ctx = np.maximum(np.repeat(lens, w) - np.tile(np.arange(w)[::-1], n), 0)
    B, hq, hk, D = n * w, case["heads"], case["kv_heads"], case["head_dim"]
    dt = DTYPES[case["dtype"]]
    wlen = int(lens.max())
    total = torch.rand((n, hk, wlen), dtype=torch.float32, device="cuda", generator=gen)
    state = dict(case=case, query=_randn((B, hq, D), dt, gen), k_cache=kc, v_cache=vc,
                 out=torch.zeros((B, hq, D), dtype=dt, device="cuda"),
                 block_tables=torch.as_tensor(np.repeat(table, w, axis=0)).cuda(),
                 context_lens=torch.as_tensor(ctx.astype(np.int32)).cuda(), max_len=wlen, scale=1.0 / math.sqrt(D),
                 weights=total, weights_out=torch.zeros_like(total), lens=ctx)
    if own:
        import paged_kv_cache_224_gb300 as pa
        state["workspace"] = pa.decode_weights_workspace(state["query"], hk, bs, wlen, queries_per_row=w)
    return state


def _prepare_evict(case, gen, rng):
    bs, hk, D, keep = case["block_size"], case["kv_heads"], case["head_dim"], case["keep"]
    lens = _lens(case)
    n = len(lens)
    old = [_blocks(int(x), bs) for x in lens]
    new = [_blocks(min(int(x), keep), bs) for x in lens]
    kc, vc, both = _pool(case, old + new, gen, rng)
    wlen = int(lens.max())
    # running totals: a few tokens gather most of the attention; many recent ones have none yet, so ties are common
    total = torch.rand((n, hk, wlen), dtype=torch.float32, device="cuda", generator=gen) ** 6
    total = torch.where(torch.rand((n, hk, wlen), device="cuda", generator=gen) < 0.15, torch.zeros_like(total), total)
    state = dict(case=case, k_cache=kc, v_cache=vc, weights=total,
                 block_tables=torch.as_tensor(both[:n, :max(old)].copy()).cuda(),
                 new_block_tables=torch.as_tensor(both[n:, :max(new)].copy()).cuda(),
                 context_lens=torch.as_tensor(lens.astype(np.int32)).cuda(), max_len=wlen,
                 new_context_lens=torch.zeros(n, dtype=torch.int32, device="cuda"),
                 new_weights=torch.zeros_like(total), kept=torch.full((n, hk, keep), -1, dtype=torch.int32, device="cuda"),
                 lens=lens)
    if own:
        import paged_kv_cache_224_gb300 as pa
        state["workspace"] = pa.evict_workspace(kc, n, keep)
    return state


def _prepare_prefix(case, gen, rng):
    g, size, bs = case["groups"], case["size"], case["block_size"]
    pre = case["prefix"] // bs
    tails = _lens(case)
    B, hq, hk, D = g * size, case["heads"], case["kv_heads"], case["head_dim"]
    kc, vc, dealt = _pool(case, [pre] * g + [_blocks(int(t), bs) for t in tails], gen, rng)
    own_blocks = max(1, max(_blocks(int(t), bs) for t in tails))
    table = np.full((B, pre + own_blocks), -1, np.int32)
    for s in range(B):
        table[s, :pre] = dealt[s // size, :pre]
        table[s, pre:] = dealt[g + s, :own_blocks]
    dt = DTYPES[case["dtype"]]
    lens = tails + case["prefix"]
    state = dict(case=case, query=_randn((B, hq, D), dt, gen), k_cache=kc, v_cache=vc,
                 out=torch.zeros((B, hq, D), dtype=dt, device="cuda"), block_tables=torch.as_tensor(table).cuda(),
                 context_lens=torch.as_tensor(lens.astype(np.int32)).cuda(), max_len=int(lens.max()),
                 scale=1.0 / math.sqrt(D), tails=tails, prefix_blocks=pre)
    if own:
        import paged_kv_cache_224_gb300 as pa
        state["workspace"] = pa.decode_common_prefix_workspace(state["query"], hk, bs, state["max_len"], size, pre)
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    return {"rotary": _run_rotary, "weights": _run_weights, "evict": _run_evict, "prefix": _run_prefix}[state["case"]["op"]](state)


def _run_rotary(s):
    if own:
        import paged_kv_cache_224_gb300 as pa
        pa.pa_rotary_and_cache(s["query_out"], s["query"], s["key"], s["value"], s["k_cache"], s["v_cache"],
                               s["positions"], s["slot_mapping"], s["inv_freq"], s["pair_axis"],
                               interleaved=s["case"]["style"] == "pairs")
        return s["query_out"], s["k_cache"], s["v_cache"]
    axis = torch.as_tensor(s["pair_axis"], dtype=torch.long, device="cuda")
    angle = s["positions"].double()[axis].t() * s["inv_freq"].double()  # [T][pairs]; far positions need 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turn(x):
        y = x.float()
        half = cos.shape[-1]
        if s["case"]["style"] == "pairs":
            a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:2 * half]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
        return torch.cat((r, y[..., 2 * half:]), dim=-1).to(x.dtype)

    s["query_out"].copy_(turn(s["query"]))
    used = s["slot_mapping"] >= 0
    slot = s["slot_mapping"][used]
    bs = s["k_cache"].shape[2]
    s["k_cache"][slot // bs, :, slot % bs] = turn(s["key"])[used]
    s["v_cache"][slot // bs, :, slot % bs] = s["value"][used]
    return s["query_out"], s["k_cache"], s["v_cache"]


def _rows(cache, blocks, n):
    """The first n rows of the blocks, per kv head: [kv heads][n][head_dim], 32 bits."""
    x = cache[blocks.long()].float()
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def _softmax(x):
    e = torch.exp(x - x.max(-1, keepdim=True).values)
    return e / e.sum(-1, keepdim=True)


def _run_weights(s):
    if own:
        import paged_kv_cache_224_gb300 as pa
        pa.pa_decode_weights(s["out"], s["query"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                             s["scale"], s["max_len"], s["weights"], s["weights_out"],
                             queries_per_row=s["case"]["queries"], workspace=s["workspace"])
        return s["out"], s["weights_out"]
    w, bs = s["case"]["queries"], s["case"]["block_size"]
    for r in range(s["weights"].shape[0]):
        longest = max(int(x) for x in s["lens"][r * w:(r + 1) * w])
        total = s["weights"][r].clone()
        for i in range(r * w, (r + 1) * w):
            n = int(s["lens"][i])
            if n == 0:
                s["out"][i] = 0
                continue
            blocks = s["block_tables"][i, :_blocks(n, bs)]
            K, V = _rows(s["k_cache"], blocks, n), _rows(s["v_cache"], blocks, n)
            q = s["query"][i].float().reshape(K.shape[0], -1, K.shape[2])
            p = _softmax(torch.matmul(q, K.transpose(1, 2)) * s["scale"])
            s["out"][i] = torch.matmul(p, V).reshape(-1, K.shape[2]).to(s["out"].dtype)
            total[:, :n] += p.sum(1)
        s["weights_out"][r, :, :longest] = total[:, :longest]
    return s["out"], s["weights_out"]


def _run_evict(s):
    c = s["case"]
    if own:
        import paged_kv_cache_224_gb300 as pa
        pa.pa_evict(s["k_cache"], s["v_cache"], s["weights"], s["block_tables"], s["context_lens"], s["new_block_tables"],
                    s["new_context_lens"], s["new_weights"], s["kept"], c["keep"], c["sink"], c["recent"], s["max_len"],
                    workspace=s["workspace"])
        return s["k_cache"], s["v_cache"], s["kept"], s["new_context_lens"], s["new_weights"]
    bs, keep, sink, recent = c["block_size"], c["keep"], c["sink"], c["recent"]
    head = torch.arange(c["kv_heads"], device="cuda")[:, None]
    for i in range(len(s["lens"])):
        n = int(s["lens"][i])
        m = min(n, keep)
        idx = torch.arange(n, device="cuda").expand(c["kv_heads"], n)
        if n > keep:
            order = torch.argsort(s["weights"][i, :, sink:n - recent], dim=-1, descending=True, stable=True) + sink
            idx = torch.cat((idx[:, :sink], order[:, :keep - sink - recent], idx[:, n - recent:]), dim=-1).sort(-1).values
        block, row = s["block_tables"][i].long()[idx // bs], idx % bs
        j = torch.arange(m, device="cuda")
        new_block, new_row = s["new_block_tables"][i].long()[j // bs], j % bs
        for cache in (s["k_cache"], s["v_cache"]):
            cache[new_block[None], head, new_row[None]] = cache[block, head, row]
        s["kept"][i, :, :m] = idx.int()
        s["kept"][i, :, m:] = -1
        s["new_weights"][i, :, :m] = s["weights"][i].gather(1, idx)
        s["new_weights"][i, :, m:] = 0
        s["new_context_lens"][i] = m
    return s["k_cache"], s["v_cache"], s["kept"], s["new_context_lens"], s["new_weights"]


def _run_prefix(s):
    c = s["case"]
    if own:
        import paged_kv_cache_224_gb300 as pa
        pa.pa_decode_common_prefix(s["out"], s["query"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                                   s["scale"], s["max_len"], c["size"], s["prefix_blocks"], workspace=s["workspace"])
        return s["out"]
    bs, pre = c["block_size"], s["prefix_blocks"]
    for g in range(c["groups"]):
        table = s["block_tables"][g * c["size"]:(g + 1) * c["size"]]
        Kp, Vp = _rows(s["k_cache"], table[0, :pre], pre * bs), _rows(s["v_cache"], table[0, :pre], pre * bs)
        for k in range(c["size"]):
            i = g * c["size"] + k
            n = int(s["tails"][i])
            blocks = table[k, pre:pre + _blocks(n, bs)]
            q = s["query"][i].float().reshape(Kp.shape[0], -1, Kp.shape[2])
            x = torch.matmul(q, Kp.transpose(1, 2))
            if n:
                x = torch.cat((x, torch.matmul(q, _rows(s["k_cache"], blocks, n).transpose(1, 2))), dim=-1)
            p = _softmax(x * s["scale"])
            o = torch.matmul(p[..., :pre * bs], Vp)
            if n:
                o = o + torch.matmul(p[..., pre * bs:], _rows(s["v_cache"], blocks, n))
            s["out"][i] = o.reshape(-1, Kp.shape[2]).to(s["out"].dtype)
    return s["out"]


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "weights": _exact_weights, "evict": _exact_evict, "prefix": _exact_prefix}[case["op"]](s)


def _exact_rotary(s):
    """Each pair is a complex number times e^(i angle)."""
    axis = s["pair_axis"]
    pos = s["positions"].cpu().numpy().astype(np.float64)
    angle = torch.as_tensor(np.stack([pos[a] for a in axis], axis=1) * s["inv_freq"].cpu().numpy().astype(np.float64)).cuda()
    unit = torch.polar(torch.ones_like(angle), angle)
    R = 2 * len(axis)

    def turn(x):
        x = x.double().clone()
        re, im = (slice(0, R, 2), slice(1, R, 2)) if s["case"]["style"] == "pairs" else (slice(0, R // 2), slice(R // 2, R))
        z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * unit[:, None]
        x[..., re], x[..., im] = z.real, z.imag
        return x

    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    rk = turn(s["key"])
    slots = s["slot_mapping"].cpu()
    bs = kc.shape[2]
    t = torch.nonzero(slots >= 0)[:, 0]
    b, r = (slots[t] // bs).cuda(), (slots[t] % bs).cuda()
    kc[b, :, r] = rk[t.cuda()]
    vc[b, :, r] = s["value"].double()[t.cuda()]
    return turn(s["query"]), kc, vc


def _gathered(cache, table, n, bs):
    """Rows 0 .. n-1 of a sequence in 64 bits, token by token through its table: [n][kv heads][head_dim]."""
    j = torch.arange(n, device="cuda")
    return cache[table.long()[j // bs], :, j % bs].double()


def _attend64(q, K, V, scale):
    """q [heads][D], K and V [n][kv heads][D] -> output [heads][D] and weights [heads][n], by definition."""
    kv = K.shape[1]
    per = q.shape[0] // kv
    out, p = [], []
    for h in range(kv):
        z = (q[h * per:(h + 1) * per] @ K[:, h].t()) * scale
        z = torch.exp(z - z.amax(1, keepdim=True))
        z = z / z.sum(1, keepdim=True)
        out.append(z @ V[:, h])
        p.append(z.sum(0))
    return torch.cat(out), torch.stack(p)


def _exact_weights(s):
    bs, w = s["case"]["block_size"], s["case"]["queries"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    total = s["weights_out"].double()
    for i in range(out.shape[0]):
        r, n = i // w, int(s["lens"][i])
        longest = int(max(s["lens"][r * w:(r + 1) * w]))
        if i % w == 0:
            total[r, :, :longest] = s["weights"][r, :, :longest].double()
        if n == 0:
            continue
        K, V = (_gathered(s[c], s["block_tables"][i], n, bs) for c in ("k_cache", "v_cache"))
        out[i], p = _attend64(s["query"][i].double(), K, V, s["scale"])
        total[r, :, :n] += p
    return out, total


def _exact_evict(s):
    """Row by row on the host: the protected tokens, then the largest totals, the lower index first among equals."""
    c, bs = s["case"], s["case"]["block_size"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    src_k, src_v = s["k_cache"], s["v_cache"]
    W = s["weights"].cpu().numpy()
    old, new = s["block_tables"].cpu().numpy(), s["new_block_tables"].cpu().numpy()
    kept = np.full(s["kept"].shape, -1, np.int32)
    lens = np.zeros(len(s["lens"]), np.int32)
    total = np.zeros(W.shape, np.float64)
    for i, n in enumerate(int(x) for x in s["lens"]):
        m = lens[i] = min(n, c["keep"])
        for h in range(c["kv_heads"]):
            rank = np.lexsort((np.arange(n), -W[i, h, :n].astype(np.float64)))
            must = np.zeros(n, bool)
            must[:c["sink"]] = True
            must[max(0, n - c["recent"]):] = True
            if n > m:
                rank = rank[~must[rank]][:m - int(must.sum())]
                must[rank] = True
                idx = np.nonzero(must)[0]
            else:
                idx = np.arange(n)
            kept[i, h, :m] = idx
            total[i, h, :m] = W[i, h, idx]
            j = np.arange(m)
            put = torch.as_tensor(new[i, j // bs].astype(np.int64)).cuda(), torch.as_tensor(j % bs).cuda()
            get = torch.as_tensor(old[i, idx // bs].astype(np.int64)).cuda(), torch.as_tensor(idx % bs).cuda()
            kc[put[0], h, put[1]] = src_k[get[0], h, get[1]].double()
            vc[put[0], h, put[1]] = src_v[get[0], h, get[1]].double()
    return kc, vc, torch.as_tensor(kept).cuda(), torch.as_tensor(lens).cuda(), torch.as_tensor(total).cuda()


def _exact_prefix(s):
    """Attention over each sequence's whole context; that a prefix is shared plays no part."""
    bs = s["case"]["block_size"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lens = s["context_lens"].tolist()
    for i, n in enumerate(lens):
        K, V = (_gathered(s[c], s["block_tables"][i], n, bs) for c in ("k_cache", "v_cache"))
        out[i] = _attend64(s["query"][i].double(), K, V, s["scale"])[0]
    return out


# ---------------------------------------------------------------- the work of one pass

def work(case):
    op, D = case["op"], case["head_dim"]
    hk = case["kv_heads"]
    if op == "rotary":
        T, hq = case["tokens"], case["heads"]
        # queries, keys and values read and written once, positions, slots and frequencies read
        return dict(bytes=2 * 2 * T * (hq + 2 * hk) * D + T * (4 * case["axes"] + 8) + 2 * case["rot_dim"],
                    flops=3 * T * (hq + hk) * case["rot_dim"])
    lens = _lens(case)
    bs = case["block_size"]
    if op == "weights":
        w, hq = case["queries"], case["heads"]
        tokens = int(lens.sum())
        B = case["seqs"] * w
        ctx = np.maximum(np.repeat(lens, w) - np.tile(np.arange(w)[::-1], case["seqs"]), 0)
        # every K and V row once, queries and outputs, tables and lengths, the totals read and written
        return dict(bytes=tokens * hk * D * 4 + 4 * B * hq * D + 4 * int(sum(_blocks(int(x), bs) for x in ctx)) + 4 * B +
                    8 * tokens * hk, flops=int(4 * D * hq * ctx.sum()))
    if op == "evict":
        kept = np.minimum(lens, case["keep"])
        tokens, m = int(lens.sum()), int(kept.sum())
        # totals read, kept K and V rows read and written, new totals and indices written, tables read
        return dict(bytes=4 * tokens * hk + 2 * 4 * m * hk * D + 4 * len(lens) * hk * int(lens.max()) +
                    4 * len(lens) * hk * case["keep"] + 4 * int(sum(_blocks(int(x), bs) for x in lens)) +
                    4 * int(sum(_blocks(int(x), bs) for x in kept)) + 8 * len(lens), flops=0)
    B, hq, pre = case["groups"] * case["size"], case["heads"], case["prefix"]
    # every prefix row once a group, every own row once, queries and outputs, tables and lengths
    return dict(bytes=(case["groups"] * pre + int(lens.sum())) * hk * D * 4 + 4 * B * hq * D +
                4 * int(sum(pre // bs + _blocks(int(t), bs) for t in lens)) + 4 * B,
                flops=int(4 * D * hq * (B * pre + lens.sum())))
