"""Cases of the operators around a paged cache held in 8 bits.

The cache holds e4m3 codes, [blocks][kv heads][block size][head dim], and for
every block and kv head one power-of-two scale (e8m0, [blocks][kv heads]); a
row's values are its codes times its block's scale.  Five operators, each in
its plain form (elementary torch operations) and as a call of the library:

  norm      RMS norms of queries and keys for each head, the rotation by
            positions and the cache write in one pass, 16-bit cache;
  write8    the same into the 8-bit cache, with or without norms and rotation:
            a block's first row gives it a fresh scale, later rows may raise it;
  decode8   single-query attention over the 8-bit cache;
  prefill8  causal attention of prompt chunks over the 8-bit cache;
  copy8     copy-on-write of blocks with their scales.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
LOWEST = -64        # exponent of the smallest scale
F16_TOP = 61440.0   # the largest code times a power of two that fp16 holds
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one new token of one conversation: latency alone
        dict(name="norm_one_token", op="norm", tokens=1, heads=32, kv_heads=8, head_dim=128, rot_dim=128, axes=1,
             style="halves", dtype="bf16", block_size=16, padded=False, shape_seed=1),
        # a long prompt of a grouped-query model
        dict(name="norm_prompt_8192", op="norm", tokens=8192, heads=64, kv_heads=8, head_dim=128, rot_dim=128, axes=1,
             style="halves", dtype="bf16", block_size=16, padded=False, shape_seed=2),
        # a decode step: one token for each of many sequences, into partly filled blocks
        dict(name="write8_step_256", op="write8", path="norm", tokens=256, run=1, heads=32, kv_heads=8, head_dim=128,
             rot_dim=128, axes=1, style="halves", dtype="bf16", block_size=16, padded=False, shape_seed=3),
        # an odd chunk with padding rows, rotated without norms, half of each head unrotated
        dict(name="write8_pairs_1021", op="write8", path="rotary", tokens=1021, run=1021, heads=40, kv_heads=40, head_dim=128,
             rot_dim=64, axes=2, style="pairs", dtype="f16", block_size=16, padded=True, shape_seed=4),
        # a long prompt
        dict(name="write8_prompt_8192", op="write8", path="norm", tokens=8192, run=8192, heads=64, kv_heads=8, head_dim=128,
             rot_dim=128, axes=1, style="halves", dtype="bf16", block_size=16, padded=False, shape_seed=5),
        # four short chats: latency alone
        dict(name="decode8_4_short", op="decode8", seqs=4, low=17, high=64, heads=4, kv_heads=4, head_dim=64, block_size=16,
             dtype="f16", shape_seed=6),
        # an ordinary serving step of many sequences
        dict(name="decode8_gqa_b256", op="decode8", seqs=256, low=1, high=4096, heads=32, kv_heads=8, head_dim=128,
             block_size=16, dtype="bf16", shape_seed=7),
        # few long sequences, eight query heads to a kv head
        dict(name="decode8_long_b8", op="decode8", seqs=8, low=32768, high=131072, heads=64, kv_heads=8, head_dim=128,
             block_size=32, dtype="bf16", shape_seed=8),
        # three ragged chunks of short prompts, the first of them of one token
        dict(name="prefill8_3_ragged", op="prefill8", chunks="1,100,37", prefixes="40,0,700", heads=16, kv_heads=16,
             head_dim=128, block_size=16, dtype="f16", shape_seed=9),
        # one chunk of a long prompt
        dict(name="prefill8_8192_512", op="prefill8", chunks="512", prefixes="8192", heads=64, kv_heads=8, head_dim=128,
             block_size=16, dtype="bf16", shape_seed=10),
        # one sample diverges from its prompt
        dict(name="copy8_one", op="copy8", pairs=1, kv_heads=8, head_dim=128, block_size=16, dtype="bf16", shape_seed=11),
        # seven of eight samples of 32 prompts diverge in their partly filled block
        dict(name="copy8_224", op="copy8", pairs=224, kv_heads=40, head_dim=128, block_size=16, dtype="f16", shape_seed=12),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "write8", "write8", "decode8", "decode8", "prefill8", "copy8"])
    seed = rng.randrange(1 << 30)
    dtype = rng.choice(["f16", "bf16"])
    bs = rng.choice([16, 16, 32, 64, 128])
    if op in ("norm", "write8"):
        dim = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8, 16, 40])
        group = rng.choice([1, 2, 4, 8])
        if kv * group > 64:
            group = 1
        tokens = _log_int(rng, 1, 8192)
        case = dict(op=op, tokens=tokens, heads=kv * group, kv_heads=kv, head_dim=dim,
                    rot_dim=rng.choice([dim, dim, dim // 2]), axes=rng.choice([1, 2, 3]),
                    style=rng.choice(["halves", "pairs"]), dtype=dtype, block_size=rng.choice([8, bs]),
                    padded=rng.random() < 0.5, shape_seed=seed)
        if op == "write8":
            # tokens a sequence has in the call: a step of single tokens, or chunks
            case.update(path=rng.choice(["norm", "norm", "rotary", "plain"]), run=_log_int(rng, 1, tokens))
        return case
    if op == "decode8":
        kv = rng.choice([1, 2, 4, 8])
        seqs = _log_int(rng, 1, 256)
        high = _log_int(rng, 16, min(131072, 524288 // seqs))
        return dict(op=op, seqs=seqs, low=max(1, high // rng.choice([1, 2, 64])), high=high,
                    heads=kv * rng.choice([1, 2, 4, 8]), kv_heads=kv, head_dim=rng.choice([64, 128, 128]),
                    block_size=rng.choice([8, bs]), dtype=dtype, shape_seed=seed)
    if op == "prefill8":
        kv = rng.choice([1, 2, 4, 8, 16])
        heads = kv * rng.choice([1, 2, 4, 8])
        if heads > 64:
            heads = kv
        n = rng.choice([1, 1, 2, 3, 5])
        chunks = [_log_int(rng, 1, 512) for _ in range(n)]
        # rows times keys stay under the largest listed case's
        most = max(1, 512 * 8192 * 64 // (heads * max(chunks) * n) - max(chunks))
        prefixes = [rng.randrange(0, min(8192, most) + 1) for _ in range(n)]
        return dict(op=op, chunks=",".join(map(str, chunks)), prefixes=",".join(map(str, prefixes)), heads=heads,
                    kv_heads=kv, head_dim=128, block_size=bs, dtype=dtype, shape_seed=seed)
    return dict(op=op, pairs=_log_int(rng, 1, 512), kv_heads=rng.choice([1, 2, 8, 40]), head_dim=rng.choice([64, 128]),
                block_size=rng.choice([8, bs]), dtype=dtype, shape_seed=seed)


# ---------------------------------------------------------------- inputs

def _shape_rng(case):
    return np.random.Generator(np.random.PCG64(case["shape_seed"]))


def _blocks(n, bs):
    return -(-n // bs)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _lens(case):
    """Context lengths: part of the case, the same for every seed."""
    if case["op"] == "prefill8":
        return np.array(_ints(case["chunks"]), np.int64) + np.array(_ints(case["prefixes"]), np.int64)
    return _shape_rng(case).integers(case["low"], case["high"] + 1, size=case["seqs"]).astype(np.int64)


def _pow2(e, wide=False):
    """2^e for whole e of normal size, exact."""
    if wide:
        return (e.long() + 1023 << 52).view(torch.float64)
    return (e.int() + 127 << 23).view(torch.float32)


def _pool8(nb, kv, bs, D, gen):
    """Codes and scales as earlier writes left them: N(0, 1) rows, each block and head of a size of its own."""
    x = torch.randn((nb, kv, bs, D), device="cuda", generator=gen)
    size = torch.exp2(0.5 * torch.randn((nb, kv, 1, 1), device="cuda", generator=gen))
    m, e = torch.frexp((x.abs().amax((2, 3), keepdim=True) * size) / 448)
    e = torch.where(m == 0.5, e - 1, e)
    codes = (x * (size * _pow2(-e))).to(torch.float8_e4m3fn)
    scales = (e.reshape(nb, kv) + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return codes, scales


def _table(counts, perm):
    """Block-table rows (int32, -1 past each row's count) with ids dealt out of perm."""
    width = max(1, max(counts))
    at = np.concatenate([[0], np.cumsum(counts)[:-1]])[:, None] + np.arange(width)
    used = np.arange(width) < np.array(counts)[:, None]
    return torch.as_tensor(np.where(used, perm[np.minimum(at, len(perm) - 1)], -1).astype(np.int32)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.Generator(np.random.PCG64(seed))
    return {"norm": _prepare_write, "write8": _prepare_write, "decode8": _prepare_decode, "prefill8": _prepare_prefill,
            "copy8": _prepare_copy}[case["op"]](case, gen, rng)


def _prepare_write(case, gen, rng):
    T, A, D, bs = case["tokens"], case["axes"], case["head_dim"], case["block_size"]
    hq, hk = case["heads"], case["kv_heads"]
    dt = DTYPES[case["dtype"]]
    # the rows of one fused projection: queries, keys and values side by side
    qkv = torch.randn((T, hq + 2 * hk, D), dtype=dt, device="cuda", generator=gen)
    run = case.get("run", T)
    n = _blocks(T, run)  # sequences
    i = np.arange(T)
    # each sequence's rows go on from where it stands, in blocks of its own
    begin = rng.integers(0, 4 * bs, size=n)[i // run] if run < T or case["op"] == "write8" else np.zeros(T, np.int64)
    place = begin % bs + i % run
    width = _blocks(bs - 1 + run, bs)
    nb = n * width + 3
    blocks = rng.permutation(nb)[:n * width].reshape(n, width)
    slots = blocks[i // run, place // bs] * bs + place % bs
    if case["padded"]:
        slots = np.where(rng.random(T) < 0.1, -1, slots)
    # text: all axes alike, each sequence some way in
    pos = (rng.integers(0, 200000, size=n)[i // run] + i % run)[None] + np.zeros((A, 1), np.int64)
    half = case["rot_dim"] // 2
    state = dict(case=case, query=qkv[:, :hq], key=qkv[:, hq:hq + hk], value=qkv[:, hq + hk:],
                 positions=torch.as_tensor(pos.astype(np.int32)).cuda(),
                 slot_mapping=torch.as_tensor(slots.astype(np.int64)).cuda(),
                 inv_freq=torch.as_tensor((1.0e6 ** (-np.arange(half) / half)).astype(np.float32)).cuda(),
                 pair_axis=np.minimum(np.arange(half) * A // half, A - 1).astype(np.int32),
                 query_norm=(1 + 0.2 * torch.randn(D, device="cuda", generator=gen)).to(dt),
                 key_norm=(1 + 0.2 * torch.randn(D, device="cuda", generator=gen)).to(dt),
                 query_out=torch.zeros((T, hq, D), dtype=dt, device="cuda"))
    if case["op"] == "norm":
        state.update(k_cache=torch.randn((nb, hk, bs, D), dtype=dt, device="cuda", generator=gen),
                     v_cache=torch.randn((nb, hk, bs, D), dtype=dt, device="cuda", generator=gen))
    else:
        kc, ks = _pool8(nb, hk, bs, D, gen)
        vc, vs = _pool8(nb, hk, bs, D, gen)
        state.update(k_cache=kc, k_scales=ks, v_cache=vc, v_scales=vs)
        if case["path"] == "plain":
            state.update(key=state["key"].contiguous(), value=state["value"].contiguous())
    return state


def _prepare_decode(case, gen, rng):
    bs, hq, hk, D = case["block_size"], case["heads"], case["kv_heads"], case["head_dim"]
    lens = _lens(case)
    counts = [_blocks(int(x), bs) for x in lens]
    nb = sum(counts) + 8
    kc, ks = _pool8(nb, hk, bs, D, gen)
    vc, vs = _pool8(nb, hk, bs, D, gen)
    dt = DTYPES[case["dtype"]]
    query = torch.randn((case["seqs"], hq, D), dtype=dt, device="cuda", generator=gen)
    return dict(case=case, query=query, out=torch.zeros_like(query), k_cache=kc, k_scales=ks, v_cache=vc, v_scales=vs,
                block_tables=_table(counts, rng.permutation(nb)),
                context_lens=torch.as_tensor(lens.astype(np.int32)).cuda(), max_len=int(lens.max()), scale=1.0 / math.sqrt(D))


def _prepare_prefill(case, gen, rng):
    bs, hq, hk, D = case["block_size"], case["heads"], case["kv_heads"], case["head_dim"]
    counts = [_blocks(int(x), bs) for x in _lens(case)]
    nb = sum(counts) + 8
    kc, ks = _pool8(nb, hk, bs, D, gen)
    vc, vs = _pool8(nb, hk, bs, D, gen)
    chunks, prefixes = _ints(case["chunks"]), _ints(case["prefixes"])
    query = torch.randn((sum(chunks), hq, D), dtype=DTYPES[case["dtype"]], device="cuda", generator=gen)
    seq = np.repeat(np.arange(len(chunks)), chunks)
    row = np.concatenate([np.arange(c) for c in chunks])
    return dict(case=case, query=query, out=torch.zeros_like(query), k_cache=kc, k_scales=ks, v_cache=vc, v_scales=vs,
                block_tables=_table(counts, rng.permutation(nb)), chunk_lens=chunks, prefix_lens=prefixes,
                row_seq=torch.as_tensor(seq).cuda(), row_in_chunk=torch.as_tensor(row).cuda(), scale=1.0 / math.sqrt(D))


def _prepare_copy(case, gen, rng):
    n, bs, hk, D = case["pairs"], case["block_size"], case["kv_heads"], case["head_dim"]
    sources = max(1, n // 7)
    nb = sources + n + 3
    kc, ks = _pool8(nb, hk, bs, D, gen)
    vc, vs = _pool8(nb, hk, bs, D, gen)
    perm = rng.permutation(nb)
    pairs = np.stack([perm[np.arange(n) % sources], perm[sources:sources + n]], axis=1).astype(np.int64)
    return dict(case=case, k_cache=kc, k_scales=ks, v_cache=vc, v_scales=vs, pairs=torch.as_tensor(pairs).cuda())


# ---------------------------------------------------------------- one pass

def run(state):
    return {"norm": _run_norm, "write8": _run_write, "decode8": _run_decode, "prefill8": _run_prefill,
            "copy8": _run_copy}[state["case"]["op"]](state)


def _turn(x, s):
    """Rotated by the positions' angles, 32 bits."""
    axis = torch.as_tensor(s["pair_axis"], dtype=torch.long, device="cuda")
    angle = s["positions"].double()[axis].t() * s["inv_freq"].double()  # [T][pairs]; far positions need 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    half = cos.shape[-1]
    if s["case"]["style"] == "pairs":
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((r, x[..., 2 * half:]), dim=-1)


def _normed(x, w):
    y = x.float()
    return y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()


def _run_norm(s):
    if own:
        import paged_kv_cache_224_gb300 as pa
        pa.pa_norm_rotary_and_cache(s["query_out"], s["query"], s["key"], s["value"], s["k_cache"], s["v_cache"],
                                    s["positions"], s["slot_mapping"], s["inv_freq"], s["query_norm"], s["key_norm"], EPS,
                                    s["pair_axis"], interleaved=s["case"]["style"] == "pairs")
        return s["query_out"], s["k_cache"], s["v_cache"]
    dt, bs = s["query"].dtype, s["k_cache"].shape[2]
    s["query_out"].copy_(_turn(_normed(s["query"], s["query_norm"]), s))
    used = s["slot_mapping"] >= 0
    slot = s["slot_mapping"][used]
    s["k_cache"][slot // bs, :, slot % bs] = _turn(_normed(s["key"], s["key_norm"]), s).to(dt)[used]
    s["v_cache"][slot // bs, :, slot % bs] = s["value"][used]
    return s["query_out"], s["k_cache"], s["v_cache"]


def _store8(cache, scales, x, slots, f16):
    """Rows x [T][kv heads][D] (32 bits) into their slots of an 8-bit cache."""
    nb, hk, bs, _ = cache.shape
    used = slots >= 0
    block, row = torch.where(used, slots // bs, 0), slots % bs
    if f16:
        x = x.clamp(-F16_TOP, F16_TOP)
    m, e = torch.frexp(x.abs().amax(-1))
    need = torch.where(m > 0.875, e - 8, e - 9)                       # 2^need is the least one with |x| <= 448 2^need
    need = torch.where(used[:, None] & (m > 0), need, LOWEST).clamp(min=LOWEST).long()
    at = block[:, None].expand(-1, hk)
    low = torch.full((nb, hk), LOWEST, dtype=torch.long, device="cuda")
    zero = torch.zeros(nb, dtype=torch.long, device="cuda")
    need = low.scatter_reduce(0, at, need, "amax")
    touched = zero.scatter_reduce(0, block, used.long(), "amax") > 0
    fresh = (zero.scatter_reduce(0, block, (used & (row == 0)).long(), "amax") > 0)[:, None]
    old = scales.view(torch.uint8).long() - 127
    new = torch.where(touched[:, None], torch.where(fresh, need, torch.maximum(old, need)), old)
    shift = torch.where(fresh, 0, old - new).clamp(min=-32)
    codes = (cache.float() * _pow2(shift)[:, :, None, None]).to(cache.dtype).view(torch.uint8)
    rows = (x * _pow2(-new[block])[..., None]).to(cache.dtype).view(torch.uint8)
    codes[block[used], :, row[used]] = rows[used]
    cache.copy_(codes.view(cache.dtype))
    scales.view(torch.uint8).copy_((new + 127).to(torch.uint8))


def _run_write(s):
    c = s["case"]
    if own:
        import paged_kv_cache_224_gb300 as pa
        if c["path"] == "plain":
            pa.pa_reshape_and_cache_fp8(s["key"], s["value"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                        s["slot_mapping"])
        else:
            norms = (s["query_norm"], s["key_norm"], EPS) if c["path"] == "norm" else ()
            pa.pa_rotary_and_cache_fp8(s["query_out"], s["query"], s["key"], s["value"], s["k_cache"], s["v_cache"],
                                       s["k_scales"], s["v_scales"], s["positions"], s["slot_mapping"], s["inv_freq"],
                                       *norms, pair_axis=s["pair_axis"], interleaved=c["style"] == "pairs")
        return s["query_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]
    f16 = c["dtype"] == "f16"
    q, k = s["query"].float(), s["key"].float()
    if c["path"] == "norm":
        q, k = _normed(q, s["query_norm"]), _normed(k, s["key_norm"])
    if c["path"] != "plain":
        s["query_out"].copy_(_turn(q, s))
        k = _turn(k, s)
    _store8(s["k_cache"], s["k_scales"], k, s["slot_mapping"], f16)
    _store8(s["v_cache"], s["v_scales"], s["value"].float(), s["slot_mapping"], f16)
    return s["query_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]


def _values(cache, scales, tables):
    """Every table row's cached values: [rows][kv heads][blocks * block size][D], 32 bits."""
    t = tables.long().clamp(min=0)
    scale = _pow2(scales.view(torch.uint8)[t].int() - 127)
    x = cache.view(torch.uint8)[t].view(cache.dtype).float().mul_(scale[..., None, None])
    return x.transpose(1, 2).flatten(2, 3)


def _softmax_(x):
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    return x.div_(x.sum(-1, keepdim=True))


def _run_decode(s):
    hk, D = s["k_cache"].shape[1], s["k_cache"].shape[3]
    if own:
        import paged_kv_cache_224_gb300 as pa
        if "workspace" not in s:
            s["workspace"] = pa.decode_fp8_workspace(s["query"], hk, s["k_cache"].shape[2], s["max_len"])
        pa.pa_decode_fp8(s["out"], s["query"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["block_tables"],
                         s["context_lens"], s["scale"], s["max_len"], workspace=s["workspace"])
        return s["out"]
    q = s["query"].float().unflatten(1, (hk, -1))
    K = _values(s["k_cache"], s["k_scales"], s["block_tables"])
    x = torch.matmul(q, K.transpose(2, 3)).mul_(s["scale"])
    del K
    beyond = torch.arange(x.shape[-1], device="cuda") >= s["context_lens"][:, None]
    p = _softmax_(x.masked_fill_(beyond[:, None, None], -math.inf))
    s["out"].copy_(torch.matmul(p, _values(s["v_cache"], s["v_scales"], s["block_tables"])).flatten(1, 2))
    return s["out"]


def _run_prefill(s):
    hk = s["k_cache"].shape[1]
    if own:
        import paged_kv_cache_224_gb300 as pa
        if "workspace" not in s:
            s["workspace"] = pa.prefill_fp8_workspace(s["query"], s["k_cache"], s["prefix_lens"], s["chunk_lens"])
        pa.pa_prefill_batch_fp8(s["out"], s["query"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                s["block_tables"], s["prefix_lens"], s["chunk_lens"], s["scale"], workspace=s["workspace"])
        return s["out"]
    n, longest = len(s["chunk_lens"]), max(s["chunk_lens"])
    # chunks side by side, padded to the longest
    q = torch.zeros((n, longest) + s["query"].shape[1:], device="cuda")
    q[s["row_seq"], s["row_in_chunk"]] = s["query"].float()
    q = q.unflatten(2, (hk, -1)).permute(0, 2, 3, 1, 4)               # [n][kv heads][group][chunk][D]
    K = _values(s["k_cache"], s["k_scales"], s["block_tables"])[:, :, None]
    x = torch.matmul(q, K.transpose(-1, -2)).mul_(s["scale"])
    at = torch.tensor(s["prefix_lens"], device="cuda")[:, None] + torch.arange(longest, device="cuda")
    later = torch.arange(x.shape[-1], device="cuda") > at[..., None]  # [n][chunk][keys]
    p = _softmax_(x.masked_fill_(later[:, None, None], -math.inf))
    o = torch.matmul(p, _values(s["v_cache"], s["v_scales"], s["block_tables"])[:, :, None])
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["row_seq"], s["row_in_chunk"]])
    return s["out"]


def _run_copy(s):
    if own:
        import paged_kv_cache_224_gb300 as pa
        if "workspace" not in s:
            s["workspace"] = torch.empty(pa.pa_copy_blocks_workspace_bytes(s["case"]["pairs"]), dtype=torch.uint8, device="cuda")
        pa.pa_copy_blocks_fp8(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["pairs"], workspace=s["workspace"])
        return s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]
    src, dst = s["pairs"][:, 0], s["pairs"][:, 1]
    kc, vc, ks, vs = (s[x].view(torch.uint8) for x in ("k_cache", "v_cache", "k_scales", "v_scales"))
    kc[dst], vc[dst], ks[dst], vs[dst] = kc[src], vc[src], ks[src], vs[src]
    return s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "write8": _exact_write, "decode8": _exact_decode, "prefill8": _exact_prefill,
            "copy8": _exact_copy}[case["op"]](s)


def _scale64(scales):
    return _pow2(scales.view(torch.uint8).long() - 127, wide=True)


def _spun(x, s, weight):
    """Each head over its root mean square, times its weights (None: as it is), each pair then times e^(i angle)."""
    x = x.double()
    if weight is not None:
        x = x * ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS) ** -0.5 * weight.double()
    pos = s["positions"].cpu().numpy().astype(np.float64)
    angle = pos[s["pair_axis"]].T * s["inv_freq"].cpu().numpy().astype(np.float64)
    unit = torch.as_tensor(np.exp(1j * angle)).cuda()[:, None]
    R = 2 * len(s["pair_axis"])
    re, im = (slice(0, R, 2), slice(1, R, 2)) if s["case"]["style"] == "pairs" else (slice(0, R // 2), slice(R // 2, R))
    z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * unit
    x = x.clone()
    x[..., re], x[..., im] = z.real, z.imag
    return x


def _exact_norm(s):
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    rk = _spun(s["key"], s, s["key_norm"])
    slots = s["slot_mapping"].cpu()
    bs = kc.shape[2]
    t = torch.nonzero(slots >= 0)[:, 0]
    b, r = (slots[t] // bs).cuda(), (slots[t] % bs).cuda()
    kc[b, :, r] = rk[t.cuda()]
    vc[b, :, r] = s["value"].double()[t.cuda()]
    return _spun(s["query"], s, s["query_norm"]), kc, vc


def _e4m3(y):
    """The nearest values of e4m3 (three bits behind the leading one, from 2^-9 on), ties to even; y within its range."""
    _, e = torch.frexp(y)
    step = _pow2(e.clamp(min=-5) - 4, wide=True)
    return torch.round(y / step) * step


def _exact_store(cache, scales, x, slots, f16):
    """Block by block as values: the written rows' largest magnitude decides the scale, then every row is on its grid."""
    nb, hk, bs, D = cache.shape
    if f16:
        x = torch.where(x.abs() > F16_TOP, x.sign() * F16_TOP, x)
    old = _scale64(scales)
    value = cache.double() * old[..., None, None]
    put = [(t, int(z) // bs, int(z) % bs) for t, z in enumerate(slots.tolist()) if z >= 0]
    t, b, r = torch.tensor(put, dtype=torch.long, device="cuda").reshape(-1, 3).unbind(1)
    written = torch.zeros((nb, bs), dtype=torch.bool, device="cuda")
    written[b, r] = True
    value[b, :, r] = x[t]
    most = torch.where(written[:, None, :, None], value.abs(), torch.zeros_like(value)).amax((2, 3))
    # the least power of two that brings it to 448 or below; -inf for a block of zeros
    size = torch.log2(most / 448).ceil().clamp(min=LOWEST)
    size = torch.where(448 * _pow2(size - 1, wide=True) >= most, size - 1, size).clamp(min=LOWEST)
    size = _pow2(torch.where(448 * _pow2(size, wide=True) < most, size + 1, size), wide=True)
    fresh, touched = written[:, 0, None], written.any(1)[:, None]
    new = torch.where(touched, torch.where(fresh, size, torch.maximum(old, size)), old)
    kept = fresh[..., None, None] & ~written[:, None, :, None]        # rows of a fresh block that nobody wrote stay as codes
    return torch.where(kept, cache.double(), _e4m3(value / new[..., None, None])), new


def _exact_write(s):
    c = s["case"]
    f16 = c["dtype"] == "f16"
    q, k = s["query_out"].double(), s["key"].double()
    if c["path"] != "plain":
        normed = c["path"] == "norm"
        q = _spun(s["query"], s, s["query_norm"] if normed else None)
        k = _spun(s["key"], s, s["key_norm"] if normed else None)
    kc, ks = _exact_store(s["k_cache"], s["k_scales"], k, s["slot_mapping"], f16)
    vc, vs = _exact_store(s["v_cache"], s["v_scales"], s["value"].double(), s["slot_mapping"], f16)
    return q, kc, vc, ks, vs


def _gathered(s, which, i, n):
    """Values of rows 0 .. n-1 of sequence i in 64 bits, token by token through its table: [n][kv heads][D]."""
    cache, scales = s[which + "_cache"], s[which + "_scales"]
    j = torch.arange(n, device="cuda")
    b, r = s["block_tables"][i].long()[j // cache.shape[2]], j % cache.shape[2]
    return cache.view(torch.uint8)[b, :, r].view(cache.dtype).double() * _scale64(scales)[b][..., None]


def _exact_decode(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["context_lens"].tolist()):
        K, V = _gathered(s, "k", i, n), _gathered(s, "v", i, n)
        per = out.shape[1] // K.shape[1]
        for h in range(K.shape[1]):
            z = (s["query"][i, h * per:(h + 1) * per].double() @ K[:, h].t()) * s["scale"]
            w = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
            out[i, h * per:(h + 1) * per] = w @ V[:, h]
    return out


def _exact_prefill(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, (p, c) in enumerate(zip(s["prefix_lens"], s["chunk_lens"])):
        K, V = _gathered(s, "k", i, p + c), _gathered(s, "v", i, p + c)
        seen = torch.arange(p + c, device="cuda")[None] <= p + torch.arange(c, device="cuda")[:, None]
        per = out.shape[1] // K.shape[1]
        for h in range(out.shape[1]):
            z = (s["query"][at:at + c, h].double() @ K[:, h // per].t()) * s["scale"]
            z = torch.where(seen, z, torch.full_like(z, -math.inf))
            out[at:at + c, h] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) @ V[:, h // per]
        at += c
    return out


def _exact_copy(s):
    new = [s["k_cache"].double(), s["v_cache"].double(), _scale64(s["k_scales"]), _scale64(s["v_scales"])]
    for x in new:
        was = x.clone()
        for a, b in s["pairs"].tolist():
            x[b] = was[a]
    return tuple(new)


# ---------------------------------------------------------------- the work of one pass

def work(case):
    op, D, hk, bs = case["op"], case["head_dim"], case["kv_heads"], case["block_size"]
    if op in ("norm", "write8"):
        T, hq = case["tokens"], case["heads"]
        wide = 1 if op == "write8" else 2                             # bytes of a cached value
        # queries read and written, keys and values read, cached rows written, positions, slots, frequencies, norms
        if case.get("path") == "plain":
            return dict(bytes=T * 2 * hk * D * (2 + wide) + 8 * T, flops=2 * T * 2 * hk * D)
        return dict(bytes=T * (4 * hq + 2 * hk * (2 + wide)) * D + T * (4 * case["axes"] + 8) + 2 * case["rot_dim"] + 4 * D,
                    flops=T * (hq + hk) * (3 * case["rot_dim"] + 4 * D))
    if op == "copy8":
        # codes and scales of K and V, read and written, and the pairs
        return dict(bytes=case["pairs"] * (4 * hk * (bs * D + 1) + 16), flops=0)
    lens = _lens(case)
    hq = case["heads"]
    blocks = int(sum(_blocks(int(x), bs) for x in lens))
    # codes of K and V once, scales, table entries
    cached = int(lens.sum()) * hk * D * 2 + blocks * (2 * hk + 4)
    if op == "decode8":
        # and queries, outputs, lengths
        return dict(bytes=cached + 4 * len(lens) * hq * D + 4 * len(lens), flops=int(4 * D * hq * lens.sum()))
    chunks = np.array(_ints(case["chunks"]), np.int64)
    seen = int((chunks * (lens - chunks) + chunks * (chunks + 1) // 2).sum())
    return dict(bytes=cached + 4 * int(chunks.sum()) * hq * D, flops=4 * D * hq * seen)
