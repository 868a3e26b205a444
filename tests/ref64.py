"""Plain 64-bit definitions of the bounded- and shared-cache operators, and a
small paged-pool builder.  Written token by token from the formulas."""
from __future__ import annotations

import numpy as np
import torch

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype: str) -> float:
    """Largest relative error of one rounding to ``dtype``."""
    return torch.finfo(DTYPES[dtype]).eps / 2


def make_pool(lens, Hkv, D, bs, dtype, device, seed, spare=4, extra=()):
    """A pool of N(0,1) values, with table rows (int32, -1 past the end) dealt
    out of a permutation for ``lens`` and then for the lengths ``extra``."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-int(n) // bs) for n in list(lens) + list(extra)]
    nb = sum(counts) + spare
    perm = torch.randperm(nb, generator=g).numpy()
    width = max(1, max(counts[:len(lens)], default=1))
    rows, at = [], 0
    for n in counts:
        rows.append(perm[at:at + n].astype(np.int32))
        at += n

    def table(rs):
        w = max(1, max((len(r) for r in rs), default=1))
        t = np.full((len(rs), w), -1, np.int32)
        for i, r in enumerate(rs):
            t[i, :len(r)] = r
        return torch.as_tensor(t, device=device)
    dt = DTYPES[dtype]
    kc = torch.randn((nb, Hkv, bs, D), generator=g).to(dt).to(device)
    vc = torch.randn((nb, Hkv, bs, D), generator=g).to(dt).to(device)
    return kc, vc, table(rows[:len(lens)]), table(rows[len(lens):]) if len(extra) else None


def gather(cache, table_row, n):
    """Rows 0 .. n-1 of a sequence, [n][Hkv][D], float64 on the CPU."""
    bs = cache.shape[2]
    c = cache.cpu()
    t = table_row.cpu().long()
    if n == 0:
        return torch.zeros((0, cache.shape[1], cache.shape[3]), dtype=torch.float64)
    j = torch.arange(n)
    return c[t[j // bs], :, j % bs].double()


def attend(q, K, V, scale):
    """q [Hq][D], K/V [n][Hkv][D] -> (out [Hq][D], weights [Hkv][n] summed over
    each kv head's query heads, largest sum_i |q_i k_i| * scale)."""
    Hq, n, Hkv = q.shape[0], K.shape[0], K.shape[1]
    G = Hq // Hkv
    if n == 0:
        return torch.zeros_like(q), torch.zeros((Hkv, 0), dtype=torch.float64), 0.0
    out = torch.zeros_like(q)
    w = torch.zeros((Hkv, n), dtype=torch.float64)
    size = 0.0
    for h in range(Hq):
        s = (K[:, h // G] @ q[h]) * scale
        size = max(size, float((K[:, h // G].abs() @ q[h].abs()).max()) * abs(scale))
        e = torch.exp(s - s.max())
        p = e / e.sum()
        out[h] = p @ V[:, h // G]
        w[h // G] += p
    return out, w, size


def rotate(x, angle, interleaved):
    """x [T][H][D] float64, angle [T][R/2] float64."""
    y = x.clone()
    half = angle.shape[1]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a_i = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b_i = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = x[..., a_i], x[..., b_i]
    y[..., a_i] = a * c - b * s
    y[..., b_i] = b * c + a * s
    return y


def evict_choice(w, n, keep, sink, recent):
    """Kept indices of one (sequence, kv head), w float32 [>= n] on the host."""
    if n <= keep:
        return list(range(n))
    must = [j for j in range(n) if j < sink or j >= n - recent]
    rest = [j for j in range(n) if sink <= j < n - recent]
    rest.sort(key=lambda j: (-(float("-inf") if np.isnan(w[j]) else float(w[j])), bool(np.isnan(w[j])), j))
    return sorted(must + rest[:keep - len(must)])
