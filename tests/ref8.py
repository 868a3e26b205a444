"""Plain 64-bit definitions of the 8-bit cache and of head norms, on the CPU."""
from __future__ import annotations

import numpy as np
import torch

from tests.ref64 import rotate

LOWEST = -64
F16_TOP = 61440.0


def pow2(e):
    """2^e for whole e from -1022 to 1023, exact."""
    return ((torch.as_tensor(e).long() + 1023) << 52).view(torch.float64)


def scale_values(scales):
    """The powers of two that scale bytes stand for, float64."""
    b = scales.cpu().view(torch.uint8).long()
    return torch.where(b == 255, torch.full(b.shape, float("nan"), dtype=torch.float64), pow2(b - 127))


def values(cache, scales):
    """[NB][Hkv][bs][D] float64."""
    return cache.cpu().double() * scale_values(scales)[..., None, None]


def to_grid(y):
    """Nearest e4m3 values, ties to even, of float64 y with |y| <= 448 or NaN."""
    a = torch.where(y == 0, torch.ones_like(y), y.abs())
    _, e = torch.frexp(a)
    step = pow2(e.clamp(min=-5) - 4)
    return torch.round(y / step) * step


def need_exponent(rows):
    """The least e >= LOWEST with |x| <= 448 * 2^e for every finite x."""
    a = rows[torch.isfinite(rows)].abs()
    top = float(a.max()) if a.numel() else 0.0
    e = LOWEST
    while top > 448.0 * 2.0 ** e:
        e += 1
    return e


def store(cache, scales, x, slots, f16):
    """Codes' values (float64) and scale exponents (long) after rows x [T][Hkv][D] (float64) are written."""
    codes = cache.cpu().double().clone()
    e = scales.cpu().view(torch.uint8).long() - 127
    bs = cache.shape[2]
    rows = {}
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < cache.shape[0] * bs:
            rows.setdefault(s // bs, {})[s % bs] = t  # the later token wins
    x = torch.where(torch.isfinite(x), x, torch.full_like(x, float("nan")))
    if f16:
        x = x.clamp(-F16_TOP, F16_TOP)
    for b, at in rows.items():
        for h in range(cache.shape[1]):
            new = need_exponent(torch.stack([x[t, h] for t in at.values()]))
            if 0 not in at and int(e[b, h]) >= new:
                new = int(e[b, h])
            if 0 not in at and new != int(e[b, h]):
                moved = to_grid(codes[b, h] * 2.0 ** (int(e[b, h]) - new))
                codes[b, h] = moved
            for r, t in at.items():
                codes[b, h, r] = to_grid(x[t, h] / 2.0 ** new)
            e[b, h] = new
    return codes, e


def normed(x, w, eps):
    x = x.cpu().double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.cpu().double()


def turned(x, pos, inv, ax, interleaved):
    """x [T][H][D] float64 rotated by its positions; pos [axes][T] or [T]."""
    pos, inv = pos.cpu().numpy().astype(np.float64), inv.cpu().numpy().astype(np.float64)
    ax = np.zeros(len(inv), int) if ax is None else np.asarray(ax)
    angle = pos.reshape(-1, pos.shape[-1])[ax].T * inv if len(inv) else np.zeros((x.shape[0], 0))
    return rotate(x, torch.as_tensor(angle), interleaved)


def quantise(x):
    """A cache (codes, scale bytes) of float x [NB][Hkv][bs][D], each block and head at the least scale."""
    a = x.double().abs().amax((2, 3))
    m, e = torch.frexp(a / 448)
    e = torch.where(m == 0.5, e - 1, e).clamp(min=LOWEST)
    codes = to_grid(x.double() / pow2(e)[..., None, None]).float().to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def make_pool(lens, Hkv, D, bs, device, seed, spare=4, spread=1.0, poison=False):
    """An 8-bit pool and table rows (int32, -1 past the end) for ``lens``; each block's rows N(0, 1) times a
    power of two within 2^(+-spread).  ``poison``: NaN codes in every row that no context covers, NaN scales in
    blocks that none does."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-int(n) // bs) for n in lens]
    nb = sum(counts) + spare
    perm = torch.randperm(nb, generator=g)
    table = torch.full((len(lens), max(1, max(counts, default=1))), -1, dtype=torch.int32)
    out = []
    at = 0
    used = torch.zeros((nb, bs), dtype=torch.bool)
    for i, n in enumerate(counts):
        table[i, :n] = perm[at:at + n].int()
        at += n
        j = torch.arange(int(lens[i]))
        used[table[i].long()[j // bs], j % bs] = True
    for _ in range(2):
        x = torch.randn((nb, Hkv, bs, D), generator=g)
        x *= torch.exp2(spread * (2 * torch.rand((nb, Hkv, 1, 1), generator=g) - 1))
        codes, scales = quantise(x)
        if poison:
            codes.view(torch.uint8)[~used[:, None].expand(-1, Hkv, -1)] = 0x7f
            scales[~used.any(1)] = 255
        out += [codes.to(device), scales.view(torch.float8_e8m0fnu).to(device)]
    kc, ks, vc, vs = out
    return kc, ks, vc, vs, table.to(device)


def rows_of(vals, table_row, n):
    """Rows 0 .. n-1 of a sequence out of ``values``: [n][Hkv][D]."""
    bs = vals.shape[2]
    t = table_row.cpu().long()
    j = torch.arange(n)
    return vals[t[j // bs], :, j % bs] if n else torch.zeros((0, vals.shape[1], vals.shape[3]), dtype=torch.float64)


def attend_sizes(q, K, V, scale):
    """out [Hq][D], the weighted mean of |v| [Hq][D], and the largest sum |q_i k_i| * scale of each head [Hq]."""
    Hq, G = q.shape[0], q.shape[0] // K.shape[1]
    out, mean, size = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(Hq, dtype=torch.float64)
    if K.shape[0] == 0:
        return out, mean, size
    for h in range(Hq):
        k, v = K[:, h // G], V[:, h // G]
        s = (k @ q[h]) * scale
        p = torch.softmax(s, 0)
        out[h], mean[h] = p @ v, p @ v.abs()
        size[h] = float((k.abs() @ q[h].abs()).max()) * abs(scale)
    return out, mean, size
