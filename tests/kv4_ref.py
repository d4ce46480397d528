"""Plain 64-bit forms of the 4-bit KV cache operators, written from the formulas
and the record layout that include/pod_kv4.h states."""
from __future__ import annotations

import math

import torch

PAGE = 16
EPS = {torch.bfloat16: 2.0 ** -7, torch.float16: 2.0 ** -10}


def places(d, group):
    """For K and V: index of the 4-bit code of (token, channel) and of its pair in a record."""
    code, pair = torch.zeros(2, PAGE, d, dtype=torch.long), torch.zeros(2, PAGE, d, dtype=torch.long)
    for t in range(PAGE):
        for ch in range(d):
            c, j, i = ch // 32, ch % 32 // 8, ch % 8
            code[0, t, ch] = 2 * (t * d // 2 + 4 * (j * (d // 32) + c)) + i
            f, j, e, r, i = t // 8, t % 8 // 2, t % 2, ch % 32 // 4, ch % 4
            code[1, t, ch] = 2 * (8 * d + 4 * ((32 * f + 4 * r + j) * (d // 32) + c) + 2 * e) + i
            for kv in range(2):
                pair[kv, t, ch] = (kv * PAGE + t) * (d // group) + ch // group
    return code, pair


def unpack(records, d, group):
    """(codes, s, m) [..., 2, PAGE, d] in fp64 of uint8 records [..., bytes] (on the CPU)."""
    code, pair = places(d, group)
    n = records[..., code // 2] >> (4 * (code % 2)).to(torch.uint8) & 15
    par = records[..., PAGE * d:].contiguous().view(torch.float16).double().unflatten(-1, (-1, 2))
    return n.double(), par[..., pair, 0], par[..., pair, 1]


def values(records, d, group):
    n, s, m = unpack(records, d, group)
    return n * s + m


def quantised(x, group):
    """(codes, s, m, distance of the quotient to the nearest border) of x [..., d]."""
    x = x.double().unflatten(-1, (-1, group))
    fine = x.isfinite().all(-1, keepdim=True)
    x = x.clamp(-65504, 65504)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi.float() - lo.float()) / torch.tensor(15.0)).half().double()
    m = lo.half().double()
    nan = torch.full_like(s, math.nan)
    t = torch.where(s > 0, (x - m) / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))
    n = t.round().clamp(0, 15)
    border = (t - t.floor() - 0.5).abs()
    s, m = torch.where(fine, s, nan), torch.where(fine, m, nan)
    n = torch.where(fine, n, torch.zeros_like(n))
    wide = lambda y: y.expand_as(n).flatten(-2)  # noqa: E731
    return n.flatten(-2), wide(s), wide(m), border.flatten(-2)


def attend(q, records, table, lens, d, group, *, keys=None):
    """O, LSE in fp64 of q [R, H, d] over the pool `records` [blocks, Hk, bytes], and the
    parts of an error bound: E[s |n - 8|], E[16 s], E|v - o|, and the largest sum |q_i k_i| / sqrt(d)."""
    R, H, _ = q.shape
    Hk = records.shape[1]
    o, spread, wide, dev = (torch.zeros(R, H, d, dtype=torch.float64) for _ in range(4))
    lse, big = torch.full((R, H), -math.inf, dtype=torch.float64), torch.zeros(R, H, dtype=torch.float64)
    for r, n in enumerate(lens):
        if n == 0:
            continue
        code, s, m = unpack(records[table[r, :-(-n // PAGE)].long()], d, group)
        val = (code * s + m).permute(2, 1, 0, 3, 4).flatten(2, 3)[:, :, :n]   # 2, Hk, n, d
        near = ((code - 8).abs() * s).permute(2, 1, 0, 3, 4).flatten(2, 3)[1, :, :n]
        step = (16 * s).permute(2, 1, 0, 3, 4).flatten(2, 3)[1, :, :n]
        for h in range(H):
            g = h // (H // Hk)
            k, v = val[0, g], val[1, g]
            x = q[r, h].double()
            sc = k @ x / math.sqrt(d)
            big[r, h] = (k.abs() @ x.abs()).max() / math.sqrt(d)
            lse[r, h] = torch.logsumexp(sc, 0)
            p = torch.softmax(sc, 0)
            o[r, h] = p @ v
            spread[r, h], wide[r, h] = p @ near[g], p @ step[g]
            dev[r, h] = p @ (v - o[r, h]).abs()
    return o, lse, (spread, wide, dev, big)


def attend_bounds(o, lse, parts, dtype):
    """How far the kernel's O and LSE may be from the exact ones.

    Each weight p s is rounded once to fp16 (half a step: 2^-11 of it), which moves O by at most
    2^-11 E[s |n - 8|]. A score carries the fp32 roundings of d products and sums (below 2^-17 of
    sum |q_i k_i| for d <= 128, 128 roundings of 2^-24 each) and moves O by twice that times
    E|v - o|, LSE by once. The fp32 products and sums over the keys are of bytes, two codes each:
    of up to 256 s, in parts of 64 keys. A part's five additions, each off by 2^-23 of that, add
    5 2^-23 16 < 2^-16 of E[16 s], the joining of the parts as much again of E[16 s] + |o|.
    The output is rounded once."""
    spread, wide, dev, big = parts
    score = big.unsqueeze(-1) * 2.0 ** -17
    bound = 2.0 ** -11 * spread + 2 * score * dev + 2.0 ** -15 * (wide + o.abs())
    bound = bound + EPS[dtype] / 2 * (o.abs() + bound) + 2.0 ** -24
    return bound, big * 2.0 ** -17 + 2.0 ** -20 * (1 + lse.abs().nan_to_num(0, 0, 0))


def norm_rope(x, w, table, pos, eps, interleaved):
    """y in fp64 and |a| + |b|, the size of the pair that each channel came from."""
    y = x.double()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    rot = table.shape[1]
    half = rot // 2
    cs = table[pos.long()].double()
    c, s = cs[:, None, :half], cs[:, None, half:]
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(half)
    ib = ia + (1 if interleaved else half)
    a, b = y[..., ia], y[..., ib]
    out, size = y.clone(), y.abs()
    out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, size
