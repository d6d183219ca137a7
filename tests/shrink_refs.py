"""Plain 64-bit forms of the operators around a shrinking cache, for their tests (CPU)."""
from __future__ import annotations

import math

import torch


def rotate(x, positions, inv_freq, *, interleaved=False, inverse=False, attn_scale=1.0):
    """x [T, H, D] (any type) turned by its positions; float64."""
    y = x.detach().cpu().double().clone()
    angle = positions.cpu().double()[:, None] * inv_freq.cpu().double()[None]
    if inverse:
        angle = -angle
    c, s = (torch.cos(angle) * attn_scale)[:, None], (torch.sin(angle) * attn_scale)[:, None]
    r = 2 * inv_freq.numel()
    lo, hi = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2),
                                                                   slice(r // 2, r))
    a, b = y[..., lo].clone(), y[..., hi].clone()
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    return y


def rotate_bound(x, positions, inv_freq, ref, dtype, *, interleaved=False, attn_scale=1.0):
    """How far a turned row may be from the 64-bit one: the final rounding, plus fp32 work.

    A cosine or sine is off by one unit of sincospif (2^-24), its argument's rounding
    (|x| <= 1/4 half turns: 2^-27 pi) and cut (2^-32 turns), and its product with attn_scale
    (2^-24): below 3 * 2^-24 in all; the two products and the sum round once each (3 * 2^-24).
    So fp32 work is off by less than 2^-21 attn_scale (|a| + |b|).  The frequency's fraction of
    a turn, from two roundings in 64 bits, is off by 2^-52 of itself, the reference's angle by
    2^-53 pos * f: together 2^-50 |pos| f radians."""
    y = x.detach().cpu().double().abs()
    r = 2 * inv_freq.numel()
    lo, hi = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2),
                                                                   slice(r // 2, r))
    pair = y[..., lo] + y[..., hi]
    angle = (positions.cpu().double().abs()[:, None] * inv_freq.cpu().double()[None])[:, None]
    work = attn_scale * pair * (2.0 ** -21 + 2.0 ** -50 * angle)
    bound = ref.abs() * (torch.finfo(dtype).eps / 2) * 1.01
    bound[..., lo] += work
    bound[..., hi] += work
    bound[..., r:] = 0
    return bound


def tokens(pool, table_row, n):
    """The first n tokens of a sequence, [n, Hkv, D] float64."""
    B = pool.shape[2]
    ids = table_row[:-(-n // B)].long()
    return pool[ids].transpose(1, 2).reshape(-1, pool.shape[1], pool.shape[3])[:n].double()


def attention(q, k, v, scale, first=0):
    """q [m, Hq, D] over k / v [n, Hkv, D], query i seeing keys 0 .. first + i: (output
    [m, Hq, D], probabilities summed over queries and group [Hkv, n], score-error scale)."""
    m, hq, d = q.shape
    n, hkv, _ = k.shape
    qg = q.double().view(m, hkv, hq // hkv, d)
    x = torch.einsum("mhgd,nhd->hgmn", qg, k) * scale
    future = torch.arange(n)[None] > (first + torch.arange(m))[:, None]
    x.masked_fill_(future[None, None], -math.inf)
    p = torch.softmax(x, -1)
    out = None if v is None else torch.einsum("hgmn,nhd->mhgd", p, v).reshape(m, hq, d)
    size = torch.einsum("mhgd,nhd->hgmn", qg.abs(), k.abs()).max() * scale if n and m else 0.0
    return out, p.sum((1, 2)), float(size)


def weight_bound(added, before, size, d, terms):
    """How far a summed weight may be from the 64-bit one.

    A score is a sum of d products in fp32, off by at most d 2^-23 (tensor cores may cut
    instead of rounding) of the sum of their absolute values, `size` at most; the same holds
    for its scaling.  exp2's argument is rounded (2^-24 of a score of at most 2 size) and its
    value off by 2^-22.  A probability carries its own and the denominator's error (the same
    again), and sums of `terms` positive terms add 2^-24 each.  decay and the last sum round
    once each."""
    score = (d + 4) * 2.0 ** -23 * size
    rel = 2 * (score + 2 * size * 2.0 ** -24 + 2.0 ** -22) + (terms + 16) * 2.0 ** -24
    return added * rel * 1.5 + (before.abs() + added) * 2.0 ** -23 + 1e-37


def evict_rows(weights, positions, tracked, seen, L, budget, sinks, recent):
    """One (sequence, kv head): (source index of each kept place, weights, positions), or None
    where nothing is evicted."""
    w = [float(x) for x in weights[:L]]
    pos = [int(positions[j]) if j < tracked else seen - L + j for j in range(L)]
    if budget < 0 or L <= budget:
        return None, w, pos
    safe = [p < sinks or p >= seen - recent for p in pos]

    def order(j):
        x = w[j]
        return (not safe[j], math.isnan(x), -x if not math.isnan(x) else 0.0, j)

    keep = set(sorted(range(L), key=order)[:budget])
    movers = [j for j in range(budget, L) if j in keep]
    source = []
    for j in range(budget):
        source.append(j if j in keep else movers.pop(0))
    assert not movers
    return source, [w[j] for j in source], [pos[j] for j in source]
