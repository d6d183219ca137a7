"""Plain 64-bit forms of the quantised cache's operators, for their tests (CPU)."""
from __future__ import annotations

import math

import torch

E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def e4m3_values():
    """The 256 values of an e4m3 byte, float64."""
    out = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        if b & 127 == 127:
            v = math.nan
        out.append(-v if b >= 128 else v)
    return torch.tensor(out, dtype=torch.float64)


def nearest(x, values):
    """The nearest of `values` (ascending, of even and odd codes in turn, 0 first) to x >= 0:
    ties to the even one, past the last the last; NaN stays."""
    hi = torch.searchsorted(values, x.clamp(max=float(values[-1])).nan_to_num(0.0))
    hi = hi.clamp(max=len(values) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = values[hi] - x, x - values[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.where(x.isnan(), x, torch.where(x >= values[-1], values[-1], values[pick]))


def kept(x, fmt):
    """What the rows x [..., D] come back as, float64."""
    x = x.detach().cpu().double()
    pos = e4m3_values()[:127]
    top = 448.0 if fmt == "fp8" else 6 * 448.0
    amax = x.abs().nan_to_num(0.0, posinf=1e300).amax(-1, keepdim=True)
    e = torch.full_like(amax, 90.0)
    for k in range(89, -91, -1):                       # the least that holds the row
        e = torch.where(amax <= top * 2.0 ** k, torch.full_like(e, float(k)), e)
    unit = 2.0 ** e
    y = x / unit
    if fmt == "fp8":
        return nearest(y.abs(), pos) * y.sign() * unit
    y = y.unflatten(-1, (-1, 16))
    nan = y.isnan().any(-1, keepdim=True)
    a = y.abs().nan_to_num(0.0, posinf=1e300).clamp(max=top).amax(-1, keepdim=True)
    s = nearest((a.float() * torch.tensor(1 / 6)).double(), pos)   # an fp32 product
    z = torch.where(s > 0, y.abs() / s, torch.zeros_like(y))
    out = nearest(z.nan_to_num(0.0, posinf=1e300), torch.tensor(E2M1, dtype=torch.float64)) * s
    out = torch.where(nan, torch.full_like(out, math.nan), out * y.sign().nan_to_num(0.0))
    return out.flatten(-2) * unit


def held(codes, scales, fmt, is_v):
    """The values a cache's bytes stand for, [num_blocks, Hkv, B, D] float64, read from the
    documented layout."""
    codes, scales = codes.cpu(), scales.cpu()
    nb, hkv, B, row = codes.shape
    D = row if fmt == "fp8" else 2 * row
    val = torch.empty(nb, hkv, B, D, dtype=torch.float64)
    side = scales.view(nb, hkv, B // 16, -1)
    table = e4m3_values()
    two = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64)
    for t in range(B):
        c, u = divmod(t, 16)
        exp = side[:, :, c, -16 + u].double() - 127
        if fmt == "fp8":
            v = table[codes[:, :, t].long()]
        else:
            b = codes[:, :, t].long()
            v = torch.stack((two[b & 15], two[b >> 4]), -1).flatten(-2)
            g = torch.arange(D // 16)
            at = (u // 4) * (D // 4) + 4 * g + u % 4 if is_v else u * (D // 16) + g
            v = v * table[side[:, :, c][:, :, at].long()].repeat_interleave(16, -1)
        val[:, :, t] = v * (2.0 ** exp)[..., None]
    return val


def rows_of(val, slots):
    """Rows of the slots, [T, Hkv, D]."""
    B = val.shape[2]
    slots = slots.cpu()
    return val[slots // B, :, slots % B]


def decode_bound(q, k, v, p, ref, scale, dtype):
    """How far a decoded output [Hq, D] may be from the 64-bit one, attending the rows k, v [n,
    Hkv, D] with weights p [Hkv, G, n].

    A score is a sum of D products, fp32 with cut or rounded partial sums: off by D 2^-23 of the
    sum of their sizes (`size`), and 2^-21 of it for q held in one (bf16: exact) or two (fp32)
    fp16 parts, 4 roundings for the row's and the head's scale and the softmax scale.  exp2's
    argument is rounded (2^-24 of at most 2 size + 181, the exponents) and its value off by
    2^-22.  A weight carries its own and the denominator's error; weights held in fp16 are off by
    2^-11 (bf16 output) or in two parts by 2^-21 (fp32), those below 2^-21 of the largest
    contribution by 2^-31 of it, which n rows of at most the largest size add up.  The sums
    over n tokens round n times, the merges 32 times more.  The output rounds once."""
    hkv, G, n = p.shape
    qg = q.double().view(hkv, G, -1)
    size = float((qg.abs()[:, :, None] * k.abs().transpose(0, 1)[:, None]).sum(-1).max()) * scale
    d = q.shape[-1]
    score = (d + 8) * 2.0 ** -23 * size + 2.0 ** -21 * size
    rel = 2 * (score + (2 * size + 181) * 2.0 ** -24 + 2.0 ** -22) + (n + 64) * 2.0 ** -23
    rel += 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21
    sizes = torch.einsum("hgn,nhd->hgd", p, v.abs())
    small = (p * v.abs().amax(-1).transpose(0, 1)[:, None]).amax(-1, keepdim=True) * n * 2.0 ** -30
    return (ref.abs() * torch.finfo(dtype).eps / 2 * 1.01
            + (sizes * rel * 1.2 + small).reshape(ref.shape) + 1e-37)
