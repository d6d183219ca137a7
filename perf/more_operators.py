"""The cases at which the operators of a quantised paged cache are measured.

Rows are quantised to 8 or 4 bits as they are written to their slots and read back by slot;
whole blocks move between a pool and the quantised cache, both ways; and one new token of
every sequence attends to the quantised cache, its own row appended in the same call.  A case
names its operator ("op") and its sizes; `prepare` makes the inputs on the GPU, `run` makes
one pass (in plain torch operations, or with `own` through the library), `work` counts what a
pass cannot do without and `exact` gives its outputs in 64 bits.

The quantised row.  A row x of D elements (one token, one kv head, K or V) has an exponent e,
from -90 to 90, the least for which no element is beyond the format's largest value times 2^e.
fp8: x_i = code_i 2^e, code_i the e4m3 value nearest to x_i 2^-e (largest: 448).
fp4: x_i = code_i s 2^e, s an e4m3 scale for each 16 elements, the nearest to a sixth of their
largest magnitude times 2^-e, and code_i the e2m1 value nearest to x_i 2^-e / s (largest value:
6 * 448).  Ties go to the even code; what is beyond the largest value takes it.

Where it lies.  The codes are uint8 [blocks, kv heads, block size, D] (fp8: e4m3 bytes) or
[..., D / 2] (fp4: pairs of e2m1, element 2 i in the low half of byte i).  Beside them lie, for
each block and kv head and 16 tokens of the block after another, the scales s of fp4, of K as
[16 tokens][D / 16], of V as [4][D / 16][4 tokens], and the 16 exponents, e + 127.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One step's new tokens of 64 sequences, written and read back: latency.
        dict(name="append step of 64 fp8", op="append", format="fp8", tokens=64, hkv=8, d=128,
             block=16, dtype="bf16", fused=True),
        # The new tokens of 16 prompts of 512, as slices of one fused projection.
        dict(name="append prompts 8192 fp8", op="append", format="fp8", tokens=8192, hkv=8,
             d=128, block=16, dtype="bf16", fused=True),
        # An odd number of fp32 rows of a short head, 4 bits.
        dict(name="append f32 4097 fp4", op="append", format="fp4", tokens=4097, hkv=16, d=64,
             block=32, dtype="f32", fused=False),
        # Finished prompts leave the pool for the compact cache and come back later.
        dict(name="freeze 2048 blocks fp4", op="freeze", format="fp4", blocks=2048, hkv=8,
             d=128, block=16, dtype="bf16"),
        # A few blocks of an fp32 pool.
        dict(name="freeze 37 blocks f32 fp8", op="freeze", format="fp8", blocks=37, hkv=4, d=64,
             block=32, dtype="f32"),
        # The cached prefixes of 16 prompts, 1024 to 8192 tokens, read into a pool for the
        # prefill of the tokens after them.
        dict(name="thaw 4608 blocks fp8", op="thaw", format="fp8", blocks=4608, hkv=8, d=128,
             block=16, dtype="bf16"),
        # One short prefix.
        dict(name="thaw 33 blocks fp4", op="thaw", format="fp4", blocks=33, hkv=8, d=128,
             block=16, dtype="bf16"),
        # Decode of 4 short sequences of an fp32 model: latency.
        dict(name="decode tiny f32 fp8", op="decode", format="fp8", seqs=4, hq=4, hkv=4, d=64,
             block=16, dtype="f32", lo=5, hi=64, append=False),
        # Decode step of a batch of 64 at 512 to 4096 tokens, the step's append in it.
        dict(name="decode 64 x 4k fp8", op="decode", format="fp8", seqs=64, hq=32, hkv=8, d=128,
             block=16, dtype="bf16", lo=512, hi=4096, append=True),
        # The same batch at 4 bits.
        dict(name="decode 64 x 4k fp4", op="decode", format="fp4", seqs=64, hq=32, hkv=8, d=128,
             block=16, dtype="bf16", lo=512, hi=4096, append=False),
        # Long contexts, groups of 8 query heads.
        dict(name="decode 16 x 128k fp8", op="decode", format="fp8", seqs=16, hq=64, hkv=8,
             d=128, block=16, dtype="bf16", lo=16384, hi=131072, append=False),
        dict(name="decode 16 x 128k fp4", op="decode", format="fp4", seqs=16, hq=64, hkv=8,
             d=128, block=16, dtype="bf16", lo=16384, hi=131072, append=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    hkv = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=rng.choice(["append", "freeze", "thaw", "decode", "decode"]),
             format=rng.choice(["fp8", "fp4"]), hkv=hkv, d=rng.choice([64, 128]),
             block=rng.choice([16, 32]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if c["op"] == "append":
        c.update(tokens=_log(rng, 1, 8192), fused=rng.random() < 0.5)
    elif c["op"] in ("freeze", "thaw"):
        c.update(blocks=_log(rng, 1, 2048))
    else:
        hi = _log(rng, 1, 65536)
        c.update(hq=hkv * rng.choice([1, 2, 4, 8]),
                 seqs=_log(rng, 1, max(1, min(64, (1 << 18) // hi))), lo=_log(rng, 1, hi), hi=hi,
                 append=rng.random() < 0.5)
    return c


def _lengths(case):
    """Context lengths of a case, the longest among them (of its own sizes alone)."""
    r = random.Random(1000003 * case["hi"] + 1009 * case["lo"] + case["seqs"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    n[r.randrange(len(n))] = case["hi"]
    return n


# ------------------------------------------------------------------ the quantised row, in 32 bits

def _side_bytes(case):
    """Bytes beside the codes of 16 tokens of one kv head."""
    return case["d"] + 16 if case["format"] == "fp4" else 16


def _layout(case, is_v):
    """Where token t's scales and exponent lie beside its block: byte offsets [B, ...]."""
    d, fp4 = case["d"], case["format"] == "fp4"
    t = torch.arange(case["block"], device="cuda")
    chunk, t = t // 16 * _side_bytes(case), t % 16
    if not fp4:
        return None, chunk + t
    g = torch.arange(d // 16, device="cuda")
    at = (t // 4 * (d // 4) + t % 4)[:, None] + 4 * g if is_v else (t * (d // 16))[:, None] + g
    return chunk[:, None] + at, chunk + d + t


def _pow2(e):
    """2^e in 32 bits, for int32 e from -126 to 127."""
    return ((e + 127) << 23).view(torch.float32)


def _encode(x, fmt):
    """Rows x [..., D] as (codes uint8, scales uint8 or None, exponents uint8)."""
    x = x.float()
    bits = torch.nan_to_num(x.abs(), nan=0.0, posinf=3.0e38).amax(-1).view(torch.int32)
    if fmt == "fp8":
        e = (((bits + 0x1FFFFF) >> 23) - 135).clamp(-90, 90)     # 448 = 1.75 * 2^8
        y = (x * _pow2(-e)[..., None]).clamp(-448, 448)
        return y.to(torch.float8_e4m3fn).view(torch.uint8), None, (e + 127).to(torch.uint8)
    e = (((bits + 0x57FFFF) >> 23) - 138).clamp(-90, 90)         # 2688 = 1.3125 * 2^11
    y = (x * _pow2(-e)[..., None]).clamp(-2688, 2688)
    y = y.unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1, keepdim=True) / 6).to(torch.float8_e4m3fn)
    u = (y / s.float()).abs()
    code = ((u > 0.25).to(torch.uint8) + (u >= 0.75) + (u > 1.25) + (u >= 1.75) + (u > 2.5)
            + (u >= 3.5) + (u > 5)) | (y < 0).to(torch.uint8) << 3
    code = code.flatten(-2)
    pairs = code[..., 0::2] | code[..., 1::2] << 4
    return pairs, s.view(torch.uint8)[..., 0], (e + 127).to(torch.uint8)


def _decode(codes, scales, exps):
    """The values in 32 bits."""
    if scales is None:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                            device="cuda")
        v = e2m1[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
        v = (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None])
        v = v.flatten(-2)
    return v * _pow2(exps.int() - 127)[..., None]


def _put_rows(cache, blk, off, rows, fmt):
    """rows [T, Hkv, D] quantised into slots off [T] of blocks blk [T]."""
    codes, side, (at_scale, at_exp) = cache
    c, s, e = _encode(rows, fmt)
    h = torch.arange(codes.shape[1], device="cuda")[None, :]
    codes[blk[:, None], h, off[:, None]] = c
    side[blk[:, None], h, at_exp[off][:, None]] = e
    if s is not None:
        side[blk[:, None, None], h[..., None], at_scale[off][:, None]] = s


def _get_rows(cache, blk, off):
    """Rows of slots off [T] of blocks blk [T], [T, Hkv, D] in 32 bits."""
    codes, side, (at_scale, at_exp) = cache
    h = torch.arange(codes.shape[1], device="cuda")[None, :]
    s = None if at_scale is None else side[blk[:, None, None], h[..., None],
                                           at_scale[off][:, None]]
    return _decode(codes[blk[:, None], h, off[:, None]], s,
                   side[blk[:, None], h, at_exp[off][:, None]])


def _get_blocks(cache, ids):
    """Values of the blocks ids [...], [..., Hkv, B, D] in 32 bits."""
    codes, side, (at_scale, at_exp) = cache
    beside = side[ids]
    return _decode(codes[ids], None if at_scale is None else beside[..., at_scale],
                   beside[..., at_exp])


def _put_blocks(cache, ids, x, fmt):
    """x [n, Hkv, B, D] quantised into the blocks ids (a slice, or [n])."""
    codes, side, (at_scale, at_exp) = cache
    c, s, e = _encode(x, fmt)
    beside = torch.zeros(x.shape[:2] + side.shape[2:], dtype=torch.uint8, device="cuda")
    beside[..., at_exp] = e
    if s is not None:
        beside[..., at_scale] = s
    codes[ids], side[ids] = c, beside


# ------------------------------------------------------------------ inputs

def _rows(shape, g, dtype):
    """Rows as a model has them: of unequal sizes, a few channels above the rest."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda")).to(dtype)
    x[..., 5::37] *= 4
    return x


def _empty_cache(nb, case, is_v):
    """(codes, what lies beside them, where in it) of nb blocks."""
    B, d, hkv = case["block"], case["d"], case["hkv"]
    row = d // 2 if case["format"] == "fp4" else d
    return (torch.zeros((nb, hkv, B, row), dtype=torch.uint8, device="cuda"),
            torch.zeros((nb, hkv, B // 16 * _side_bytes(case)), dtype=torch.uint8,
                        device="cuda"), _layout(case, is_v))


def _quantised(nb, case, g, is_v):
    """nb blocks of quantised rows, made a part at a time."""
    cache = _empty_cache(nb, case, is_v)
    step = max(1, (1 << 25) // (case["hkv"] * case["block"] * case["d"]))
    for i in range(0, nb, step):
        n = min(step, nb - i)
        x = _rows((n, case["hkv"], case["block"], case["d"]), g, torch.bfloat16)
        _put_blocks(cache, slice(i, i + n), x, case["format"])
    return cache


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt, hkv, d, B = case["op"], DTYPES[case["dtype"]], case["hkv"], case["d"], case["block"]
    s = dict(case=case, op=op)
    if op == "append":
        T = case["tokens"]
        nb = -(-T // B) + 1 + T // (4 * B)
        x = _rows((T, 2 * hkv, d), g, dt)
        s["k"], s["v"] = x[:, :hkv], x[:, hkv:]                      # views of one projection
        if not case["fused"]:
            s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
        if T >= 2:
            s["v"][T // 3] = 0                                       # a row of zeros
        s["slots"] = torch.randperm(nb * B, generator=g, device="cuda", dtype=torch.int64)[:T]
        s["slots"] = s["slots"].contiguous()
        if T >= 16:
            s["slots"][T // 2] = -1                                  # a padding row
        s["k_cache"], s["v_cache"] = (_empty_cache(nb, case, v) for v in (False, True))
        s["k_out"], s["v_out"] = (torch.empty((T, hkv, d), device="cuda", dtype=dt)
                                  for _ in range(2))
        return s
    if op in ("freeze", "thaw"):
        n = case["blocks"]
        nb = n + n // 8 + 1
        src, dst = (torch.randperm(nb, generator=g, device="cuda")[:n] for _ in range(2))
        s["pairs"] = torch.stack((src, dst), 1).to(torch.int32).contiguous()
        s["back"] = s["pairs"].flip(1).contiguous()
        shape = (nb, hkv, B, d)
        if op == "freeze":
            s["k_pool"], s["v_pool"] = (_rows(shape, g, dt) for _ in range(2))
            s["k_cache"], s["v_cache"] = (_empty_cache(nb, case, v) for v in (False, True))
        else:
            s["k_cache"], s["v_cache"] = (_quantised(nb, case, g, v) for v in (False, True))
        s["k_out"], s["v_out"] = (torch.zeros(shape, device="cuda", dtype=dt) for _ in range(2))
        return s
    lens = _lengths(case)
    S = case["seqs"]
    need = [-(-n // B) for n in lens]
    total, cols = sum(need), max(need)
    nb = total + total // 8 + 1
    perm = torch.randperm(nb, generator=g, device="cuda", dtype=torch.int64)
    first = torch.tensor([sum(need[:i]) for i in range(S)], device="cuda")
    j = torch.arange(cols, device="cuda")
    at = (first[:, None] + j[None]).clamp_(max=nb - 1)
    there = j[None] < torch.tensor(need, device="cuda")[:, None]
    s["table"] = torch.where(there, perm[at], -1).to(torch.int32)
    s["k_cache"], s["v_cache"] = (_quantised(nb, case, g, v) for v in (False, True))
    s["q"] = torch.randn((S, case["hq"], d), generator=g, device="cuda", dtype=dt)
    s["out"] = torch.empty_like(s["q"])
    s["lens"], s["max_context"], s["scale"] = _i32(lens), max(lens), 1.0 / math.sqrt(d)
    s["k_new"] = s["v_new"] = None
    if case["append"]:
        s["k_new"], s["v_new"] = (_rows((S, hkv, d), g, dt) for _ in range(2))
        last = s["lens"].long() - 1
        blk = s["table"].gather(1, (last // B)[:, None])[:, 0].long()
        s["slots"] = blk * B + last % B
        s["k_out"], s["v_out"] = (torch.empty((S, hkv, d), device="cuda", dtype=dt)
                                  for _ in range(2))
    return s


# ------------------------------------------------------------------ plain forms

def _plain_append(s):
    c = s["case"]
    B, there = c["block"], s["slots"] >= 0
    slots = s["slots"][there]
    got = []
    for cache, rows in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        _put_rows(cache, slots // B, slots % B, rows[there], c["format"])
        back = torch.zeros(rows.shape, dtype=rows.dtype, device="cuda")   # padding reads zeros
        back[there] = _get_rows(cache, slots // B, slots % B).to(rows.dtype)
        got.append(back)
    return tuple(got)


def _plain_freeze(s):
    src, dst = s["pairs"].long().unbind(1)
    for pool, cache, out in ((s["k_pool"], s["k_cache"], s["k_out"]),
                             (s["v_pool"], s["v_cache"], s["v_out"])):
        _put_blocks(cache, dst, pool[src], s["case"]["format"])
        out[src] = _get_blocks(cache, dst).to(out.dtype)
    return s["k_out"], s["v_out"]


def _plain_thaw(s):
    src, dst = s["pairs"].long().unbind(1)
    for cache, out in ((s["k_cache"], s["k_out"]), (s["v_cache"], s["v_out"])):
        out[dst] = _get_blocks(cache, src).to(out.dtype)
    return s["k_out"], s["v_out"]


def _sequences(cache, table, n):
    """The first n tokens of each sequence, [S, Hkv, n, D] in 32 bits."""
    got = _get_blocks(cache, table.clamp(min=0).long())              # [S, nb, Hkv, B, D]
    S, nb, hkv, B, d = got.shape
    return got.permute(0, 2, 1, 3, 4).reshape(S, hkv, nb * B, d)[:, :, :n]


def _plain_decode(s):
    c = s["case"]
    S, hq, d = s["q"].shape
    hkv, B, n = c["hkv"], c["block"], s["max_context"]
    if c["append"]:
        blk, off = s["slots"] // B, s["slots"] % B
        _put_rows(s["k_cache"], blk, off, s["k_new"], c["format"])
        _put_rows(s["v_cache"], blk, off, s["v_new"], c["format"])
    q = s["q"].float().view(S, hkv, hq // hkv, d)
    x = torch.matmul(q, _sequences(s["k_cache"], s["table"], n).transpose(-1, -2))
    x *= s["scale"]
    there = torch.arange(n, device="cuda")[None] < s["lens"].long()[:, None]
    x.masked_fill_(~there[:, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x /= x.sum(-1, keepdim=True)
    out = torch.matmul(x, _sequences(s["v_cache"], s["table"], n))
    out = out.reshape(S, hq, d).to(s["q"].dtype)
    if not c["append"]:
        return out
    return (out, _get_rows(s["k_cache"], blk, off).to(s["q"].dtype),
            _get_rows(s["v_cache"], blk, off).to(s["q"].dtype))


_PLAIN = {"append": _plain_append, "freeze": _plain_freeze, "thaw": _plain_thaw,
          "decode": _plain_decode}


# ------------------------------------------------------------------ the library's calls

def _own_run(s):
    import paged_kv_cache_58_gb300 as pkv
    c, op = s["case"], s["op"]
    if "cache" not in s:             # a handle, kept beside the pools as a serving loop keeps it
        (k, ks, _), (v, vs, _) = s["k_cache"], s["v_cache"]
        s["cache"] = pkv.QuantCache(k, v, ks, vs, format=c["format"])
    cache = s["cache"]
    if op == "append":
        pkv.kv_append_quant(cache, s["slots"], s["k"], s["v"])
        return pkv.kv_read_quant(cache, s["slots"], k_out=s["k_out"], v_out=s["v_out"])
    if op == "freeze":
        pkv.quantize_blocks(cache, s["k_pool"], s["v_pool"], s["pairs"])
        pkv.dequantize_blocks(cache, s["k_out"], s["v_out"], s["back"])
        return s["k_out"], s["v_out"]
    if op == "thaw":
        pkv.dequantize_blocks(cache, s["k_out"], s["v_out"], s["pairs"])
        return s["k_out"], s["v_out"]
    if "workspace" not in s:
        need = pkv.decode_quant_workspace_bytes(cache, c["seqs"], c["hq"], s["max_context"])
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    out = pkv.paged_decode_quant(s["q"], cache, s["table"], s["lens"], s["scale"],
                                 max_context=s["max_context"], k_new=s["k_new"],
                                 v_new=s["v_new"], out=s["out"], workspace=s["workspace"])
    if not c["append"]:
        return out
    return (out,) + tuple(pkv.kv_read_quant(cache, s["slots"], k_out=s["k_out"],
                                            v_out=s["v_out"]))


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ work

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    hkv, d, B = case["hkv"], case["d"], case["block"]
    kept = (d // 2 if case["format"] == "fp4" else d) + _side_bytes(case) / 16
    row = d * es                                         # bytes of a row, and of it quantised
    if case["op"] == "append":                           # rows in, kept, read, rows out
        return {"bytes": case["tokens"] * (2 * hkv * (2 * row + 2 * kept) + 8), "flops": 0}
    if case["op"] == "freeze":
        return {"bytes": case["blocks"] * (2 * hkv * B * (2 * row + 2 * kept) + 16), "flops": 0}
    if case["op"] == "thaw":
        return {"bytes": case["blocks"] * (2 * hkv * B * (row + kept) + 8), "flops": 0}
    lens = _lengths(case)
    S, total = case["seqs"], sum(lens)
    new = S * hkv * 2 * (2 * row + 2 * kept) if case["append"] else 0
    return {"bytes": total * hkv * 2 * kept + 2 * S * case["hq"] * row + new
            + 4 * sum(-(-n // B) for n in lens),
            "flops": 4 * d * case["hq"] * total}


# ------------------------------------------------------------------ in 64 bits

def _two64(e):
    """2^e in 64 bits, exactly (pow and exp2 may be off in the last place)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest64(y, bits, low):
    """y at the nearest value with `bits` digits after the first, none finer than those at
    2^low (ties to even)."""
    exp = (torch.frexp(y)[1] - 1).clamp(min=low) - bits
    unit = _two64(exp)
    return torch.round(y / unit) * unit


def _kept64(x, fmt):
    """What the rows x [..., D] come back as."""
    x = x.double()
    m, ex = torch.frexp(x.abs().amax(-1, keepdim=True))
    top, where, digit = (448, 9, 0.875) if fmt == "fp8" else (2688, 12, 0.65625)
    e = torch.where(m == 0, -90, (ex - where + (m > digit)).clamp(-90, 90))
    unit = _two64(e)
    y = (x / unit).clamp(-top, top)
    if fmt == "fp8":
        return _nearest64(y, 3, -6) * unit
    y = y.unflatten(-1, (-1, 16))
    s = _nearest64(y.abs().amax(-1, keepdim=True) / 6, 3, -6)
    z = torch.where(s > 0, y / s.clamp(min=1e-300), torch.zeros_like(y))
    return (_nearest64(z, 1, 0).clamp(-6, 6) * s).flatten(-2) * unit


def _e4m3_64(b):
    """The values of e4m3 bytes: sign, four bits of exponent, three digits."""
    b = b.long()
    e, m = b >> 3 & 15, (b & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * _two64(e - 7), m / 512)
    return torch.where(b >= 128, -v, v)


def _tokens64(cache, case, is_v, ids, n):
    """Tokens 0 .. n - 1 of the blocks ids, [n, Hkv, D] in 64 bits, 16 by 16."""
    d, hkv = case["d"], case["hkv"]
    codes = cache[0][ids].transpose(1, 2).reshape(len(ids) * case["block"], hkv, -1)
    side = cache[1][ids].view(len(ids), hkv, -1, _side_bytes(case)).transpose(1, 2)
    side = side.reshape(-1, hkv, side.shape[-1])                     # [chunks, Hkv, bytes]
    if case["format"] == "fp4":
        sc = side[..., :d]
        sc = sc.reshape(-1, hkv, 4, d // 16, 4).transpose(-1, -2).reshape(-1, hkv, 16, d // 16) \
            if is_v else sc.reshape(-1, hkv, 16, d // 16)
        sc = sc.transpose(1, 2).reshape(-1, hkv, d // 16)
        nib = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
        e, m = nib >> 1 & 3, (nib & 1).double()
        val = torch.where(e > 0, (1 + m / 2) * _two64(e - 1), m / 2)
        val = torch.where(nib >= 8, -val, val)
        val = (val.unflatten(-1, (-1, 16)) * _e4m3_64(sc)[..., None]).flatten(-2)
    else:
        val = _e4m3_64(codes)
    exps = side[..., -16:].transpose(1, 2).reshape(-1, hkv, 1).long() - 127
    return (val * _two64(exps))[:n]


def _exact_decode(s):
    c = s["case"]
    hkv, d, B = c["hkv"], c["d"], c["block"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    if c["append"]:
        kn, vn = _kept64(s["k_new"], c["format"]), _kept64(s["v_new"], c["format"])
    for i, n in enumerate(s["lens"].tolist()):
        ids = s["table"][i, :-(-n // B)].long()
        k, v = (_tokens64(s[x], c, x == "v_cache", ids, n) for x in ("k_cache", "v_cache"))
        if c["append"]:
            k[n - 1], v[n - 1] = kn[i], vn[i]
        q = s["q"][i].double().view(hkv, -1, d)
        p = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) * s["scale"], -1)
        out[i] = torch.einsum("hgn,nhd->hgd", p, v).reshape(-1, d)
    return (out, kn, vn) if c["append"] else out


def _exact_freeze(s):
    back = []
    for pool in (s["k_pool"], s["v_pool"]):
        out = torch.zeros(pool.shape, dtype=torch.float64, device="cuda")
        src = s["pairs"][:, 0].long()
        out[src] = _kept64(pool[src], s["case"]["format"])
        back.append(out)
    return tuple(back)


def _exact_thaw(s):
    c = s["case"]
    src, dst = s["pairs"].long().unbind(1)
    got = []
    for cache, shape, is_v in ((s["k_cache"], s["k_out"].shape, False),
                               (s["v_cache"], s["v_out"].shape, True)):
        out = torch.zeros(shape, dtype=torch.float64, device="cuda")
        x = _tokens64(cache, c, is_v, src, len(src) * c["block"])
        out[dst] = x.view(len(src), c["block"], c["hkv"], c["d"]).transpose(1, 2)
        got.append(out)
    return tuple(got)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "append":
        there = (s["slots"] >= 0)[:, None, None]
        return tuple(_kept64(s[x], case["format"]) * there for x in ("k", "v"))
    return {"freeze": _exact_freeze, "thaw": _exact_thaw, "decode": _exact_decode}[s["op"]](s)
