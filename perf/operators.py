"""The cases at which the operators around a shrinking paged cache are measured.

Rotary positions (alone, and with the append of the rotated keys), decode and prefill
forms that accumulate the attention weight each cached token receives, and the eviction
that goes by it.  A case names its operator ("op") and its sizes; `prepare` makes the
inputs on the GPU, `run` makes one pass (in plain torch operations, or with `own` through
the library), `work` counts what a pass cannot do without and `exact` gives its outputs
in 64 bits.  Lengths follow from the case, values from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One decode step of a batch of 64: rotate q and k of the new tokens, k and v to
        # their slots.  A few microseconds: latency.
        dict(name="rope step of 64", op="rope_append", tokens=64, hq=32, hkv=8, d=128, block=16,
             dtype="bf16", rotary=128, interleaved=False, far=4096, fused=True),
        # The new tokens of 16 prompts of 512, as slices of one fused projection.
        dict(name="rope prompts 8192", op="rope_append", tokens=8192, hq=32, hkv=8, d=128,
             block=16, dtype="bf16", rotary=128, interleaved=False, far=131072, fused=True),
        # The gradient's rotation (inverse), neighbouring pairs, half of a short head, an
        # odd number of tokens, fp32.
        dict(name="rope inverse f32 4097", op="rope", tokens=4097, hq=16, hkv=16, d=64, block=16,
             dtype="f32", rotary=32, interleaved=True, far=1000000, fused=False),
        # Decode of 4 short sequences on an fp32 pool: latency.
        dict(name="decode tiny f32", op="decode_weights", seqs=4, hq=4, hkv=4, d=64, block=16,
             dtype="f32", lo=5, hi=64, append=True),
        # Decode step of a batch of 64 at 512 to 4096 tokens, the step's append in it.
        dict(name="decode 64 x 4k", op="decode_weights", seqs=64, hq=32, hkv=8, d=128, block=16,
             dtype="bf16", lo=512, hi=4096, append=True),
        # Long contexts, groups of 8 query heads.
        dict(name="decode 16 x 128k", op="decode_weights", seqs=16, hq=64, hkv=8, d=128, block=16,
             dtype="bf16", lo=16384, hi=131072, append=False),
        # Three short prompts on an fp32 pool, every new token counted.
        dict(name="prompt weights small f32", op="prefill_weights", seqs=3, hq=8, hkv=4, d=64,
             block=16, dtype="f32", lo=0, hi=200, new=77, window=0),
        # The last 64 tokens of each prompt's chunk as the observers of the cache.
        dict(name="prompt weights last 64", op="prefill_weights", seqs=16, hq=32, hkv=8, d=128,
             block=16, dtype="bf16", lo=1024, hi=8192, new=512, window=64),
        # Every new token of the chunk counted.
        dict(name="prompt weights all 512", op="prefill_weights", seqs=16, hq=32, hkv=8, d=128,
             block=16, dtype="bf16", lo=1024, hi=8192, new=512, window=0),
        # A running batch in which every sequence has grown a block past its budget.
        dict(name="evict a block of 64", op="evict", seqs=64, hkv=8, d=128, block=16,
             dtype="bf16", lo=1040, hi=1040, budget=1024, sinks=4, recent=256, tracked=1024),
        # After the prompts: 512 to 4096 tokens down to 1024.
        dict(name="evict 64 x 4k", op="evict", seqs=64, hkv=8, d=128, block=16, dtype="bf16",
             lo=512, hi=4096, budget=1024, sinks=4, recent=256, tracked=0),
        # Long contexts down to 8192.
        dict(name="evict 16 x 128k", op="evict", seqs=16, hkv=8, d=128, block=16, dtype="bf16",
             lo=16384, hi=131072, budget=8192, sinks=16, recent=1024, tracked=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    d = rng.choice([64, 128])
    block = rng.choice([16, 32])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["rope", "rope_append", "decode_weights", "prefill_weights", "evict"])
    c = dict(op=op, hkv=hkv, d=d, block=block, dtype=dtype)
    if op in ("rope", "rope_append"):
        c.update(hq=hkv * group, tokens=_log(rng, 1, 4096), rotary=16 * rng.randint(1, d // 16),
                 interleaved=rng.random() < 0.5, far=_log(rng, 1, 1 << 20),
                 fused=rng.random() < 0.5)
        return c
    if op == "decode_weights":
        hi = _log(rng, 1, 32768)
        c.update(hq=hkv * group, seqs=_log(rng, 1, max(1, min(64, (1 << 18) // hi))),
                 lo=_log(rng, 1, hi), hi=hi, append=rng.random() < 0.5)
        return c
    if op == "prefill_weights":
        new = _log(rng, 1, 512)
        hi = _log(rng, 1, 8192 if dtype == "bf16" else 2048)
        c.update(hq=hkv * group, seqs=_log(rng, 1, max(1, min(16, (1 << 15) // (hi + new)))),
                 lo=rng.choice([0, _log(rng, 1, hi)]), hi=hi, new=new,
                 window=rng.choice([0, 0, _log(rng, 1, 128)]))
        return c
    hi = _log(rng, 2, 65536)
    budget = _log(rng, 1, hi)
    c.update(seqs=_log(rng, 1, max(1, min(64, (1 << 18) // hi))), lo=_log(rng, 1, hi), hi=hi,
             budget=budget, sinks=rng.randint(0, min(16, budget)),
             recent=rng.randint(0, budget), tracked=rng.choice([0, budget]))
    c["lo"] = max(c["lo"], min(hi, c["tracked"]))
    return c


def _lengths(case):
    """Context lengths of a case, the longest among them (of its own sizes alone)."""
    r = random.Random(1000003 * case["hi"] + 1009 * case["lo"] + case["seqs"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    n[r.randrange(len(n))] = case["hi"]
    return n


# ------------------------------------------------------------------ inputs

def _paged(lens, case, g):
    """K and V pools of scattered blocks, and the block table of sequences of these lengths."""
    B, dt = case["block"], DTYPES[case["dtype"]]
    need = [-(-n // B) for n in lens]
    cols = max(max(need), 1)
    total = max(sum(need), 1)
    nb = total + total // 8 + 1
    perm = torch.randperm(nb, generator=g, device="cuda", dtype=torch.int64)
    first = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")
    have = torch.tensor(need, device="cuda")
    j = torch.arange(cols, device="cuda")
    at = (first[:, None] + j[None]).clamp_(max=nb - 1)
    table = torch.where(j[None] < have[:, None], perm[at], -1).to(torch.int32)
    shape = (nb, case["hkv"], B, case["d"])
    k = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    v = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    return k, v, table


def _frequencies(rotary, far):
    """Rotary frequencies of base 10000; past 8192 positions they are stretched linearly."""
    i = torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-i / rotary)
    return f / 4 if far > 8192 else f


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case=case, op=op)
    if op in ("rope", "rope_append"):
        T, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        heads = hq + 2 * hkv
        x = torch.randn((T, heads, d), generator=g, device="cuda", dtype=dt)
        parts = [x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]]   # views of one projection
        s["q"], s["k"], s["v"] = parts if case["fused"] else [p.contiguous() for p in parts]
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda",
                                       dtype=torch.int32)
        s["inv_freq"] = _frequencies(case["rotary"], case["far"])
        s["attn_scale"] = 1.0 if case["far"] <= 8192 else 1.125
        s["q_out"] = torch.empty((T, hq, d), device="cuda", dtype=dt)
        if op == "rope_append":
            B = case["block"]
            nb = -(-T // B) + 1 + T // (4 * B)
            s["k_pool"] = torch.randn((nb, hkv, B, d), generator=g, device="cuda", dtype=dt)
            s["v_pool"] = torch.randn((nb, hkv, B, d), generator=g, device="cuda", dtype=dt)
            s["slots"] = torch.randperm(nb * B, generator=g, device="cuda", dtype=torch.int64)[:T]
            s["slots"] = s["slots"].contiguous()
            if T >= 16:
                s["slots"][T // 2] = -1   # a padding row
        return s
    lens = _lengths(case)
    S, hkv, d = case["seqs"], case["hkv"], case["d"]
    if op == "decode_weights":
        s["k_pool"], s["v_pool"], s["table"] = _paged(lens, case, g)
        W = max(lens) + 5
        s["q"] = torch.randn((S, case["hq"], d), generator=g, device="cuda", dtype=dt)
        s["out"] = torch.empty_like(s["q"])
        s["k_new"] = s["v_new"] = None
        if case["append"]:
            s["k_new"] = torch.randn((S, hkv, d), generator=g, device="cuda", dtype=dt)
            s["v_new"] = torch.randn((S, hkv, d), generator=g, device="cuda", dtype=dt)
        s["lens"], s["max_context"] = _i32(lens), max(lens)
        # what earlier steps left, in rows of the sequences' own
        s["weights"] = torch.rand((S + 2, hkv, W), generator=g, device="cuda") * (4.0 / max(lens))
        s["row_ids"] = torch.randperm(S + 2, generator=g, device="cuda")[:S].to(torch.int32)
        s["decay"] = 0.98
    elif op == "prefill_weights":
        new = [max(1, case["new"] - 3 * (i % 4)) for i in range(S)]
        total = [c + n for c, n in zip(lens, new)]
        s["k_pool"], s["v_pool"], s["table"] = _paged(total, case, g)
        s["cached"], s["new"] = _i32(lens), _i32(new)
        s["offsets"] = _i32([sum(new[:i]) for i in range(S + 1)])
        s["new_host"], s["total_host"] = new, total
        s["q"] = torch.randn((sum(new), case["hq"], d), generator=g, device="cuda", dtype=dt)
        s["weights"] = torch.zeros((S, hkv, max(total) + 64), device="cuda")
    else:
        s["k_pool"], s["v_pool"], s["table"] = _paged(lens, case, g)
        W = max(lens) + 7
        w = torch.exp(2.0 * torch.randn((S, hkv, W), generator=g, device="cuda"))
        none = torch.rand((S, hkv, W), generator=g, device="cuda") < 0.05
        s["weights"] = torch.where(none, torch.zeros_like(w), w)   # some were never looked at
        s["weights_out"] = torch.zeros_like(w)
        gone, t = 100, case["tracked"]
        s["positions"] = torch.zeros((S, hkv, W), dtype=torch.int32, device="cuda")
        if t:
            order = torch.rand((S, hkv, t + gone), generator=g, device="cuda").argsort(-1)
            s["positions"][..., :t] = order[..., :t]
        s["positions_out"] = torch.zeros_like(s["positions"])
        s["lens"], s["budgets"] = _i32(lens), _i32([case["budget"]] * S)
        s["seen"] = _i32([n + (gone if t else 0) for n in lens])
        s["tracked"] = _i32([min(t, n) for n in lens])
        s["new_lens"] = torch.zeros((S,), dtype=torch.int32, device="cuda")
        s["max_context"] = max(lens)
    if op != "evict":
        s["scale"] = 1.0 / math.sqrt(d)
    return s


# ------------------------------------------------------------------ plain forms

def _rotate(x, positions, inv_freq, interleaved, sign, scale):
    """x [T, H, D] rotated in 32 bits; the angles of far positions in 64."""
    angle = positions.double()[:, None] * inv_freq[None]
    cos = (torch.cos(angle) * scale).float()[:, None]
    sin = (torch.sin(angle) * (sign * scale)).float()[:, None]
    r = 2 * inv_freq.numel()
    y = x.float()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, y[..., r:]), -1).to(x.dtype)


def _gather(pool, table, n):
    """The first n tokens of each sequence, [S, Hkv, n, D] in 32 bits."""
    got = pool[table.clamp(min=0).long()].float()            # [S, nb, Hkv, B, D]
    S, nb, hkv, B, d = got.shape
    return got.permute(0, 2, 1, 3, 4).reshape(S, hkv, nb * B, d)[:, :, :n]


def _plain_rope(s):
    c = s["case"]
    T, B = c["tokens"], c["block"]
    if c["op"] == "rope":
        return _rotate(s["q"], s["positions"], s["inv_freq"], c["interleaved"], -1.0,
                       s["attn_scale"])
    q = _rotate(s["q"], s["positions"], s["inv_freq"], c["interleaved"], 1.0, s["attn_scale"])
    k = _rotate(s["k"], s["positions"], s["inv_freq"], c["interleaved"], 1.0, s["attn_scale"])
    there = s["slots"] >= 0
    blk, off = s["slots"][there] // B, s["slots"][there] % B
    s["k_pool"][blk, :, off] = k[there]
    s["v_pool"][blk, :, off] = s["v"][there]
    return q, s["k_pool"], s["v_pool"]


def _plain_decode(s):
    c = s["case"]
    S, hq, d = s["q"].shape
    hkv, B, n = c["hkv"], c["block"], s["max_context"]
    lens = s["lens"].long()
    if c["append"]:
        at = lens - 1
        blk = s["table"].gather(1, (at // B)[:, None])[:, 0].long()
        s["k_pool"][blk, :, at % B] = s["k_new"]
        s["v_pool"][blk, :, at % B] = s["v_new"]
    k, v = _gather(s["k_pool"], s["table"], n), _gather(s["v_pool"], s["table"], n)
    q = s["q"].float().view(S, hkv, hq // hkv, d)
    x = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    there = torch.arange(n, device="cuda")[None] < lens[:, None]
    x.masked_fill_(~there[:, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    p = x / x.sum(-1, keepdim=True)
    out = torch.matmul(p, v).reshape(S, hq, d).to(s["q"].dtype)
    rows = s["row_ids"].long()
    w = s["weights"][rows]
    w[..., :n] = torch.where(there[:, None], w[..., :n] * s["decay"] + p.sum(2), w[..., :n])
    s["weights"][rows] = w
    return (out, s["weights"]) + ((s["k_pool"], s["v_pool"]) if c["append"] else ())


def _plain_prefill(s):
    c = s["case"]
    S, hkv, d = c["seqs"], c["hkv"], c["d"]
    n, rows = max(s["total_host"]), max(s["new_host"])
    rows = min(rows, c["window"]) if c["window"] else rows
    new, cached = s["new"].long(), s["cached"].long()
    i = torch.arange(rows, device="cuda")[None] + (new[:, None] - rows)       # a token's place
    seen = i >= 0                                                            # in the chunk
    q = s["q"][(s["offsets"][:-1].long()[:, None] + i).clamp(min=0)].float()  # [S, rows, Hq, D]
    q = q.view(S, rows, hkv, -1, d).permute(0, 2, 3, 1, 4)                   # [S, Hkv, G, rows, D]
    k = _gather(s["k_pool"], s["table"], n)
    x = torch.matmul(q, k[:, :, None].transpose(-1, -2)) * s["scale"]
    j = torch.arange(n, device="cuda")
    sees = j[None, None] <= (cached[:, None] + i)[..., None]                 # [S, rows, n]
    x.masked_fill_(~sees[:, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-37) * seen[:, None, None, :, None]
    s["weights"][..., :n] += x.sum((2, 3))
    return s["weights"]


def _plain_evict(s):
    c = s["case"]
    B, n = c["block"], s["max_context"]
    lens, budget = s["lens"].long()[:, None, None], s["budgets"].long()[:, None, None]
    seen, tracked = s["seen"].long()[:, None, None], s["tracked"].long()[:, None, None]
    j = torch.arange(n, device="cuda")[None, None]
    w, pos = s["weights"][..., :n], s["positions"][..., :n].long()
    pos = torch.where(j < tracked, pos, seen - lens + j)
    there = j < lens
    safe = there & ((pos < c["sinks"]) | (pos >= seen - c["recent"]))
    # by class, then weight, then index: two stable sorts, the lesser key first
    first = torch.sort(w, dim=-1, descending=True, stable=True).indices
    rank = torch.where(there, torch.where(safe, 2, 1), 0)
    second = torch.sort(rank.gather(-1, first), dim=-1, descending=True, stable=True).indices
    order = first.gather(-1, second)
    keep = torch.zeros_like(there.expand_as(w))
    keep.scatter_(-1, order, (j < budget).expand_as(w))
    keep &= there
    hole, mover = ~keep & (j < budget) & there, keep & (j >= budget)
    sh, hh, jh = hole.nonzero(as_tuple=True)   # the k-th mover goes to the k-th hole
    sm, hm, jm = mover.nonzero(as_tuple=True)
    table = s["table"].long()
    for pool in (s["k_pool"], s["v_pool"]):
        pool[table[sh, jh // B], hh, jh % B] = pool[table[sm, jm // B], hm, jm % B]
    left = torch.minimum(lens, budget)
    wo = torch.where(j < left, w, torch.zeros_like(w))
    po = pos.to(torch.int32)
    wo[sh, hh, jh] = w[sm, hm, jm]
    po[sh, hh, jh] = po[sm, hm, jm]
    s["weights_out"][..., :n] = torch.where(there, wo, s["weights_out"][..., :n])
    s["positions_out"][..., :n] = torch.where(j < left, po, s["positions_out"][..., :n])
    s["new_lens"].copy_(left[:, 0, 0])
    return s["weights_out"], s["positions_out"], s["new_lens"], s["k_pool"], s["v_pool"]


_PLAIN = {"rope": _plain_rope, "rope_append": _plain_rope, "decode_weights": _plain_decode,
          "prefill_weights": _plain_prefill, "evict": _plain_evict}


# ------------------------------------------------------------------ the library's calls

def _workspace(s, nbytes):
    """A workspace kept beside the inputs, as a serving loop keeps it."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(nbytes(), 16), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_run(s):
    import paged_kv_cache_58_gb300 as pkv
    c, op = s["case"], s["op"]
    if op == "rope":
        return pkv.rope(s["q"], s["positions"], s["inv_freq"], interleaved=c["interleaved"],
                        inverse=True, attn_scale=s["attn_scale"], out=s["q_out"])
    if op == "rope_append":
        q = pkv.rope_append(s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["slots"],
                            s["positions"], s["inv_freq"], interleaved=c["interleaved"],
                            attn_scale=s["attn_scale"], q_out=s["q_out"])
        return q, s["k_pool"], s["v_pool"]
    if op == "decode_weights":
        ws = _workspace(s, lambda: pkv.decode_weights_workspace_bytes(
            s["k_pool"], c["seqs"], c["hq"], s["max_context"]))
        out = pkv.paged_decode_weights(
            s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["scale"], s["weights"],
            max_context=s["max_context"], k_new=s["k_new"], v_new=s["v_new"],
            row_ids=s["row_ids"], decay=s["decay"], out=s["out"], workspace=ws)
        return (out, s["weights"]) + ((s["k_pool"], s["v_pool"]) if c["append"] else ())
    if op == "prefill_weights":
        ws = _workspace(s, lambda: pkv.prefill_weights_workspace_bytes(
            s["k_pool"], c["seqs"], c["hq"], max(s["new_host"]), max(s["total_host"]),
            c["window"]))
        return pkv.paged_prefill_weights(
            s["q"], s["k_pool"], s["table"], s["cached"], s["new"], s["offsets"], s["scale"],
            s["weights"], max_new=max(s["new_host"]), max_context=max(s["total_host"]),
            window=c["window"], workspace=ws)
    ws = _workspace(s, lambda: pkv.evict_workspace_bytes(s["k_pool"], c["seqs"],
                                                         s["max_context"]))
    pkv.evict(s["k_pool"], s["v_pool"], s["table"], s["lens"], s["budgets"], s["weights"],
              s["positions"], max_context=s["max_context"], sinks=c["sinks"],
              recent=c["recent"], seen_lens=s["seen"], tracked_lens=s["tracked"],
              weights_out=s["weights_out"], positions_out=s["positions_out"],
              new_lens=s["new_lens"], workspace=ws)
    return s["weights_out"], s["positions_out"], s["new_lens"], s["k_pool"], s["v_pool"]


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ work

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op, hkv, d = case["op"], case["hkv"], case["d"]
    row = d * es
    if op == "rope":
        return {"bytes": case["tokens"] * (2 * case["hq"] * row + 4),
                "flops": case["tokens"] * case["hq"] * 3 * case["rotary"]}
    if op == "rope_append":
        t = case["tokens"]
        return {"bytes": t * (2 * (case["hq"] + 2 * hkv) * row + 12),
                "flops": t * (case["hq"] + hkv) * 3 * case["rotary"]}
    lens = _lengths(case)
    S, total = case["seqs"], sum(lens)
    if op == "decode_weights":
        new = S * hkv * 2 * 2 * row if case["append"] else 0
        return {"bytes": total * hkv * (2 * row + 8) + 2 * S * case["hq"] * row + new
                + 4 * sum(-(-n // case["block"]) for n in lens),
                "flops": 4 * d * case["hq"] * total}
    if op == "prefill_weights":
        by = fl = 0
        for i, c in enumerate(lens):
            n = max(1, case["new"] - 3 * (i % 4))
            m = min(n, case["window"]) if case["window"] else n
            by += (c + n) * hkv * (row + 8) + m * case["hq"] * row
            fl += 2 * d * case["hq"] * (m * (c + n - m) + m * (m + 1) // 2)
        return {"bytes": by, "flops": fl}
    by = 0
    for n in lens:
        b = min(n, case["budget"])
        read = n + min(n, case["tracked"])                 # weights, and positions on record
        late = max(0, n - b)                               # entries past the budget
        safe = min(case["recent"], n)
        free = max(1, n - safe - min(case["sinks"], n))
        share = max(0, b - safe - min(case["sinks"], n)) / free
        moved = min(late, min(late, safe) + max(0, late - safe) * min(1.0, share))
        by += hkv * (4 * read + 4 * n + 4 * b + int(moved) * 4 * row)
    return {"bytes": by, "flops": 0}


# ------------------------------------------------------------------ in 64 bits

def _tokens64(pool, table, i, n):
    """Tokens 0 .. n - 1 of sequence i, [n, Hkv, D] in 64 bits."""
    B = pool.shape[2]
    ids = table[i, :-(-n // B)].long()
    return pool[ids].transpose(1, 2).reshape(-1, pool.shape[1], pool.shape[3])[:n].double()


def _exact_rope(s):
    c = s["case"]
    f, pos = s["inv_freq"], s["positions"].double()
    turn = torch.polar(torch.full((pos.numel(), f.numel()), float(s["attn_scale"]),
                                  dtype=torch.float64, device="cuda"), pos[:, None] * f[None])
    if c["op"] == "rope":
        turn = turn.conj()
    r = 2 * f.numel()

    def rotated(x):
        y = x.double().clone()
        lo, hi = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2),
                                                                            slice(r // 2, r))
        z = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * turn[:, None]
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    if c["op"] == "rope":
        return rotated(s["q"])
    k, v = s["k_pool"].double(), s["v_pool"].double()
    rk, rv = rotated(s["k"]), s["v"].double()
    B, hkv, d = c["block"], c["hkv"], c["d"]
    at = torch.nonzero(s["slots"] >= 0)[:, 0]
    flat = (s["slots"][at] // B) * (hkv * B) + s["slots"][at] % B
    flat = (flat[:, None] + B * torch.arange(hkv, device="cuda")[None]).reshape(-1)
    k.view(-1, d).index_copy_(0, flat, rk[at].reshape(-1, d))
    v.view(-1, d).index_copy_(0, flat, rv[at].reshape(-1, d))
    return rotated(s["q"]), k, v


def _exact_decode(s):
    c = s["case"]
    hkv, d = c["hkv"], c["d"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    w = s["weights"].double()
    if c["append"]:
        for i, n in enumerate(s["lens"].tolist()):
            at = int(s["table"][i, (n - 1) // c["block"]])
            s["k_pool"][at, :, (n - 1) % c["block"]] = s["k_new"][i]
            s["v_pool"][at, :, (n - 1) % c["block"]] = s["v_new"][i]
    for i, n in enumerate(s["lens"].tolist()):
        k, v = _tokens64(s["k_pool"], s["table"], i, n), _tokens64(s["v_pool"], s["table"], i, n)
        q = s["q"][i].double().view(hkv, -1, d)
        p = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) * s["scale"], -1)
        out[i] = torch.einsum("hgn,nhd->hgd", p, v).reshape(-1, d)
        r = int(s["row_ids"][i])
        w[r, :, :n] = w[r, :, :n] * s["decay"] + p.sum(1)
    return (out, w) + ((s["k_pool"], s["v_pool"]) if c["append"] else ())


def _exact_prefill(s):
    c = s["case"]
    hkv, d = c["hkv"], c["d"]
    w = s["weights"].double()
    o = s["offsets"].tolist()
    for i, n in enumerate(s["total_host"]):
        new = s["new_host"][i]
        m = min(new, c["window"]) if c["window"] else new
        k = _tokens64(s["k_pool"], s["table"], i, n)
        q = s["q"][o[i + 1] - m:o[i + 1]].double().view(m, hkv, -1, d)
        for h in range(hkv):
            x = torch.einsum("mgd,nd->mgn", q[:, h], k[:, h]) * s["scale"]
            future = torch.ones((m, n), dtype=torch.bool, device="cuda").triu(n - m + 1)
            x.masked_fill_(future[:, None], -math.inf)
            w[i, h, :n] += torch.softmax(x, -1).sum((0, 1))
    return w


def _exact_evict(s):
    c = s["case"]
    B, budget = c["block"], c["budget"]
    wo, po = s["weights_out"].double(), s["positions_out"].clone()
    table, left = s["table"].long(), []
    for i, n in enumerate(s["lens"].tolist()):
        seen, tracked = int(s["seen"][i]), int(s["tracked"][i])
        b = min(n, budget)
        left.append(b)
        for h in range(c["hkv"]):
            w = s["weights"][i, h, :n].double()
            pos = torch.arange(seen - n, seen, device="cuda")
            pos[:tracked] = s["positions"][i, h, :tracked]
            safe = (pos < c["sinks"]) | (pos >= seen - c["recent"])
            # a number that orders by class first, then by weight
            value = torch.unique(w, return_inverse=True)[1] + torch.where(safe, n, 0)
            best = torch.argsort(value, descending=True, stable=True)[:b]
            keep = torch.zeros(n, dtype=torch.bool, device="cuda")
            keep[best] = True
            source = torch.arange(b, device="cuda")
            source[~keep[:b]] = torch.nonzero(keep[b:])[:, 0] + b
            wo[i, h, :n] = 0
            wo[i, h, :b], po[i, h, :b] = w[source], pos[source].to(torch.int32)
            old, new = source[source >= b], torch.nonzero(source >= b)[:, 0]
            for pool in (s["k_pool"], s["v_pool"]):
                pool[table[i, new // B], h, new % B] = pool[table[i, old // B], h, old % B]
    return wo, po, _i32(left), s["k_pool"], s["v_pool"]


_EXACT = {"rope": _exact_rope, "rope_append": _exact_rope, "decode_weights": _exact_decode,
          "prefill_weights": _exact_prefill, "evict": _exact_evict}


def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)
