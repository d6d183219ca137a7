"""Decode and prefill forms that accumulate the attention weight of each cached token,
against the 64-bit sums; the decode's output and pools against the calls without weights."""
import os

import pytest
import torch

from tests.shrink_refs import attention, tokens, weight_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_58_gb300 import build
    build.build()
    import paged_kv_cache_58_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def paged(lens, hkv, bs, d, dtype, g, extra=3):
    """Pools in which every row outside the sequences is NaN, and their table."""
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + extra
    perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32, device="cuda")
    kp = torch.full((nb, hkv, bs, d), float("nan"), device="cuda", dtype=dtype)
    vp = kp.clone()
    at = 0
    for i, n in enumerate(lens):
        ids = perm[at:at + need[i]]
        at += need[i]
        table[i, :need[i]] = ids
        for pool in (kp, vp):
            rows = torch.randn(need[i] * bs, hkv, d, generator=g, device="cuda").to(dtype)
            rows[n:] = float("nan")
            pool[ids.long()] = rows.view(need[i], bs, hkv, d).transpose(1, 2)
    return kp, vp, table


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


DECODE = [  # lens, hkv, group, d, bs, dtype, partition_blocks
    ([1], 1, 1, 64, 16, torch.bfloat16, 0),
    ([17, 33, 5, 64], 4, 1, 64, 16, torch.float32, 0),
    ([17, 33, 5, 64], 4, 1, 64, 16, torch.float32, 1),
    ([1, 2, 15, 16, 17, 31, 32, 33], 2, 2, 128, 32, torch.bfloat16, 0),
    ([700, 1, 129], 3, 4, 128, 16, torch.bfloat16, 0),
    ([700, 1, 129], 3, 8, 64, 16, torch.bfloat16, 2),
    ([513, 512, 511, 1500], 8, 4, 128, 16, torch.bfloat16, 8),
    ([300, 90], 2, 8, 128, 32, torch.float32, 3),
    ([2100, 64], 1, 8, 128, 16, torch.bfloat16, 0),
    ([600], 2, 2, 64, 32, torch.float32, 0),
]


@pytest.mark.parametrize("case", DECODE)
@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("simt", [False, True])
def test_decode_weights(pkv, case, append, simt, monkeypatch):
    lens, hkv, group, d, bs, dtype, pb = case
    if simt:
        if dtype == torch.float32:
            pytest.skip("fp32 always runs there")
        monkeypatch.setenv("PKV_DECODE_KERNEL", "simt")
    g = gen(sum(lens))
    S, hq = len(lens), hkv * group
    kp, vp, table = paged(lens, hkv, bs, d, dtype, g)
    q = torch.randn(S, hq, d, generator=g, device="cuda").to(dtype)
    kn = torch.randn(S, hkv, d, generator=g, device="cuda").to(dtype) if append else None
    vn = torch.randn(S, hkv, d, generator=g, device="cuda").to(dtype) if append else None
    W = max(lens) + 3
    w0 = torch.rand(S + 2, hkv, W, generator=g, device="cuda")
    ids = torch.randperm(S + 2, generator=g, device="cuda")[:S].to(torch.int32)
    kp2, vp2, w = kp.clone(), vp.clone(), w0.clone()
    cl, scale = i32(lens), d ** -0.5
    out = pkv.paged_decode_weights(q, kp, vp, table, cl, scale, w, max_context=max(lens),
                                   k_new=kn, v_new=vn, row_ids=ids, decay=0.75,
                                   partition_blocks=pb)
    if append:
        same = pkv.paged_decode_append(q, kp2, vp2, kn, vn, table, cl, scale,
                                       max_context=max(lens), partition_blocks=pb)
    else:
        same = pkv.paged_decode(q, kp2, vp2, table, cl, scale, max_context=max(lens),
                                partition_blocks=pb)
    assert pkv.read_device_status() == 0
    assert torch.equal(out, same)                       # output and pools of the plain call
    for a, b in ((kp, kp2), (vp, vp2)):
        assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
    kc, tc = kp.cpu(), table.cpu()
    untouched = torch.ones(S + 2, dtype=torch.bool)
    for i, n in enumerate(lens):
        k = tokens(kc, tc[i], n)
        _, p, size = attention(q[i:i + 1].cpu(), k, None, scale, first=n - 1)
        row = int(ids[i])
        untouched[row] = False
        before = w0[row, :, :n].cpu().double()
        got = w[row].cpu().double()
        ref = 0.75 * before + p
        err = (got[:, :n] - ref).abs()
        assert bool((err <= weight_bound(p, before, size, d, n + group)).all()), err.max()
        assert torch.equal(w[row, :, n:], w0[row, :, n:])          # past the context
        total = (got[:, :n] - 0.75 * before).sum(-1)               # each head's sum is 1
        assert float((total - group).abs().max()) < 1e-3 * group
    assert torch.equal(w.cpu()[untouched], w0.cpu()[untouched])
    # the same call gives the same bits; decay 0 overwrites, whatever was there
    w2 = w0.clone()
    pkv.paged_decode_weights(q, kp, vp, table, cl, scale, w2, max_context=max(lens), k_new=kn,
                             v_new=vn, row_ids=ids, decay=0.75, partition_blocks=pb)
    assert torch.equal(w2, w)
    w3 = torch.full_like(w0, float("nan"))
    pkv.paged_decode_weights(q, kp, vp, table, cl, scale, w3, max_context=max(lens), k_new=kn,
                             v_new=vn, row_ids=ids, decay=0.0, partition_blocks=pb)
    for i, n in enumerate(lens):
        row = int(ids[i])
        got, base = w3[row, :, :n].cpu().double(), w[row, :, :n].cpu().double()
        before = w0[row, :, :n].cpu().double()
        bound = 4 * 2.0 ** -24 * (before + base.abs() + got)
        assert bool(((got + 0.75 * before - base).abs() <= bound).all())


def test_decode_weights_padding_and_lengths(pkv):
    """Rows of padding sequences, empty contexts and lengths out of range."""
    g = gen(4)
    lens = [40, 40, 40, 40]
    kp, vp, table = paged(lens, 2, 16, 64, torch.bfloat16, g)
    q = torch.randn(4, 4, 64, generator=g, device="cuda").bfloat16()
    w = torch.ones(4, 2, 48, device="cuda")
    pkv.paged_decode_weights(q, kp, vp, table, i32(lens), 0.125, w, max_context=40,
                             row_ids=i32([-1, 2, -1, 0]))
    assert pkv.read_device_status() == 0
    assert bool((w[1] == 1).all()) and bool((w[3] == 1).all())
    assert bool((w[0, :, :40] > 1).all()) and bool((w[2, :, :40] > 1).all())
    assert bool((w[:, :, 40:] == 1).all())
    w.fill_(1)
    pkv.paged_decode_weights(q, kp, vp, table, i32(lens), 0.125, w, max_context=40,
                             row_ids=i32([1, 4, 0, 1 << 30]))
    assert pkv.read_device_status() == 5                     # rows past the array
    assert bool((w[2] == 1).all()) and bool((w[3] == 1).all()) and float(w[0, 0, 0]) > 1
    w.fill_(1)
    out = pkv.paged_decode_weights(q, kp, vp, table, i32([0, 40, -3, 40]), 0.125, w,
                                   max_context=40)
    assert pkv.read_device_status() == 1
    assert bool((w[0] == 1).all()) and bool((w[2] == 1).all()) and bool((out[0] == 0).all())
    assert bool((w[1, :, :40] > 1).all())
    # a length beyond the table is clamped to it and reported, the weights to their row
    w.fill_(1)
    short = w[:, :, :40].contiguous()
    pkv.paged_decode_weights(q, kp, vp, table, i32([40, 1 << 20, 40, 40]), 0.125, short,
                             max_context=40)
    assert pkv.read_device_status() == 5
    with pytest.raises(pkv.PkvError):
        pkv.paged_decode_weights(q, kp, vp, table, i32(lens), 0.125, w[:, :, :39].contiguous(),
                                 max_context=40)
    with pytest.raises(ValueError):
        pkv.paged_decode_weights(q, kp, vp, table, i32(lens), 0.125, w[:, :1].contiguous(),
                                 max_context=40)
    with pytest.raises(TypeError):
        pkv.paged_decode_weights(q, kp, vp, table, i32(lens), 0.125, w.double(), max_context=40)
    with pytest.raises(pkv.PkvError):
        pkv.paged_decode_weights(q, kp, vp, table, i32(lens), 0.125, w, max_context=40,
                                 workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_decode_weights_many_sequences(pkv):
    """Enough sequences that the finishing launch works through several tiles per CTA, and a
    partition far longer than the context: a few sequences against the 64-bit sums, all of them
    against one another (each head's weights add up to the group)."""
    g = gen(44)
    S, hkv, group, d = 64, 8, 1, 64
    lens = torch.randint(700, 2049, (S,), generator=torch.Generator().manual_seed(1)).tolist()
    lens[5] = 2048
    kp, vp, table = paged(lens, hkv, 16, d, torch.bfloat16, g)
    q = torch.randn(S, hkv * group, d, generator=g, device="cuda").bfloat16()
    w = torch.full((S, hkv, 2048), float("nan"), device="cuda")
    for pb in (0, 1 << 20):
        out = pkv.paged_decode_weights(q, kp, vp, table, i32(lens), 0.125, w, max_context=2048,
                                       decay=0.0, partition_blocks=pb)
        assert pkv.read_device_status() == 0
        assert torch.equal(out, pkv.paged_decode(q, kp, vp, table, i32(lens), 0.125,
                                                 max_context=2048,
                                                 partition_blocks=min(pb, 128)))
        kc, tc = kp.cpu(), table.cpu()
        for i in range(S):
            n = lens[i]
            got = w[i, :, :n].cpu().double()
            assert float((got.sum(-1) - group).abs().max()) < 1e-4
            assert bool(torch.isnan(w[i, :, n:]).all())
            if i % 16 == 5:
                k = tokens(kc, tc[i], n)
                _, p, size = attention(q[i:i + 1].cpu(), k, None, 0.125, first=n - 1)
                assert bool(((got - p).abs() <= weight_bound(p, p * 0, size, d, n + group)).all())


def test_decode_weights_growing_scores(pkv):
    """Scores that grow along the context, so that every partition's maximum differs and early
    tokens' weights underflow: nothing is lost where it counts, nothing is NaN."""
    n, d = 1200, 128
    g = gen(9)
    kp, vp, table = paged([n], 1, 16, d, torch.bfloat16, g)
    q = torch.zeros(1, 4, d, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = torch.tensor([1.0, -1.0, 0.5, 0.0], device="cuda").bfloat16()
    ramp = (torch.arange(n, device="cuda") // 8).float().bfloat16()
    flat = kp[table[0, :75].long()].transpose(1, 2).reshape(-1, d).clone()
    flat[:n, 0] = ramp
    kp[table[0, :75].long()] = flat.view(75, 16, 1, d).transpose(1, 2)
    w = torch.zeros(1, 1, n, device="cuda")
    pkv.paged_decode_weights(q, kp, vp, table, i32([n]), 1.0, w, max_context=n, partition_blocks=4)
    assert pkv.read_device_status() == 0
    k = tokens(kp.cpu(), table.cpu()[0], n)
    _, p, _ = attention(q.cpu(), k, None, 1.0, first=n - 1)
    # scores are whole or half numbers below 2^8 from one product: exact; what is left is the
    # rounding of score * log2(e) (twice 2^-24 of 2^8), exp2 and the sums
    err = (w[0].cpu().double() - p).abs()
    assert bool((err <= p * 2.0 ** -14 + 1e-37).all())


PREFILL = [  # cached, new, hkv, group, d, bs, dtype, window
    ([0], [1], 1, 1, 64, 16, torch.float32, 0),
    ([0, 5, 31], [3, 70, 1], 2, 2, 64, 16, torch.float32, 0),
    ([200, 0], [33, 130], 1, 4, 128, 32, torch.float32, 10),
    ([0], [1], 1, 1, 64, 16, torch.bfloat16, 0),
    ([0, 63, 64, 65], [64, 65, 1, 129], 2, 1, 64, 16, torch.bfloat16, 0),
    ([127, 128, 0, 1000], [5, 128, 127, 40], 2, 4, 128, 16, torch.bfloat16, 0),
    ([127, 128, 0, 1000], [5, 128, 127, 40], 2, 4, 128, 32, torch.bfloat16, 32),
    ([300, 17], [200, 90], 1, 8, 128, 16, torch.bfloat16, 64),
    ([300, 17], [200, 90], 3, 8, 64, 32, torch.bfloat16, 1),
    ([2500, 4000], [20, 3], 1, 2, 128, 16, torch.bfloat16, 0),
    ([2500], [260], 2, 8, 64, 16, torch.bfloat16, 128),
    # few key tiles and many rows: the rows of a key tile are split over CTAs
    ([100], [512], 1, 8, 64, 16, torch.bfloat16, 0),
    ([0, 400, 3], [450, 130, 0], 1, 8, 128, 32, torch.bfloat16, 0),
    ([2000], [500], 1, 4, 128, 16, torch.bfloat16, 0),
    ([40, 0], [300, 7], 1, 8, 128, 16, torch.float32, 0),
    ([700], [257], 1, 8, 64, 32, torch.float32, 200),
]


@pytest.mark.parametrize("case", PREFILL)
def test_prefill_weights(pkv, case):
    cached, new, hkv, group, d, bs, dtype, window = case
    g = gen(sum(cached) + sum(new))
    R, hq = len(new), hkv * group
    total = [c + n for c, n in zip(cached, new)]
    kp, _, table = paged(total, hkv, bs, d, dtype, g)
    q = torch.randn(sum(new), hq, d, generator=g, device="cuda").to(dtype)
    off = [sum(new[:i]) for i in range(R + 1)]
    W = max(total) + 1
    w0 = torch.rand(R + 1, hkv, W, generator=g, device="cuda")
    ids = torch.randperm(R + 1, generator=g, device="cuda")[:R].to(torch.int32)
    scale = d ** -0.5

    def call(w, decay):
        return pkv.paged_prefill_weights(q, kp, table, i32(cached), i32(new), i32(off), scale, w,
                                         max_new=max(new), max_context=max(total), window=window,
                                         row_ids=ids, decay=decay)

    w = w0.clone()
    assert call(w, 0.5) is w
    assert pkv.read_device_status() == 0
    kc, tc, qc = kp.cpu(), table.cpu(), q.cpu()
    for i, n in enumerate(total):
        m = min(new[i], window) if window else new[i]
        k = tokens(kc, tc[i], n)
        _, p, size = attention(qc[off[i + 1] - m:off[i + 1]], k, None, scale, first=n - m)
        row = int(ids[i])
        before = w0[row, :, :n].cpu().double()
        if m == 0:   # no new tokens: left alone
            assert torch.equal(w[row], w0[row])
            continue
        err = (w[row, :, :n].cpu().double() - (0.5 * before + p)).abs()
        bound = weight_bound(p, before, size, d, n + m * group)
        assert bool((err <= bound).all()), ((err - bound).max(), i)
        assert torch.equal(w[row, :, n:], w0[row, :, n:])
    rest = [r for r in range(R + 1) if r not in ids.tolist()]
    assert torch.equal(w[rest], w0[rest])
    again = w0.clone()
    call(again, 0.5)
    assert torch.equal(again, w)
    nans = torch.full_like(w0, float("nan"))
    call(nans, 0.0)
    for i, n in enumerate(total):
        assert bool(torch.isfinite(nans[int(ids[i]), :, :n]).all()) == (new[i] > 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_weights_growing_scores(pkv, dtype):
    """Scores that grow far beyond a row's first tile (2^96 and more above it), then fall: the
    sums are taken again from a larger reference, and nothing is lost where it counts."""
    n, d = 900, 64
    g = gen(19)
    kp, _, table = paged([n], 1, 16, d, dtype, g)
    ids = table[0, :57].long()
    flat = kp[ids].transpose(1, 2).reshape(-1, d).clone()
    flat[:n] = 0
    j = torch.arange(n, device="cuda")
    flat[:n, 0] = torch.where(j < 600, j // 4, 150 - (j - 600) // 4).to(dtype)   # 0 .. 150 .. 75
    kp[ids] = flat.view(57, 16, 1, d).transpose(1, 2)
    q = torch.zeros(40, 4, d, device="cuda", dtype=dtype)
    q[..., 0] = torch.tensor([1.0, -1.0, 0.5, 2.0], device="cuda").to(dtype)
    w = torch.zeros(1, 1, n, device="cuda")
    pkv.paged_prefill_weights(q, kp, table, i32([n - 40]), i32([40]), i32([0, 40]), 1.0, w,
                              max_new=40, max_context=n)
    assert pkv.read_device_status() == 0
    k = tokens(kp.cpu(), table.cpu()[0], n)
    _, p, _ = attention(q.cpu(), k, None, 1.0, first=n - 40)
    # scores are whole or half numbers up to 300 < 2^9, exact; times log2(e) and less the row's
    # statistic, up to 2^9 each, they round by 2^-24 of that thrice: below 2^-13 of a weight; the
    # exponentials and sums of 40 x 4 + 900 terms stay below 2^-13 too
    err = (w[0].cpu().double() - p).abs()
    assert bool((err <= p * 2.0 ** -12 + 160 * 2.0 ** -120).all()), (err / p.clamp(min=1e-30)).max()


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_weights_odd_and_even_row_tiles(pkv, d):
    """Requests of one and of three row tiles in turn, many items to a CTA: half of the consumers
    sit some items out."""
    g = gen(47)
    R, hkv, group = 24, 4, 4
    new = [(7, 90, 30, 5, 70, 96)[i % 6] for i in range(R)]
    cached = [(911 * i) % 1300 + 200 * (i % 2) for i in range(R)]
    total = [c + n for c, n in zip(cached, new)]
    kp, _, table = paged(total, hkv, 16, d, torch.bfloat16, g)
    q = torch.randn(sum(new), hkv * group, d, generator=g, device="cuda").bfloat16()
    off = [sum(new[:i]) for i in range(R + 1)]

    def call():
        w = torch.zeros(R, hkv, max(total), device="cuda")
        return pkv.paged_prefill_weights(q, kp, table, i32(cached), i32(new), i32(off), d ** -0.5, w,
                                         max_new=max(new), max_context=max(total))

    w = call()
    assert pkv.read_device_status() == 0
    for _ in range(20):
        assert torch.equal(call(), w)
    kc, tc, qc, wc = kp.cpu(), table.cpu(), q.cpu(), w.cpu().double()
    for i, n in enumerate(total):
        k = tokens(kc, tc[i], n)
        _, p, size = attention(qc[off[i]:off[i + 1]], k, None, d ** -0.5, first=cached[i])
        err = (wc[i, :, :n] - p).abs()
        assert bool((err <= weight_bound(p, p * 0, size, d, n + new[i] * group)).all()), i


@pytest.mark.parametrize("max_new,max_context", [(1024, 4096),     # a launch per kv head
                                                 (16384, 4096)])   # scores computed twice
@pytest.mark.parametrize("window", [0, 50])
def test_prefill_weights_wide_bounds(pkv, max_new, max_context, window):
    """Bounds far above the lengths: what the call keeps goes by the bounds (fp32)."""
    hkv, group, d, bs = 2, 8, 64, 16
    cached, new = [70, 0, 300], [130, 9, 40]
    total = [c + n for c, n in zip(cached, new)]
    g = gen(43)
    kp, _, table = paged(total, hkv, bs, d, torch.float32, g)
    wide = torch.full((3, max_context // bs), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = torch.randn(sum(new), hkv * group, d, generator=g, device="cuda")
    off = [0, 130, 139, 179]
    if window:   # the window counts for the bound on rows, unless it is above it
        max_new = 2 * max_new
    w0 = torch.rand(3, hkv, max_context, generator=g, device="cuda")
    w = w0.clone()
    need = pkv.prefill_weights_workspace_bytes(kp, 3, hkv * group, max_new, max_context, window)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ws.view(torch.float32).fill_(float("nan"))   # whatever was there does not count
    pkv.paged_prefill_weights(q, kp, wide, i32(cached), i32(new), i32(off), 0.125, w,
                              max_new=max_new, max_context=max_context, window=window,
                              decay=0.5, workspace=ws)
    assert pkv.read_device_status() == 0
    for i, n in enumerate(total):
        m = min(new[i], window) if window else new[i]
        k = tokens(kp.cpu(), table.cpu()[i], n)
        _, p, size = attention(q.cpu()[off[i + 1] - m:off[i + 1]], k, None, 0.125, first=n - m)
        before = w0[i, :, :n].cpu().double()
        err = (w[i, :, :n].cpu().double() - (0.5 * before + p)).abs()
        assert bool((err <= weight_bound(p, before, size, d, n + m * group)).all()), i
        assert torch.equal(w[i, :, n:], w0[i, :, n:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_weights_infinite_keys(pkv, dtype):
    """Keys whose score is -inf, more of them than a row's first tiles hold, before keys whose
    scores are far below zero: a softmax over the latter alone."""
    n, d = 700, 64
    g = gen(37)
    kp, _, table = paged([n], 1, 16, d, dtype, g)
    ids = table[0, :44].long()
    flat = kp[ids].transpose(1, 2).reshape(-1, d).clone()
    flat[:n] = 0
    j = torch.arange(n, device="cuda")
    flat[:n, 0] = torch.where(j < 300, float("-inf"), -500.0 - (j % 4)).to(dtype)
    kp[ids] = flat.view(44, 16, 1, d).transpose(1, 2)
    q = torch.zeros(40, 2, d, device="cuda", dtype=dtype)
    q[..., 0] = torch.tensor([1.0, 0.5], device="cuda").to(dtype)
    q[..., 1] = 1.0
    w = torch.zeros(1, 1, n, device="cuda")
    pkv.paged_prefill_weights(q, kp, table, i32([n - 40]), i32([40]), i32([0, 40]), 1.0, w,
                              max_new=40, max_context=n)
    assert pkv.read_device_status() == 0
    x = kp.cpu()[ids.cpu()].transpose(1, 2).reshape(-1, d)[:n, 0].double()
    want = torch.zeros(n, dtype=torch.float64)
    for i in range(40):
        for f in (1.0, 0.5):
            want[:n - 39 + i] += torch.softmax(x[:n - 39 + i] * f, 0)
    got = w[0, 0].cpu().double()
    assert bool((got[:300] == 0).all())
    # scores are whole or half numbers below 2^9, exact; times log2(e) and less the row's statistic
    # they round by 2^-24 of 2^10 thrice at most: below 2^-12 of a weight; the exponentials and sums
    # of 80 + 700 terms stay below 2^-13
    assert bool(((got - want).abs() <= want * 2.0 ** -11).all()), ((got - want).abs() / want).max()


@pytest.mark.parametrize("rows", [False, True])
def test_prefill_weights_many_requests(pkv, rows):
    """More requests than one round of launches takes: 300 short ones, odd lengths."""
    g = gen(23)
    R, hkv, group, d = 300, 2, 2, 64
    cached = [(7 * i) % 150 for i in range(R)]
    new = [1 + (5 * i) % 9 for i in range(R)]
    new[17] = 0
    total = [c + n for c, n in zip(cached, new)]
    kp, _, table = paged(total, hkv, 16, d, torch.bfloat16, g)
    q = torch.randn(sum(new), hkv * group, d, generator=g, device="cuda").bfloat16()
    off = [sum(new[:i]) for i in range(R + 1)]
    ids = torch.randperm(R + 7, generator=g, device="cuda")[:R].to(torch.int32) if rows else None
    w = torch.zeros(R + 7 if rows else R, hkv, max(total), device="cuda")
    pkv.paged_prefill_weights(q, kp, table, i32(cached), i32(new), i32(off), 0.125, w, max_new=9,
                              max_context=max(total), row_ids=ids)
    assert pkv.read_device_status() == 0
    kc, tc, qc, wc = kp.cpu(), table.cpu(), q.cpu(), w.cpu().double()
    for i in range(R):
        row = int(ids[i]) if rows else i
        n = total[i]
        if new[i] == 0:
            assert bool((wc[row] == 0).all())
            continue
        k = tokens(kc, tc[i], n)
        _, p, size = attention(qc[off[i]:off[i + 1]], k, None, 0.125, first=cached[i])
        err = (wc[row, :, :n] - p).abs()
        assert bool((err <= weight_bound(p, p * 0, size, d, n + new[i] * group)).all()), i
        assert bool((wc[row, :, n:] == 0).all())


def test_two_streams_at_once(pkv):
    """Calls of both forms on two streams at the same time, each with its own workspace."""
    g = gen(29)
    lens, hkv, group, d = [900, 300, 1200], 2, 4, 128
    kp, vp, table = paged(lens, hkv, 16, d, torch.bfloat16, g)
    qs = torch.randn(2, 3, hkv * group, d, generator=g, device="cuda").bfloat16()
    qp = torch.randn(2, 90, hkv * group, d, generator=g, device="cuda").bfloat16()
    off, nl = i32([0, 40, 50, 90]), i32([40, 10, 40])
    cached, cl = i32([860, 290, 1160]), i32(lens)

    def run(i, w, stream=None):
        for _ in range(5):
            pkv.paged_prefill_weights(qp[i], kp, table, cached, nl, off, 0.09, w, max_new=40,
                                      max_context=1200, stream=stream)
            pkv.paged_decode_weights(qs[i], kp, vp, table, cl, 0.09, w, max_context=1200,
                                     stream=stream)

    want = [torch.zeros(3, hkv, 1200, device="cuda") for _ in range(2)]
    for i in range(2):
        run(i, want[i])
    got = [torch.zeros(3, hkv, 1200, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        run(i, got[i], streams[i])
    torch.cuda.synchronize()
    assert pkv.read_device_status() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_prefill_weights_of_one_token_are_the_decodes(pkv):
    """A chunk of one token attends as a decode step does."""
    g = gen(33)
    lens, hkv, group, d = [50, 700, 129], 2, 4, 128
    kp, vp, table = paged(lens, hkv, 16, d, torch.bfloat16, g)
    q = torch.randn(3, hkv * group, d, generator=g, device="cuda").bfloat16()
    a = torch.zeros(3, hkv, 704, device="cuda")
    b = torch.zeros_like(a)
    pkv.paged_decode_weights(q, kp, vp, table, i32(lens), d ** -0.5, a, max_context=700)
    pkv.paged_prefill_weights(q, kp, table, i32([n - 1 for n in lens]), i32([1, 1, 1]),
                              i32([0, 1, 2, 3]), d ** -0.5, b, max_new=1, max_context=700)
    assert pkv.read_device_status() == 0
    # scores of size below 16 whose products differ in order alone (see weight_bound)
    assert bool(((a - b).abs() <= a * (d + 8) * 2.0 ** -23 * 16 * 4).all())


def test_prefill_weights_skipped_requests(pkv):
    """No new tokens, padding rows, and lengths out of range: reported, and left alone."""
    g = gen(7)
    total = [40, 40, 40]
    kp, _, table = paged(total, 2, 16, 64, torch.bfloat16, g)
    q = torch.randn(30, 4, 64, generator=g, device="cuda").bfloat16()

    def call(cached, new, off, ids=None, max_new=10, mc=40):
        w = torch.ones(3, 2, 40, device="cuda")
        pkv.paged_prefill_weights(q, kp, table, i32(cached), i32(new), i32(off), 0.125, w,
                                  max_new=max_new, max_context=mc, row_ids=ids)
        return pkv.read_device_status(), [bool((w[i] == 1).all()) for i in range(3)]

    ok = [0, 10, 20, 30]
    assert call([30, 30, 30], [10, 0, 10], [0, 10, 10, 20]) == (0, [False, True, False])
    assert call([30, 30, 30], [10] * 3, ok, i32([-1, 0, 2])) == (0, [False, True, False])
    assert call([30, 30, 30], [10] * 3, ok, i32([1, 3, 0])) == (5, [False, False, True])
    assert call([30, -1, 30], [10] * 3, ok) == (5, [False, True, False])
    assert call([30, 31, 30], [10] * 3, ok) == (5, [False, True, False])
    assert call([30, 29, 30], [10, 11, 10], ok) == (5, [False, True, False])
    assert call([30, 30, 30], [10] * 3, [0, 10, 21, 30]) == (5, [False, False, True])
    assert call([30, 30, 30], [10] * 3, [-1, 10, 20, 30]) == (5, [True, False, False])
    table[1, 1] = 1 << 20                                    # a block outside the pool
    st, left = call([30, 30, 30], [10] * 3, ok)
    assert st == 5 and not left[0] and not left[2]


def test_weights_streams_and_capture(pkv):
    """Both forms on another stream, and captured into one graph and replayed."""
    g = gen(15)
    lens, new, hkv, group, d = [300, 45, 130], [20, 45, 7], 2, 4, 128
    kp, vp, table = paged(lens, hkv, 16, d, torch.bfloat16, g)
    q = torch.randn(sum(new), hkv * group, d, generator=g, device="cuda").bfloat16()
    q1 = torch.randn(3, hkv * group, d, generator=g, device="cuda").bfloat16()
    off = i32([0, 20, 65, 72])
    cached, nl, cl = i32([c - n for c, n in zip(lens, new)]), i32(new), i32(lens)

    def both(w, stream=None, out=None, ws=(None, None)):
        pkv.paged_prefill_weights(q, kp, table, cached, nl, off, 0.09, w, max_new=45,
                                  max_context=300, workspace=ws[0], stream=stream)
        return pkv.paged_decode_weights(q1, kp, vp, table, cl, 0.09, w, max_context=300, out=out,
                                        workspace=ws[1], stream=stream)

    w = torch.zeros(3, hkv, 301, device="cuda")
    want_out = both(w)
    want = w.clone()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        w.zero_()
        s.wait_stream(torch.cuda.current_stream())
        out = both(w, stream=stream)
        s.synchronize()
        assert torch.equal(w, want) and torch.equal(out, want_out)
    ws = tuple(torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
        pkv.prefill_weights_workspace_bytes(kp, 3, hkv * group, 45, 300),
        pkv.decode_weights_workspace_bytes(kp, 3, hkv * group, 300)))
    out = torch.empty_like(q1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both(w, out=out, ws=ws)
    torch.cuda.synchronize()
    for x in ws:
        x.fill_(255)                        # a replay needs nothing from the workspace
    w.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, want) and torch.equal(out, want_out)
    graph.replay()                          # accumulates
    torch.cuda.synchronize()
    assert bool((w[0, :, :300] > want[0, :, :300]).all())
    assert pkv.read_device_status() == 0


def test_decode_weights_after_a_timeout(pkv, monkeypatch):
    """A pipeline wait that runs out is reported, and the next call is right."""
    g = gen(2)
    kp, vp, table = paged([200, 90], 2, 16, 128, torch.bfloat16, g)
    q = torch.randn(2, 8, 128, generator=g, device="cuda").bfloat16()
    w = torch.zeros(2, 2, 200, device="cuda")
    want = torch.zeros_like(w)
    args = (q, kp, vp, table, i32([200, 90]), 0.09)
    pkv.paged_decode_weights(*args, want, max_context=200)
    monkeypatch.setenv("PKV_TEST_DECODE_STALL", "1")
    pkv.paged_decode_weights(*args, torch.zeros_like(w), max_context=200)
    assert pkv.read_device_status() == 4
    monkeypatch.delenv("PKV_TEST_DECODE_STALL")
    assert os.environ.get("PKV_TEST_DECODE_STALL") is None
    pkv.paged_decode_weights(*args, w, max_context=200)
    assert pkv.read_device_status() == 0
    assert torch.equal(w, want)
