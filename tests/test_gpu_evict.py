"""Eviction by accumulated weight against its definition, entry by entry; the run of a
shrinking sequence (rotary append, prefill with weights, evict, decode with weights, evict
again) against 64-bit attention over the kept tokens."""
import pytest
import torch

from tests.helpers import check_attention
from tests.shrink_refs import attention, evict_rows, rotate, weight_bound

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def setup(lens, hkv, bs, d, dtype, seed):
    """Pools whose rows all differ, bit patterns included, and a scattered table."""
    g = gen(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 3
    perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    kp = torch.randn(nb, hkv, bs, d, generator=g, device="cuda").to(dtype)
    vp = torch.randn(nb, hkv, bs, d, generator=g, device="cuda").to(dtype)
    return kp, vp, table, g


def expect(kp, vp, table, lens, budgets, w, pos, sinks, recent, seen, tracked, rows):
    """What an eviction leaves (CPU): pools, weights, positions, lengths."""
    kp, vp, w, pos, table = (t.cpu().clone() for t in (kp, vp, w, pos, table))
    bs = kp.shape[2]
    w0, pos0, k0, v0 = w.clone(), pos.clone(), kp.clone(), vp.clone()
    left = []
    for i, L in enumerate(lens):
        b = budgets[i]
        if rows[i] < 0:
            left.append(L)
            continue
        left.append(L if b < 0 else min(L, b))
        for h in range(w.shape[1]):
            src, ww, pp = evict_rows(w0[rows[i], h], pos0[rows[i], h], tracked[i], seen[i], L, b,
                                     sinks, recent)
            pos[rows[i], h, :len(pp)] = torch.tensor(pp, dtype=torch.int32)
            if src is None:
                continue
            w[rows[i], h, :b] = torch.tensor(ww)
            w[rows[i], h, b:L] = 0
            for to, fr in enumerate(src):
                if to != fr:
                    t, f = int(table[i, to // bs]), int(table[i, fr // bs])
                    kp[t, h, to % bs] = k0[f, h, fr % bs]
                    vp[t, h, to % bs] = v0[f, h, fr % bs]
    return kp, vp, w, pos, left


def bits(t):
    return t.cpu().contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


def same_positions(got, want, rows, left):
    """positions_out holds left[i] entries per head; the rest is not specified in place."""
    return all(torch.equal(got[r, :, :n].cpu(), want[r, :, :n]) for r, n in zip(rows, left)
               if r >= 0)


CASES = [  # lens, budgets, hkv, bs, d, dtype, sinks, recent
    ([1], [0], 1, 16, 64, torch.float32, 0, 0),
    ([1, 2, 3], [1, 1, 1], 2, 16, 64, torch.bfloat16, 0, 0),
    ([40, 17, 5, 0], [16, 16, 16, 16], 3, 16, 64, torch.bfloat16, 2, 4),
    ([40, 17, 5, 9], [-1, 0, 100, 9], 2, 32, 128, torch.float32, 1, 3),
    ([100], [10], 1, 16, 128, torch.bfloat16, 20, 0),        # more protected than the budget
    ([100], [10], 2, 32, 64, torch.bfloat16, 4, 30),
    ([100], [33], 2, 16, 64, torch.bfloat16, 0, 0),
    ([1025, 1024, 1023, 2049], [512, 1023, 1, 1500], 2, 16, 64, torch.bfloat16, 4, 64),
    ([3000], [2999], 1, 16, 128, torch.bfloat16, 0, 128),
    ([5000, 130], [700, 128], 1, 32, 64, torch.float32, 1, 100),
    ([20000], [1000], 1, 16, 64, torch.bfloat16, 4, 256),
    ([5000, 3000], [50, 2999], 1, 16, 64, torch.bfloat16, 60, 10),   # protected ones compete
    ([9000], [0], 1, 16, 64, torch.bfloat16, 4, 4),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["spread", "ties", "zeros", "odd"])
def test_evict(pkv, case, in_place, kind):
    lens, budgets, hkv, bs, d, dtype, sinks, recent = case
    kp, vp, table, g = setup(lens, hkv, bs, d, dtype, sum(lens) + hkv)
    S, W = len(lens), max(lens) + 5
    w = torch.rand(S + 1, hkv, W, generator=g, device="cuda")
    if kind == "ties":
        w = (w * 4).floor() / 4
    elif kind == "zeros":
        w.zero_()
    elif kind == "odd":   # every kind of float, signed zeros and NaN among them
        some = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), -1.0, 1e-42,
                             -1e-42, 3e38, 1.0], device="cuda")
        pick = torch.randint(0, 20, w.shape, generator=g, device="cuda")
        w = torch.where(pick < 10, some[pick.clamp(max=9)], w - 0.5)
    tracked = [min(n, (7 * i) % (n + 1)) for i, n in enumerate(lens)]
    seen = [n + 11 * i for i, n in enumerate(lens)]
    pos = torch.randint(0, max(seen) + 1, w.shape, generator=g, device="cuda", dtype=torch.int32)
    order = torch.randperm(S + 1, generator=g, device="cuda")
    rows = order[:S].tolist()
    want = expect(kp, vp, table, lens, budgets, w, pos, sinks, recent, seen, tracked, rows)
    wo = w.clone() if in_place else torch.full_like(w, 5.0)
    po = pos.clone() if in_place else torch.full_like(pos, -9)
    left = pkv.evict(kp, vp, table, i32(lens), i32(budgets), wo if in_place else w,
                     po if in_place else pos, max_context=max(lens), sinks=sinks, recent=recent,
                     seen_lens=i32(seen), tracked_lens=i32(tracked), row_ids=i32(rows),
                     weights_out=wo, positions_out=po)
    assert pkv.read_device_status() == 0
    assert left.tolist() == want[4]
    assert torch.equal(bits(kp), bits(want[0])) and torch.equal(bits(vp), bits(want[1]))
    for i, n in enumerate(lens):
        assert torch.equal(bits(wo[rows[i], :, :n]), bits(want[2][rows[i], :, :n]))
        past = wo[rows[i], :, n:]
        assert torch.equal(bits(past), bits(w[rows[i], :, n:])) if in_place else bool(
            (past == 5).all())
        if not in_place:
            assert bool((po[rows[i], :, want[4][i]:] == -9).all())
    assert same_positions(po, want[3], rows, want[4])
    other = int(order[S])
    assert torch.equal(bits(wo[other]), bits(w[other])) if in_place else bool(
        (wo[other] == 5).all())


@pytest.mark.parametrize("kind", ["spread", "zeros"])
def test_evict_many_rows(pkv, kind):
    """Enough rows that each is one CTA's, over more entries than it lists."""
    lens = [2100 - 37 * i for i in range(40)]
    budgets = [300 + 40 * (i % 7) for i in range(40)]
    kp, vp, table, g = setup(lens, 8, 16, 64, torch.bfloat16, 6)
    w = torch.rand(40, 8, 2100, generator=g, device="cuda")
    if kind == "zeros":
        w = torch.where(w < 0.9, torch.zeros_like(w), w)
    pos = torch.zeros(40, 8, 2100, dtype=torch.int32, device="cuda")
    want = expect(kp, vp, table, lens, budgets, w, pos, 4, 64, lens, [0] * 40, list(range(40)))
    left = pkv.evict(kp, vp, table, i32(lens), i32(budgets), w, pos, max_context=2100, sinks=4,
                     recent=64)
    assert pkv.read_device_status() == 0 and left.tolist() == want[4]
    assert torch.equal(w.cpu(), want[2]) and same_positions(pos, want[3], range(40), want[4])
    assert torch.equal(bits(kp), bits(want[0])) and torch.equal(bits(vp), bits(want[1]))


def test_evict_long_row(pkv):
    """A context past eight slices of 16384 entries, and one of the largest the call takes."""
    lens = [140001]
    kp, vp, table, g = setup(lens, 1, 32, 64, torch.bfloat16, 12)
    w = torch.exp(2 * torch.randn(1, 1, 140001, generator=g, device="cuda"))
    pos = torch.zeros(1, 1, 140001, dtype=torch.int32, device="cuda")
    want = expect(kp, vp, table, lens, [9000], w, pos, 4, 1000, lens, [0], [0])
    left = pkv.evict(kp, vp, table, i32(lens), i32([9000]), w, pos, max_context=140001, sinks=4,
                     recent=1000)
    assert pkv.read_device_status() == 0 and left.tolist() == [9000]
    assert torch.equal(w.cpu(), want[2]) and same_positions(pos, want[3], [0], [9000])
    assert torch.equal(bits(kp), bits(want[0])) and torch.equal(bits(vp), bits(want[1]))

    n = 1 << 20
    kp, vp, table, g = setup([n], 1, 32, 64, torch.bfloat16, 13)
    w = torch.rand(1, 1, n, generator=g, device="cuda")
    w0, k0 = w.clone(), kp.clone()
    pos = torch.zeros(1, 1, n, dtype=torch.int32, device="cuda")
    left = pkv.evict(kp, vp, table, i32([n]), i32([100000]), w, pos, max_context=n)
    assert pkv.read_device_status() == 0 and left.tolist() == [100000]
    order = torch.sort(w0[0, 0], descending=True, stable=True).indices[:100000]
    kept = pos[0, 0, :100000].long()
    assert torch.equal(kept.sort().values, order.sort().values)
    assert torch.equal(w[0, 0, :100000], w0[0, 0][kept])
    assert bool((w[0, 0, 100000:] == 0).all())
    at = torch.arange(100000, device="cuda")
    rows = kp[table[0].long()[at // 32], 0, at % 32]
    src = k0[table[0].long()[kept // 32], 0, kept % 32]
    assert torch.equal(rows, src)


def test_two_evictions_at_once(pkv):
    """Different sequences of one pool on two streams at the same time."""
    lens = [700, 800]
    kp, vp, table, g = setup(lens, 2, 16, 64, torch.bfloat16, 15)
    w = torch.rand(2, 2, 800, generator=g, device="cuda")
    pos = torch.zeros(2, 2, 800, dtype=torch.int32, device="cuda")
    want = expect(kp, vp, table, lens, [200, 300], w, pos, 2, 20, lens, [0, 0], [0, 1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    cl, b = i32(lens), i32([200, 300])
    ids = i32([0, 1])
    torch.cuda.synchronize()
    left = [pkv.evict(kp, vp, table[i:i + 1], cl[i:i + 1], b[i:i + 1], w, pos, max_context=800,
                      sinks=2, recent=20, row_ids=ids[i:i + 1], stream=streams[i])
            for i in range(2)]
    torch.cuda.synchronize()
    assert pkv.read_device_status() == 0
    assert [int(x) for x in left] == [200, 300]
    assert torch.equal(w.cpu(), want[2]) and same_positions(pos, want[3], [0, 1], [200, 300])
    assert torch.equal(bits(kp), bits(want[0])) and torch.equal(bits(vp), bits(want[1]))


def test_defaults_and_padding(pkv):
    """No row_ids, seen or tracked lengths; padding rows; out-of-range lengths and rows."""
    lens = [50, 60, 70]
    kp, vp, table, g = setup(lens, 2, 16, 64, torch.bfloat16, 1)
    w = torch.rand(3, 2, 80, generator=g, device="cuda")
    pos = torch.full((3, 2, 80), 123456, dtype=torch.int32, device="cuda")   # not read
    keep = [t.clone() for t in (kp, vp, w, pos)]
    want = expect(kp, vp, table, lens, [20] * 3, w, pos, 2, 8, lens, [0] * 3, [0, 1, 2])
    left = pkv.evict(kp, vp, table, i32(lens), i32([20] * 3), w, pos, max_context=70, sinks=2,
                     recent=8)
    assert pkv.read_device_status() == 0
    assert left.tolist() == [20] * 3 and torch.equal(bits(kp), bits(want[0]))
    assert torch.equal(w.cpu(), want[2]) and same_positions(pos, want[3], [0, 1, 2], [20] * 3)

    kp, vp, w, pos = (t.clone() for t in keep)
    left = pkv.evict(kp, vp, table, i32(lens), i32([20] * 3), w, pos, max_context=70,
                     row_ids=i32([-1, -5, -1]))
    assert pkv.read_device_status() == 0 and left.tolist() == lens
    for a, b in zip((kp, vp, w, pos), keep):
        assert torch.equal(a, b)
    left = pkv.evict(kp, vp, table, i32([-2, 1000, 0]), i32([20] * 3), w, pos, max_context=70)
    assert pkv.read_device_status() in (1, 5) and left.tolist() == [0, 1000, 0]
    left = pkv.evict(kp, vp, table, i32(lens), i32([20] * 3), w, pos, max_context=70,
                     row_ids=i32([3, 1 << 30, -1]))
    assert pkv.read_device_status() == 5 and left.tolist() == lens
    for a, b in zip((kp, vp, w, pos), keep):
        assert torch.equal(a, b)


def test_bad_block_skips_its_rows(pkv):
    lens = [64]
    kp, vp, table, g = setup(lens, 1, 16, 64, torch.bfloat16, 8)
    w = torch.arange(64, device="cuda").float().view(1, 1, 64).contiguous()   # the last 32 stay
    pos = torch.zeros(1, 1, 64, dtype=torch.int32, device="cuda")
    k0, t0 = kp.clone(), table.clone()
    table[0, 2] = 1 << 28                       # rows 32 .. 47, sources of places 0 .. 15
    left = pkv.evict(kp, vp, table, i32(lens), i32([32]), w, pos, max_context=64)
    assert pkv.read_device_status() == 5 and left.tolist() == [32]
    a, b, c = (int(t0[0, i]) for i in (0, 1, 3))
    assert torch.equal(kp[a], k0[a]) and torch.equal(kp[b], k0[c])


def test_refusals(pkv):
    kp, vp, table, g = setup([30], 2, 16, 64, torch.bfloat16, 2)
    w = torch.rand(1, 2, 32, device="cuda")
    pos = torch.zeros(1, 2, 32, dtype=torch.int32, device="cuda")
    cl, b = i32([30]), i32([8])
    with pytest.raises(pkv.PkvError):
        pkv.evict(kp, vp, table, cl, b, w, pos, max_context=30, new_lens=cl)
    with pytest.raises(pkv.PkvError):
        pkv.evict(kp, vp, table, cl, b, w, pos, max_context=33)
    with pytest.raises(pkv.PkvError):
        pkv.evict(kp, vp, table, cl, b, w, pos, max_context=30, sinks=-1)
    with pytest.raises(pkv.PkvError):
        pkv.evict(kp, vp, table, cl, b, w, pos, max_context=30,
                  workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        pkv.evict(kp, vp, table, cl, b, w, pos.float(), max_context=30)
    with pytest.raises(ValueError):
        pkv.evict(kp, vp, table, cl, b, w, pos[:, :, :31].contiguous(), max_context=30)
    with pytest.raises(ValueError):
        pkv.evict(kp, vp, table.cpu(), cl, b, w, pos, max_context=30)


def test_streams_and_capture(pkv):
    """On another stream, and captured: a replay works on the state as it then is."""
    lens, budget = [900, 300, 1030], [256, 256, 256]
    kp, vp, table, g = setup(lens, 2, 16, 128, torch.bfloat16, 5)
    w = torch.rand(3, 2, 1040, generator=g, device="cuda")
    pos = torch.zeros(3, 2, 1040, dtype=torch.int32, device="cuda")
    start = [t.clone() for t in (kp, vp, w, pos)]
    cl, b = i32(lens), i32(budget)

    def back():
        for t, s in zip((kp, vp, w, pos), start):
            t.copy_(s)

    def call(**kw):
        return pkv.evict(kp, vp, table, cl, b, w, pos, max_context=1030, sinks=4, recent=32, **kw)

    left = call()
    want = [t.clone() for t in (kp, vp, w, pos)]
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        back()
        s.wait_stream(torch.cuda.current_stream())
        got = call(stream=stream)
        s.synchronize()
        assert torch.equal(got, left)
        assert all(torch.equal(a, c) for a, c in zip((kp, vp, w, pos), want))
    back()
    ws = torch.empty(pkv.evict_workspace_bytes(kp, 3, 1030), dtype=torch.uint8, device="cuda")
    out = torch.zeros(3, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        call(workspace=ws, new_lens=out)
    torch.cuda.synchronize()
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, left)
    assert all(torch.equal(a, c) for a, c in zip((kp, vp, w, pos), want))
    assert pkv.read_device_status() == 0


@pytest.mark.parametrize("dtype,hkv,group,d,bs", [(torch.bfloat16, 2, 4, 128, 16),
                                                  (torch.float32, 2, 1, 64, 32)])
def test_shrinking_sequences(pkv, dtype, hkv, group, d, bs):
    """Two sequences, one forked from the other, as a serving loop runs them: prompts with
    rotary append, prefill and weights, an eviction, decode steps that append and accumulate,
    another eviction, more steps.  A mirror keeps each head's kept tokens in 64 bits."""
    g = gen(77)
    hq, scale, sinks, recent, budget = hkv * group, d ** -0.5, 2, 6, 40
    alloc = pkv.BlockAllocator(64, bs, seed=3)
    kp = torch.full((64, hkv, bs, d), float("nan"), device="cuda", dtype=dtype)
    vp = kp.clone()
    S, W, cols = 2, 160, 8
    weights = torch.zeros(S, hkv, W, device="cuda")
    positions = torch.zeros(S, hkv, W, dtype=torch.int32, device="cuda")
    f, _ = pkv.rope_frequencies(d, 10000.0)

    def draw(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    # the shared prompt of 50 tokens, then each sequence's own 33 and 20
    mirror = [[[] for _ in range(hkv)] for _ in range(S)]   # (position, k64, v64, weight)

    def prompt(seq, n, first):
        slots, cow = alloc.append(seq, n)
        if cow:
            pkv.copy_blocks(kp, vp, i32([cow]))
        q, k, v = draw(n, hq, d), draw(n, hkv, d), draw(n, hkv, d)
        pos = torch.arange(first, first + n, dtype=torch.int32, device="cuda")
        qr = pkv.rope_append(q, k, v, kp, vp, torch.tensor(slots, device="cuda"), pos, f)
        kr = pkv.rope(k, pos, f)
        assert float((kr.cpu().double() - rotate(k, pos, f)).abs().max()) < 0.05
        return qr, kr.cpu().double(), v.cpu().double()

    alloc.add_seq(0, 0)
    qr, kr, vr = prompt(0, 50, 0)
    alloc.fork(0, 1)
    own = [prompt(0, 33, 50), prompt(1, 20, 50)]
    lens = [83, 70]
    table = alloc.block_table([0, 1], cols).cuda()
    new = [33, 20]
    q = torch.cat([own[0][0], own[1][0]])
    out = pkv.paged_prefill(q, kp, vp, table, i32([50, 50]), i32(new), i32([0, 33, 53]), scale,
                            max_new=33)
    pkv.paged_prefill_weights(q, kp, table, i32([50, 50]), i32(new), i32([0, 33, 53]), scale,
                              weights, max_new=33, max_context=83)
    assert pkv.read_device_status() == 0
    at = 0
    for i in range(S):
        k = torch.cat([kr, own[i][1]])
        v = torch.cat([vr, own[i][2]])
        ref, p, size = attention(q[at:at + new[i]].cpu(), k, v, scale, first=50)
        check_attention(out[at:at + new[i]], ref.numpy())
        err = (weights[i, :, :lens[i]].cpu().double() - p).abs()
        assert bool((err <= weight_bound(p, p * 0, size, d, lens[i] + new[i] * group)).all())
        at += new[i]
        for h in range(hkv):
            mirror[i][h] = [(j, k[j, h], v[j, h], float(weights[i, h, j])) for j in range(lens[i])]

    seen, tracked = list(lens), [0, 0]

    def shrink():
        nonlocal tracked, table, lens
        for i in range(S):
            pairs = alloc.privatize(i, min(budget, lens[i]))
            if pairs:
                pkv.copy_blocks(kp, vp, i32(pairs))
        table = alloc.block_table([0, 1], cols).cuda()
        left = pkv.evict(kp, vp, table, i32(lens), i32([budget] * S), weights, positions,
                         max_context=max(lens), sinks=sinks, recent=recent, seen_lens=i32(seen),
                         tracked_lens=i32(tracked))
        assert pkv.read_device_status() == 0
        for i in range(S):
            for h in range(hkv):
                m = mirror[i][h]
                src, _, _ = evict_rows(torch.tensor([x[3] for x in m]), [x[0] for x in m],
                                       len(m), seen[i], lens[i], budget, sinks, recent)
                if src is not None:
                    mirror[i][h] = [m[j] for j in src]
                n = int(left[i])
                assert positions[i, h, :n].tolist() == [x[0] for x in mirror[i][h]]
                assert weights[i, h, :n].tolist() == [x[3] for x in mirror[i][h]]
                kept = {x[0] for x in mirror[i][h]}
                assert {0, 1} <= kept and set(range(seen[i] - recent, seen[i])) <= kept
            alloc.truncate(i, int(left[i]))
        lens = left.tolist()
        tracked = left.tolist()
        table = alloc.block_table([0, 1], cols).cuda()

    def step():
        nonlocal table, lens
        for i in range(S):
            _, cow = alloc.append(i, 1)
            if cow:
                pkv.copy_blocks(kp, vp, i32([cow]))
            lens[i] += 1
            seen[i] += 1
        table = alloc.block_table([0, 1], cols).cuda()
        q, k, v = draw(S, hq, d), draw(S, hkv, d), draw(S, hkv, d)
        pos = i32([n - 1 for n in seen])                    # the place in the text
        qr, kr = pkv.rope(q, pos, f), pkv.rope(k, pos, f)
        before = weights.cpu().double()
        out = pkv.paged_decode_weights(qr, kp, vp, table, i32(lens), scale, weights,
                                       max_context=max(lens), k_new=kr, v_new=v, decay=0.9)
        assert pkv.read_device_status() == 0
        refs = []
        for i in range(S):
            for h in range(hkv):
                mirror[i][h].append((seen[i] - 1, kr[i, h].cpu().double(),
                                     v[i, h].cpu().double(), 0.0))
                assert len(mirror[i][h]) == lens[i]
            kk = torch.stack([torch.stack([x[1] for x in mirror[i][h]]) for h in range(hkv)], 1)
            vv = torch.stack([torch.stack([x[2] for x in mirror[i][h]]) for h in range(hkv)], 1)
            ref, p, size = attention(qr[i:i + 1].cpu(), kk, vv, scale, first=lens[i] - 1)
            refs.append(ref)
            b = before[i, :, :lens[i]]
            err = (weights[i, :, :lens[i]].cpu().double() - (0.9 * b + p)).abs()
            assert bool((err <= weight_bound(p, b, size, d, lens[i] + group)).all())
            for h in range(hkv):
                mirror[i][h] = [(x[0], x[1], x[2], float(weights[i, h, j]))
                                for j, x in enumerate(mirror[i][h])]
        check_attention(out, torch.cat(refs).numpy())

    shrink()
    assert lens == [40, 40] and alloc.num_free == 64 - 2 * -(-40 // bs)
    for _ in range(7):
        step()
    shrink()
    for _ in range(20):
        step()
    shrink()
    assert lens == [40, 40]
    step()
