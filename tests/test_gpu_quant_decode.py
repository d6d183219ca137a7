"""Decode over a quantised cache, against 64-bit attention over the rows as held."""
import os

import pytest
import torch

from tests.quant_refs import decode_bound, held, kept

pytestmark = pytest.mark.gpu

INVALID, TIMEOUT, OOB, NOMEM = 1, 4, 5, 6


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_58_gb300 import build
    build.build()
    import paged_kv_cache_58_gb300 as m
    assert m.read_device_status() == 0
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def paged(pkv, lens, hkv, block, d, fmt, g, dtype=torch.bfloat16, extra=3, make=None):
    """A cache whose bytes outside the sequences are all ones (NaN codes and scales), its table,
    and the sequences' slots."""
    need = [-(-n // block) for n in lens]
    nb = sum(need) + extra
    c = pkv.QuantCache.empty(nb, hkv, d, block_size=block, format=fmt)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        t.fill_(0xFF)
    perm = torch.randperm(nb, generator=g, device="cuda")
    table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32, device="cuda")
    slots, at = [], 0
    for i, n in enumerate(lens):
        ids = perm[at:at + need[i]]
        at += need[i]
        table[i, :need[i]] = ids.int()
        t = torch.arange(n, device="cuda")
        slots.append(ids[t // block] * block + t % block if n else t)
        if n:
            k, v = (torch.randn(n, hkv, d, generator=g, device="cuda") for _ in range(2))
            if make:
                k, v = make(i, k, v)
            pkv.kv_append_quant(c, slots[-1], k.to(dtype), v.to(dtype))
    return c, table, slots


def reference(c, q, table, lens, scale, vals=None):
    """(outputs, bounds) [S, Hq, D] float64 on the CPU."""
    ks, vs = vals or (held(c.k, c.k_scales, c.format, False), held(c.v, c.v_scales, c.format, True))
    B, hkv = c.block_size, c.num_kv_heads
    outs, bounds = [], []
    for i, n in enumerate(lens):
        ids = table[i, :-(-n // B)].long().cpu()
        k, v = (x[ids].transpose(1, 2).reshape(-1, hkv, c.head_dim)[:n] for x in (ks, vs))
        qi = q[i].cpu().double()
        x = torch.einsum("hgd,nhd->hgn", qi.view(hkv, -1, c.head_dim), k) * scale
        p = torch.softmax(x, -1)
        ref = torch.einsum("hgn,nhd->hgd", p, v).reshape(qi.shape)
        outs.append(ref)
        bounds.append(decode_bound(qi, k, v, p, ref, scale, q.dtype))
    return torch.stack(outs), torch.stack(bounds)


def check(out, want):
    ref, bound = want
    off = (out.double().cpu() - ref).abs() - bound
    assert bool((off <= 0).all()), (float(off.max()), float(bound.max()))


SHAPES = [  # lens, hkv, group, d, block, partition_blocks
    ([1], 1, 1, 64, 16, 0),
    ([17, 33, 5, 64], 4, 1, 64, 16, 1),
    ([1, 2, 15, 16, 17, 31, 32, 33], 2, 2, 128, 32, 0),
    ([700, 1, 129], 3, 4, 128, 16, 0),
    ([300, 90, 257], 2, 8, 64, 32, 3),
    ([513, 512, 511, 1500], 8, 4, 128, 16, 8),
    ([2100, 64], 1, 8, 128, 16, 0),
]


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_decode(pkv, fmt, dtype, shape):
    lens, hkv, group, d, block, parts = SHAPES[shape]
    g = gen(10 + shape)
    c, table, _ = paged(pkv, lens, hkv, block, d, fmt, g)
    q = torch.randn(len(lens), hkv * group, d, generator=g, device="cuda").to(dtype)
    out = pkv.paged_decode_quant(q, c, table, i32(lens), d ** -0.5, max_context=max(lens),
                                 partition_blocks=parts)
    assert pkv.read_device_status() == 0
    check(out, reference(c, q, table, lens, d ** -0.5))


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_in_it(pkv, fmt, dtype, shape):
    """The fused append: the bytes and outputs of the append and then the decode."""
    lens, hkv, group, d, block, parts = SHAPES[shape]
    g = gen(20 + shape)
    c, table, slots = paged(pkv, lens, hkv, block, d, fmt, g)
    q = torch.randn(len(lens), hkv * group, d, generator=g, device="cuda").to(dtype)
    kn, vn = (torch.randn(len(lens), hkv, d, generator=g, device="cuda").to(dtype)
              for _ in range(2))
    vn[0] = 0
    two = pkv.QuantCache(*(t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales)), format=fmt)
    pkv.kv_append_quant(two, torch.stack([s[-1] for s in slots]), kn, vn)
    want = pkv.paged_decode_quant(q, two, table, i32(lens), d ** -0.5, max_context=max(lens),
                                  partition_blocks=parts)
    out = pkv.paged_decode_quant(q, c, table, i32(lens), d ** -0.5, max_context=max(lens),
                                 partition_blocks=parts, k_new=kn, v_new=vn)
    assert pkv.read_device_status() == 0
    assert torch.equal(out, want)
    for name in ("k", "v", "k_scales", "v_scales"):
        assert torch.equal(getattr(c, name), getattr(two, name)), name
    check(out, reference(c, q, table, lens, d ** -0.5))


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", ["growing", "sizes", "zeros", "rising", "falling", "ends"])
def test_rows_of_unequal_sizes(pkv, fmt, dtype, how):
    """Scores that grow token by token; V rows of any sizes; rows of zeros among them; sizes that
    rise and fall by a power of two a token; both ends of the exponents."""
    lens, hkv, group, d = [150, 700], 2, 4, 128
    g = gen(31)

    def make(i, k, v):
        n = len(k)
        e = torch.arange(n, device="cuda").float()
        if how == "growing":
            k = k * 0.05
            k[:, :, 0] += e[:, None] * 0.4
        elif how == "sizes":
            v = v * 2.0 ** torch.randint(-30, 30, (n, hkv, 1), generator=g, device="cuda").float()
        elif how == "zeros":
            v[::3] = 0
            v[:40] = 0
            v[100:] *= 2.0 ** 40
        elif how == "rising":
            v = v * 2.0 ** (e / n * 120 - 60)[:, None, None]
        elif how == "falling":
            v = v * 2.0 ** (60 - e / n * 120)[:, None, None]
        else:
            v = v * torch.where(e % 2 == 0, 2.0 ** -88, 2.0 ** 88)[:, None, None]
        return k, v

    c, table, _ = paged(pkv, lens, hkv, 16, d, fmt, g, torch.float32, make=make)
    q = torch.randn(2, hkv * group, d, generator=g, device="cuda")
    q[:, :, 0] = q[:, :, 0].abs() + 1
    q[1, 3] *= 1e-30
    q = q.to(dtype)
    for parts in (0, 2):
        out = pkv.paged_decode_quant(q, c, table, i32(lens), d ** -0.5, max_context=700,
                                     partition_blocks=parts)
        assert pkv.read_device_status() == 0
        check(out, reference(c, q, table, lens, d ** -0.5))


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_far_scales(pkv, fmt):
    """Queries and keys whose sizes are far apart, their products ordinary."""
    lens, hkv, d = [65], 2, 64
    g = gen(5)
    c, table, _ = paged(pkv, lens, hkv, 16, d, fmt, g, torch.float32,
                        make=lambda i, k, v: (k * 2.0 ** -70, v))
    q = torch.randn(1, hkv * 2, d, generator=g, device="cuda") * 2.0 ** 70
    out = pkv.paged_decode_quant(q, c, table, i32(lens), d ** -0.5, max_context=65)
    check(out, reference(c, q, table, lens, d ** -0.5))


def test_nan_rows_show(pkv):
    """A NaN in a token that is attended reaches the output; one past the length does not."""
    for fmt in ("fp8", "fp4"):
        c, table, slots = paged(pkv, [40, 40], 1, 16, 64, fmt, gen(1))
        x = torch.zeros(1, 1, 64, device="cuda", dtype=torch.bfloat16)
        bad = x.clone()
        bad[..., 3] = float("nan")
        pkv.kv_append_quant(c, slots[0][20:21].contiguous(), x, bad)
        q = torch.randn(2, 1, 64, generator=gen(2), device="cuda").bfloat16()
        out = pkv.paged_decode_quant(q, c, table, i32([40, 40]), 0.1, max_context=40)
        assert out[0].isnan().any() and not out[1].isnan().any()
        out = pkv.paged_decode_quant(q, c, table, i32([20, 40]), 0.1, max_context=40)
        assert not out.isnan().any()
        assert pkv.read_device_status() == 0


def test_lengths_and_ids_out_of_range(pkv):
    lens, hkv, d = [20, 20, 20], 2, 64
    c, table, _ = paged(pkv, lens, hkv, 16, d, "fp8", gen(3))
    q = torch.randn(3, 4, d, generator=gen(4), device="cuda").bfloat16()
    out = torch.full_like(q, 9.0)
    pkv.paged_decode_quant(q, c, table, i32([20, 0, 20]), 0.1, max_context=20, out=out)
    assert pkv.read_device_status() == INVALID
    assert not out[1].any()
    ok = pkv.paged_decode_quant(q, c, table, i32(lens), 0.1, max_context=20)
    assert torch.equal(out[0], ok[0]) and torch.equal(out[2], ok[2])
    before = [t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales)]
    kn = torch.ones(3, hkv, d, device="cuda", dtype=torch.bfloat16)
    pkv.paged_decode_quant(q[:1], c, table[:1, :2].contiguous(), i32([400]), 0.1, max_context=20,
                           k_new=kn[:1], v_new=kn[:1])                # clamped, nothing stored
    assert pkv.read_device_status() == OOB
    far = table.clone()
    far[2, 1] = c.num_blocks
    out = pkv.paged_decode_quant(q, c, far, i32(lens), 0.1, max_context=20)
    assert pkv.read_device_status() == OOB
    assert torch.equal(out[0], ok[0])
    far[:, 1] = -1                                                    # the new tokens' block
    pkv.paged_decode_quant(q, c, far, i32(lens), 0.1, max_context=20, k_new=kn, v_new=kn)
    assert pkv.read_device_status() == OOB
    assert all(torch.equal(t, w) for t, w in zip((c.k, c.v, c.k_scales, c.v_scales), before))


def test_refusals(pkv):
    c, table, _ = paged(pkv, [20], 2, 16, 64, "fp8", gen(3))
    q = torch.zeros(1, 4, 64, device="cuda", dtype=torch.bfloat16)
    n = i32([20])

    def call(**kw):
        a = dict(q=q, cache=c, block_tables=table, context_lens=n, scale=0.1, max_context=20)
        a.update(kw)
        return pkv.paged_decode_quant(**a)

    new = torch.zeros(1, 2, 64, device="cuda", dtype=torch.bfloat16)
    for wrong in (dict(k_new=new), dict(max_context=1000), dict(max_context=0)):
        with pytest.raises(pkv.PkvError) as e:
            call(**wrong)
        assert e.value.status == INVALID
    with pytest.raises(pkv.PkvError) as e:
        call(q=torch.zeros(1, 6, 64, device="cuda", dtype=torch.bfloat16))   # groups of 3
    assert e.value.status == 2
    with pytest.raises(pkv.PkvError) as e:
        call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), partition_blocks=1)
    assert e.value.status == NOMEM
    with pytest.raises(TypeError):
        call(q=q.half())
    with pytest.raises(TypeError):
        call(k_new=new.float(), v_new=new.float())
    with pytest.raises(TypeError):
        call(out=torch.empty(1, 4, 64, device="cuda"))
    with pytest.raises(ValueError):
        call(q=torch.zeros(1, 4, 128, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        call(block_tables=table[:, ::2])
    with pytest.raises(ValueError):
        call(context_lens=n.repeat(2))
    assert pkv.read_device_status() == 0


def test_graph_and_streams(pkv):
    """Two steps captured and replayed with other inputs; two streams with workspaces of their
    own at once."""
    lens, hkv, d = [700, 333], 2, 128
    for fmt in ("fp8", "fp4"):
        c, table, slots = paged(pkv, lens, hkv, 16, d, fmt, gen(6))
        q = torch.randn(2, 8, d, generator=gen(7), device="cuda").bfloat16()
        kn = torch.randn(2, hkv, d, generator=gen(8), device="cuda").bfloat16()
        vn = torch.randn(2, hkv, d, generator=gen(9), device="cuda").bfloat16()
        need = pkv.decode_quant_workspace_bytes(c, 2, 8, 700, 4)
        ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
        out = torch.empty_like(q)
        n = i32(lens)
        slot = torch.stack([s[-1] for s in slots])
        rows = [torch.empty(2, hkv, d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]

        def step():
            pkv.paged_decode_quant(q, c, table, n, 0.1, max_context=700, partition_blocks=4,
                                   k_new=kn, v_new=vn, out=out, workspace=ws[0])
            pkv.kv_read_quant(c, slot, k_out=rows[0], v_out=rows[1])

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        for seed in (1, 2):
            q.copy_(torch.randn(2, 8, d, generator=gen(seed), device="cuda"))
            kn.copy_(torch.randn(2, hkv, d, generator=gen(seed + 5), device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            got, got_rows = out.clone(), rows[0].clone()
            step()
            assert torch.equal(out, got) and torch.equal(rows[0], got_rows)
            assert torch.equal(got_rows.double().cpu(), kept(kn, fmt))
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [torch.empty_like(q) for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(20):
            for s, w, o in zip(streams, ws, outs):
                pkv.paged_decode_quant(q, c, table, n, 0.1, max_context=700, partition_blocks=4,
                                       out=o, workspace=w, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], out) and torch.equal(outs[1], out)
        assert pkv.read_device_status() == 0


def test_far_blocks(pkv):
    """Blocks whose bytes lie past 2^31 from the cache's start."""
    nb = 17 * (1 << 17) // 16                     # 2.28 GB of codes
    c = pkv.QuantCache.empty(nb, 8, 128, format="fp8")
    g = gen(11)
    table = torch.randint(nb - 5000, nb, (1, 40), generator=g, device="cuda").int()
    table[0, :] = torch.unique(table)[:40] if len(torch.unique(table)) >= 40 else \
        torch.arange(nb - 40, nb, device="cuda").int()
    t = torch.arange(640, device="cuda")
    slots = table[0].long()[t // 16] * 16 + t % 16
    k, v = (torch.randn(640, 8, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    pkv.kv_append_quant(c, slots, k, v)
    rk, rv = pkv.kv_read_quant(c, slots)
    assert torch.equal(rk.double().cpu(), kept(k, "fp8"))
    small = pkv.QuantCache.empty(40, 8, 128, format="fp8")
    pkv.kv_append_quant(small, t, k, v)
    q = torch.randn(1, 32, 128, generator=g, device="cuda").bfloat16()
    out = pkv.paged_decode_quant(q, c, table, i32([640]), 0.09, max_context=640)
    want = pkv.paged_decode_quant(q, small, torch.arange(40, device="cuda").int()[None].contiguous(),
                                  i32([640]), 0.09, max_context=640)
    assert torch.equal(out, want)
    assert pkv.read_device_status() == 0


def test_wait_that_runs_out(pkv):
    c, table, _ = paged(pkv, [100, 37], 2, 16, 128, "fp8", gen(3))
    q = torch.randn(2, 8, 128, generator=gen(4), device="cuda").bfloat16()
    os.environ["PKV_TEST_DECODE_STALL"] = "1"
    try:
        pkv.paged_decode_quant(q, c, table, i32([100, 37]), 0.1, max_context=100)
        torch.cuda.synchronize()
        assert pkv.read_device_status() == TIMEOUT
    finally:
        del os.environ["PKV_TEST_DECODE_STALL"]
    out = pkv.paged_decode_quant(q, c, table, i32([100, 37]), 0.1, max_context=100)
    assert pkv.read_device_status() == 0
    check(out, reference(c, q, table, [100, 37], 0.1))
