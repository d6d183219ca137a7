"""Rows and blocks in and out of a quantised cache, against the 64-bit rounding: what is held
is the nearest value exactly, at every border, and nothing else is written."""
import pytest
import torch

from tests.quant_refs import held, kept, rows_of

pytestmark = pytest.mark.gpu

INVALID, OOB = 1, 5


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


def filled(pkv, nb, hkv, d, block, fmt, byte=0xA5):
    c = pkv.QuantCache.empty(nb, hkv, d, block_size=block, format=fmt)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        t.fill_(byte)
    return c


def both(c):
    return held(c.k, c.k_scales, c.format, False), held(c.v, c.v_scales, c.format, True)


def same(a, b):
    """Equal values, NaN in the same places, -0 as 0."""
    a, b = a.double().cpu(), b.double().cpu()
    return a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


def hard_rows(shape, g, dtype):
    """Rows of unequal sizes: zeros, far ends of the range, one outlier, NaN and infinities."""
    x = torch.randn(shape, generator=g, device="cuda")
    n = shape[0] * shape[1]
    flat = x.view(n, -1)
    for i, f in enumerate([0.0, 1e-30, 1e-38, 1e30, 3e38, 2.0 ** -98, 2.0 ** 98]):
        flat[(3 * i + 1) % n] *= f
    if n > 24:
        flat[23, 5] = 1e4
        flat[24, 5] = float("inf")
        flat[24, 6] = -float("inf")
        flat[22, 40] = float("nan")
        flat[21] = -0.0
    return x.to(dtype)


CASES = [(fmt, dt, d, b, hkv) for fmt in ("fp8", "fp4") for dt in (torch.bfloat16, torch.float32)
         for d, b, hkv in ((128, 16, 8), (64, 32, 3), (128, 32, 1), (64, 16, 2))]


@pytest.mark.parametrize("fmt,dtype,d,block,hkv", CASES)
@pytest.mark.parametrize("T", [1, 7, 130])
def test_append_then_read(pkv, fmt, dtype, d, block, hkv, T):
    g = gen(T + d)
    nb = T // block + 3
    c = filled(pkv, nb, hkv, d, block, fmt)
    before = [t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales)]
    x = torch.cat((hard_rows((T, hkv, d), g, dtype), hard_rows((T, hkv, d), g, dtype).flip(0)), 1)
    k, v = x[:, :hkv], x[:, hkv:]                     # slices of one projection
    slots = torch.randperm(nb * block, generator=g, device="cuda")[:T]
    if T > 4:
        slots[3] = -1
    pkv.kv_append_quant(c, slots, k, v)
    ks, vs = both(c)
    there = slots.cpu() >= 0
    assert same(rows_of(ks, slots[slots >= 0]), kept(k, fmt)[there])
    assert same(rows_of(vs, slots[slots >= 0]), kept(v, fmt)[there])
    # every other row is as it was
    other = torch.ones(nb * block, dtype=torch.bool)
    other[slots[slots >= 0].cpu()] = False
    for t, old in zip((c.k, c.v), before):
        rows = t.transpose(1, 2).reshape(nb * block, -1).cpu()
        assert torch.equal(rows[other], old.transpose(1, 2).reshape(nb * block, -1).cpu()[other])
    old_k, old_v = (held(before[i], before[i + 2], fmt, bool(i)) for i in range(2))
    idx = torch.arange(nb * block)[other]
    assert same(rows_of(ks, idx), rows_of(old_k, idx)) and same(rows_of(vs, idx),
                                                                rows_of(old_v, idx))
    # read back, rounded once, into slices of one array; padding reads zeros
    out = torch.full((T, 2 * hkv + 1, d), 7.0, device="cuda", dtype=dtype)
    rk, rv = pkv.kv_read_quant(c, slots, k_out=out[:, :hkv], v_out=out[:, hkv + 1:])
    for got, ref in ((rk, kept(k, fmt)), (rv, kept(v, fmt))):
        ref[~there] = 0
        assert same(got, ref.to(dtype))
    assert bool((out[:, hkv] == 7.0).all())
    assert pkv.read_device_status() == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_border(pkv, fmt, dtype):
    """Every bf16 value of a range beside a row's (fp4: a group's) largest one, all of the
    largest's digits: each code's borders, met and missed by one unit (fp32: the smallest)."""
    tops = torch.arange(128, 256, dtype=torch.float64) * 2.0 ** -7      # 8 digits
    vals = torch.arange(0x3a00, 0x4080, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    vals = vals.double()
    vals = vals[: len(vals) // 15 * 15].view(-1, 15)                    # 2^-11 .. 4 and more
    x = torch.empty(len(tops), len(vals), 16, dtype=torch.float64)
    x[..., 0] = tops[:, None]
    x[..., 1:] = torch.minimum(vals[None], tops[:, None, None])
    x[..., 1::2] *= -1
    if dtype == torch.float32:
        step = torch.tensor([0, 1, -1]).repeat(6)[:16]
        x = (x.float().view(torch.int32) + torch.where(x == 0, 0, step)).view(torch.float32)
    rows = x.reshape(-1, 64)
    rows = rows[: len(rows) // 4 * 4].view(-1, 4, 64).to(dtype).cuda()
    T = len(rows)
    c = filled(pkv, -(-T // 16), 4, 64, 16, fmt)
    slots = torch.arange(T, device="cuda")
    pkv.kv_append_quant(c, slots, rows, rows)
    ref = kept(rows, fmt)
    for val in both(c):
        assert same(rows_of(val, slots), ref)


@pytest.mark.parametrize("fmt,dtype,d,block,hkv", CASES)
def test_blocks_both_ways(pkv, fmt, dtype, d, block, hkv):
    g = gen(5 * d + block)
    nb, pool_nb = 9, 12
    kp, vp = (hard_rows((pool_nb * hkv, block, d), g, dtype).view(pool_nb, hkv, block, d)
              for _ in range(2))
    c = filled(pkv, nb, hkv, d, block, fmt)
    src = torch.randperm(pool_nb, generator=g, device="cuda")[:6]
    dst = torch.randperm(nb, generator=g, device="cuda")[:6]
    pairs = torch.stack((src, dst), 1).int().contiguous()
    before = both(c)
    pkv.quantize_blocks(c, kp, vp, pairs)
    for val, pool, old in zip(both(c), (kp, vp), before):
        assert same(val[dst.cpu()], kept(pool[src], fmt))
        rest = [i for i in range(nb) if i not in dst.tolist()]
        assert same(val[rest], old[rest])
    # as the rows would have been
    rowwise = filled(pkv, nb, hkv, d, block, fmt)
    slots = (dst[:, None] * block + torch.arange(block, device="cuda")).flatten()
    pkv.kv_append_quant(rowwise, slots, kp[src].transpose(1, 2).reshape(-1, hkv, d).contiguous(),
                        vp[src].transpose(1, 2).reshape(-1, hkv, d).contiguous())
    for name in ("k", "v", "k_scales", "v_scales"):
        assert torch.equal(getattr(c, name), getattr(rowwise, name)), name
    # and back, into other blocks
    ko, vo = (torch.full((pool_nb, hkv, block, d), 3.0, device="cuda", dtype=dtype)
              for _ in range(2))
    to = torch.randperm(pool_nb, generator=g, device="cuda")[:6]
    pkv.dequantize_blocks(c, ko, vo, torch.stack((dst, to), 1).int().contiguous())
    for got, pool in ((ko, kp), (vo, vp)):
        assert same(got[to], kept(pool[src], fmt).to(dtype))
        rest = [i for i in range(pool_nb) if i not in to.tolist()]
        assert bool((got[rest] == 3.0).all())
    assert pkv.read_device_status() == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_copy_blocks(pkv, fmt):
    c = pkv.QuantCache.empty(11, 3, 64, block_size=32, format=fmt)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        t.random_(0, 256, generator=gen(4))
    want = [t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales)]
    pairs = torch.tensor([[0, 10], [0, 4], [7, 1]], dtype=torch.int32, device="cuda")
    pkv.copy_blocks_quant(c, pairs)
    for t, w in zip((c.k, c.v, c.k_scales, c.v_scales), want):
        w[10], w[4], w[1] = w[0], w[0], w[7]
        assert torch.equal(t, w)
    assert pkv.read_device_status() == 0


def test_ids_outside(pkv):
    c = filled(pkv, 3, 2, 64, 16, "fp4")
    want = [t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales)]
    x = torch.ones(2, 2, 64, device="cuda", dtype=torch.bfloat16)
    far = torch.tensor([48, 1 << 40], device="cuda")
    pool = torch.ones(2, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    bad = torch.tensor([[2, 0], [-1, 0], [0, 3], [0, -5]], dtype=torch.int32, device="cuda")
    back = torch.tensor([[3, 0], [-1, 0], [0, 2], [0, -5]], dtype=torch.int32, device="cuda")
    for call in (lambda: pkv.kv_append_quant(c, far, x, x),
                 lambda: pkv.quantize_blocks(c, pool, pool, bad),
                 lambda: pkv.dequantize_blocks(c, pool, pool.clone(), back),
                 lambda: pkv.copy_blocks_quant(c, bad[1:])):
        call()
        assert pkv.read_device_status() == OOB
        assert all(torch.equal(t, w) for t, w in zip((c.k, c.v, c.k_scales, c.v_scales), want))
    assert bool((pool == 1).all())
    k, v = pkv.kv_read_quant(c, far)
    assert pkv.read_device_status() == OOB and not k.any() and not v.any()


def test_nothing_to_do(pkv):
    c = filled(pkv, 2, 2, 64, 16, "fp8")
    none = torch.empty(0, 2, 64, device="cuda", dtype=torch.float32)
    pkv.kv_append_quant(c, torch.empty(0, dtype=torch.int64, device="cuda"), none, none)
    k, v = pkv.kv_read_quant(c, torch.empty(0, dtype=torch.int64, device="cuda"),
                             dtype=torch.float32)
    assert k.shape == v.shape == (0, 2, 64) and k.dtype == torch.float32
    pairs = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    pool = torch.empty(2, 2, 16, 64, device="cuda")
    pkv.quantize_blocks(c, pool, pool, pairs)
    pkv.dequantize_blocks(c, pool, pool, pairs)
    pkv.copy_blocks_quant(c, pairs)
    assert bool((c.k == 0xA5).all()) and pkv.read_device_status() == 0


def test_refusals(pkv):
    c = filled(pkv, 4, 2, 64, 16, "fp8")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    x = torch.zeros(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkv.kv_append_quant(c, slots, x[:2], x[:2])            # other token counts
    with pytest.raises(TypeError):
        pkv.kv_append_quant(c, slots, x, x.float())            # two types
    with pytest.raises(TypeError):
        pkv.kv_append_quant(c, slots, x.half(), x.half())
    with pytest.raises(TypeError):
        pkv.kv_append_quant(c, slots.int(), x, x)
    with pytest.raises(ValueError):
        pkv.kv_append_quant(c, slots, x.transpose(1, 2).contiguous().transpose(1, 2), x)
    with pytest.raises(pkv.PkvError) as e:                     # tokens 2-byte aligned
        y = torch.zeros(3 * 129, device="cuda", dtype=torch.bfloat16).as_strided((3, 2, 64),
                                                                                (129, 64, 1))
        pkv.kv_append_quant(c, slots, y, x)
    assert e.value.status == INVALID
    with pytest.raises(pkv.PkvError) as e:                     # outputs in one another
        pkv.kv_read_quant(c, slots, k_out=x, v_out=x)
    assert e.value.status == INVALID
    with pytest.raises(TypeError):
        pkv.kv_read_quant(c, slots, dtype=torch.float16)
    pool = torch.zeros(4, 2, 32, 64, device="cuda")
    with pytest.raises(pkv.PkvError) as e:                     # other block sizes
        pkv.quantize_blocks(c, pool, pool, torch.zeros(1, 2, dtype=torch.int32, device="cuda"))
    assert e.value.status == INVALID
    with pytest.raises(ValueError):
        pkv.copy_blocks_quant(c, torch.zeros(1, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        pkv.QuantCache(c.k, c.v, c.k_scales[:, :, :8].contiguous(), c.v_scales)
    with pytest.raises(ValueError):
        pkv.QuantCache(c.k, c.v, c.k_scales, c.v_scales, format="fp4")   # heads of 128, scales short
    with pytest.raises(ValueError):
        pkv.QuantCache(c.k, c.v, c.k_scales, c.v_scales, format="int8")
    with pytest.raises(ValueError):
        pkv.QuantCache.empty(4, 2, 96)
    with pytest.raises(ValueError):
        pkv.QuantCache.empty(4, 2, 64, block_size=8)
    assert bool((c.k == 0xA5).all())
