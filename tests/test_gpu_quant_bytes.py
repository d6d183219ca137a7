"""Bytes that a quantised cache holds: scales next to a border, zeros with a sign, the same from
rows of either type; and what a description may not share."""
import pytest
import torch

from tests.quant_refs import e4m3_values, held, nearest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_58_gb300 import build
    build.build()
    import paged_kv_cache_58_gb300 as m
    assert m.read_device_status() == 0
    return m


def cleared(pkv, nb, hkv, d, fmt):
    c = pkv.QuantCache.empty(nb, hkv, d, format=fmt)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        t.zero_()
    return c


def test_fp4_scales_next_to_every_border(pkv):
    """A group's scale is the e4m3 value nearest to a sixth of its largest magnitude, taken in 64
    bits: fp32 magnitudes on six times each border and up to three units to both sides."""
    pos = e4m3_values()[:127]
    border = (pos[1:] + pos[:-1]) / 2
    at = (6 * border).float()
    near = torch.stack([(at.view(torch.int32) + u).view(torch.float32) for u in range(-3, 4)], 1)
    near = torch.cat((near.flatten(), torch.tensor([float.fromhex("0x1.c7fffep+9"),
                                                    float.fromhex("0x1.c7fffep+10")])))
    d, T = 128, -(-len(near) // 7)
    a = torch.zeros(T * 7)
    a[:len(near)] = near
    rows = torch.zeros(T, 8, 16)
    rows[:, 0, 3] = 2688.0                     # the row's exponent is 0
    rows[:, 1:, 5] = a.view(T, 7)
    rows[:, 1:, 9] = a.view(T, 7) / 4          # beside the largest one
    x = rows.view(T, 1, d).cuda()
    c = cleared(pkv, -(-T // 16), 1, d, "fp4")
    pkv.kv_append_quant(c, torch.arange(T, device="cuda"), x, -x)
    want = nearest(a.double() / 6, pos).view(T, 7)
    t = torch.arange(T)
    for is_v, side in ((False, c.k_scales), (True, c.v_scales)):
        side = side.cpu().view(-1, d + 16)
        assert bool((side[t // 16, d + t % 16] == 127).all())
        g = torch.arange(8)
        byte = ((t % 16)[:, None] // 4 * (d // 4) + 4 * g + (t % 16)[:, None] % 4 if is_v
                else (t % 16)[:, None] * 8 + g)
        got = e4m3_values()[side[t // 16][t[:, None], byte].long()]
        assert torch.equal(got[:, 1:], want), (got[:, 1:] - want).abs().max()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_zeros_with_a_sign(pkv, fmt):
    """Small negative elements, negative zeros, groups and rows of them: rows of bf16 and the same
    in fp32 leave the same bytes, whatever the other elements of their group are."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(96, 2, 128, generator=g, device="cuda")
    x[::3] *= 2.0 ** -torch.randint(0, 20, (32, 2, 128), generator=g, device="cuda").float()
    x[1::3, :, ::2] = -0.0
    x[4, :, 16:32] = -0.0
    x[5, :, 16:32] = -1e-6
    x[6] = -0.0
    x[8, :, 1:] = -1e-30
    x = x.bfloat16()
    caches = [cleared(pkv, 6, 1, 128, fmt) for _ in range(3)]
    slots = torch.arange(96, device="cuda")
    y = x.float()
    z = y.clone()
    off = torch.rand(96, 2, 8, generator=g, device="cuda") * 1e-6      # off the borders' grid
    part = z[:, :, 40:48]
    part += torch.where(part.abs() < 0.5 * z.abs().amax(-1, keepdim=True), off, 0.0)
    pkv.kv_append_quant(caches[0], slots, x[:, :1], x[:, 1:])
    pkv.kv_append_quant(caches[1], slots, y[:, :1], y[:, 1:])
    for name in ("k", "v", "k_scales", "v_scales"):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name
    # other groups of the rows that changed keep their bytes
    pkv.kv_append_quant(caches[2], slots, z[:, :1], z[:, 1:])
    keep = slice(64, 128) if fmt == "fp8" else slice(32, 64)
    for a, b in ((caches[1].k, caches[2].k), (caches[1].v, caches[2].v)):
        assert torch.equal(a.view(96, -1)[:, keep], b.view(96, -1)[:, keep])
    if fmt == "fp4":
        for c in caches[:2]:
            assert not any(bool((t & 15 == 8).any() or (t >> 4 == 8).any()) for t in (c.k, c.v))
    assert pkv.read_device_status() == 0


def test_fresh_pools_and_arrays_apart(pkv):
    """One tensor for K and V, or for codes and scales of both, is refused; halves of one are not."""
    c = cleared(pkv, 3, 2, 64, "fp8")
    with pytest.raises(ValueError):
        pkv.QuantCache(c.k, c.k, c.k_scales, c.v_scales)
    with pytest.raises(ValueError):
        pkv.QuantCache(c.k, c.v, c.k_scales, c.k_scales)
    flat = torch.zeros(2 * c.k.numel(), dtype=torch.uint8, device="cuda")
    n = c.k.numel()
    with pytest.raises(ValueError):
        pkv.QuantCache(c.k, flat[64:64 + n].view(c.k.shape), flat[:n].view(c.k.shape)[:, :, :, 0]
                       .contiguous(), flat[:c.k_scales.numel()].view(c.k_scales.shape))
    both = pkv.QuantCache(flat[:n].view(c.k.shape), flat[n:].view(c.k.shape), c.k_scales,
                          c.v_scales)
    x = torch.randn(5, 2, 64, generator=torch.Generator(device="cuda").manual_seed(1),
                    device="cuda")
    pkv.kv_append_quant(both, torch.arange(5, device="cuda"), x, -x)
    pool = torch.full((3, 2, 16, 64), 7.0, device="cuda")
    pairs = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    with pytest.raises(pkv.PkvError) as e:
        pkv.dequantize_blocks(both, pool, pool, pairs)
    assert e.value.status == 1
    assert bool((pool == 7.0).all())
    two = torch.zeros(2, 3, 2, 16, 64, device="cuda")
    pkv.dequantize_blocks(both, two[0], two[1], pairs)
    assert torch.equal(two[0, 1, :, :5].double().cpu(),
                       held(both.k, both.k_scales, "fp8", False)[0, :, :5])
    assert torch.equal(two[0, 1, :, :5], -two[1, 1, :, :5])
    pkv.quantize_blocks(both, two[1], two[1], pairs)         # sources may be one pool
    assert pkv.read_device_status() == 0
