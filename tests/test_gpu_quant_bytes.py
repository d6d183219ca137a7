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