"""Rotary positions on the GPU against the 64-bit rotation: layouts, partial heads, strided
inputs, far and negative positions, in place, inverse and gradient, and the fused append."""
import pytest
import torch

from tests.shrink_refs import rotate, rotate_bound

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


def check(got, x, pos, f, dtype, **kw):
    inverse = kw.pop("inverse", False)
    ref = rotate(x, pos, f, inverse=inverse, **kw)
    bound = rotate_bound(x, pos, f, ref, dtype, **kw)
    err = (got.detach().cpu().double() - ref).abs()
    assert bool((err <= bound).all()), (err - bound).max()
    r = 2 * f.numel()
    assert torch.equal(got[..., r:].cpu(), x[..., r:].cpu())       # passed on, bit for bit


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (64, 64), (128, 32), (128, 112), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (5, 3), (33, 40)])
def test_rope(pkv, dtype, d, rot, interleaved, T, H):
    g = gen(T * 1000 + rot)
    x = torch.randn(T, H, d, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 17, (T,), generator=g, device="cuda", dtype=torch.int32)
    f, _ = pkv.rope_frequencies(rot)
    before = x.clone()
    out = pkv.rope(x, pos, f, interleaved=interleaved)
    assert torch.equal(x, before)
    check(out, x, pos, f, dtype, interleaved=interleaved)
    out = pkv.rope(x, pos, f, interleaved=interleaved, inverse=True, attn_scale=1.25)
    check(out, x, pos, f, dtype, interleaved=interleaved, inverse=True, attn_scale=1.25)


@pytest.mark.parametrize("T", [2047, 2048, 2050, 4099])   # around the launch rule's border
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_many_tokens(pkv, T, dtype):
    g = gen(T)
    x = torch.randn(T, 3, 128, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 4096, (T,), generator=g, device="cuda", dtype=torch.int32)
    f, _ = pkv.rope_frequencies(96)
    check(pkv.rope(x, pos, f), x, pos, f, dtype)


def test_far_and_negative_positions(pkv):
    """The whole int32 range; frequencies of a turn and more per position, and negative ones."""
    pos = torch.tensor([0, 1, -1, 2, 1 << 20, -(1 << 20), (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)],
                       dtype=torch.int32, device="cuda")
    x = torch.randn(pos.numel(), 2, 64, generator=gen(3), device="cuda")
    f, _ = pkv.rope_frequencies(64, 1e6)
    check(pkv.rope(x, pos, f), x, pos, f, torch.float32)
    f2 = torch.tensor([7.0, 6.283185307179586, -0.5, 1e-9, 0.0, 3.0, 100.25, 1e-300],
                      dtype=torch.float64, device="cuda")
    near = torch.arange(-4, 5, dtype=torch.int32, device="cuda")
    check(pkv.rope(x, near, f2), x, near, f2, torch.float32)


def test_strided_in_place_and_slices(pkv):
    g = gen(5)
    for dtype in (torch.bfloat16, torch.float32):
        qkv = torch.randn(7, 12, 64, generator=g, device="cuda").to(dtype)
        keep = qkv.clone()
        pos = torch.arange(100, 107, dtype=torch.int32, device="cuda")
        f, _ = pkv.rope_frequencies(64)
        q = qkv[:, 2:6]
        out = pkv.rope(q, pos, f)
        assert out.is_contiguous()
        check(out, keep[:, 2:6], pos, f, dtype)
        assert pkv.rope(q, pos, f, out=q) is q                  # in place, among its neighbours
        assert torch.equal(qkv[:, 2:6], out)
        assert torch.equal(qkv[:, :2], keep[:, :2]) and torch.equal(qkv[:, 6:], keep[:, 6:])
        one = torch.randn(1, 4, 64, generator=g, device="cuda").to(dtype).expand(7, 4, 64)
        check(pkv.rope(one, pos, f), one, pos, f, dtype)        # one row, every position
    x = torch.randn(4, 2, 64, device="cuda")
    f, _ = pkv.rope_frequencies(64)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (x.transpose(0, 1), x[..., ::2], x[:, :, :32]):
        with pytest.raises((ValueError, pkv.PkvError)):
            pkv.rope(bad, pos[:bad.shape[0]], f)
    with pytest.raises(ValueError):
        pkv.rope(x, pos[:3], f)
    with pytest.raises(TypeError):
        pkv.rope(x, pos.long(), f)
    with pytest.raises(TypeError):
        pkv.rope(x, pos, f.float())
    with pytest.raises(TypeError):
        pkv.rope(x.half(), pos, f)
    assert pkv.rope(x[:0], pos[:0], f).shape == (0, 2, 64)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(pkv, interleaved):
    """d loss / d x is the inverse turn of d loss / d out: against the formula, and against
    differences of the loss.  The loss <out, w> is linear in x, so a difference of step h has
    no truncation error; its rounding is that of the outputs: each is off by at most 2^-21
    attn_scale (|a| + |b|) (see rotate_bound), the sum over 2 elements with |w| and |x| below
    8 and h = 8: below 2 * 2^-21 * 1.5 * 32 * 8 * 2 / 8 < 2^-13."""
    g = gen(11)
    x = torch.randn(3, 2, 64, generator=g, device="cuda")
    w = torch.randn(3, 2, 64, generator=g, device="cuda")
    pos = torch.tensor([5, 77777, 3], dtype=torch.int32, device="cuda")
    f, _ = pkv.rope_frequencies(48)
    grad = pkv.rope(w, pos, f, interleaved=interleaved, inverse=True, attn_scale=1.5)
    check(grad, w, pos, f, torch.float32, interleaved=interleaved, inverse=True, attn_scale=1.5)
    # the plain gradient: autograd through the 64-bit rotation
    y = x.cpu().double().requires_grad_()
    angle = pos.cpu().double()[:, None, None] * f.cpu()
    c, s = torch.cos(angle) * 1.5, torch.sin(angle) * 1.5
    lo, hi = (slice(0, 48, 2), slice(1, 48, 2)) if interleaved else (slice(0, 24), slice(24, 48))
    wd = w.cpu().double()
    loss = ((y[..., lo] * c - y[..., hi] * s) * wd[..., lo]).sum() + \
        ((y[..., hi] * c + y[..., lo] * s) * wd[..., hi]).sum() + (y[..., 48:] * wd[..., 48:]).sum()
    loss.backward()
    assert float((grad.cpu().double() - y.grad).abs().max()) < 2.0 ** -17
    for at in ((0, 0, 0), (1, 1, 25), (2, 0, 47), (1, 0, 63)):
        h = torch.zeros_like(x)
        h[at] = 8.0
        up = pkv.rope(x + h, pos, f, interleaved=interleaved, attn_scale=1.5).double()
        dn = pkv.rope(x - h, pos, f, interleaved=interleaved, attn_scale=1.5).double()
        diff = float(((up - dn) * w.double()).sum()) / (
            float((x + h)[at]) - float((x - h)[at]))
        assert abs(diff - float(grad[at])) < 2.0 ** -13
    # forward then inverse gives the input back
    back = pkv.rope(pkv.rope(x, pos, f, interleaved=interleaved), pos, f, interleaved=interleaved,
                    inverse=True)
    assert float((back - x).abs().max()) < 2.0 ** -18


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,bs,hkv,group", [(64, 16, 1, 1), (64, 32, 3, 2), (128, 16, 8, 4),
                                            (128, 32, 2, 8)])
@pytest.mark.parametrize("T", [1, 37, 2051])
def test_rope_append(pkv, dtype, d, bs, hkv, group, T):
    """q_out, the rows in the pools, every other row untouched; padding rows skipped; and the
    same rows as rope followed by kv_append, bit for bit."""
    g = gen(T + d)
    hq = hkv * group
    qkv = torch.randn(T, hq + 2 * hkv, d, generator=g, device="cuda").to(dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    nb = -(-T // bs) + 2
    kp = torch.randn(nb, hkv, bs, d, generator=g, device="cuda").to(dtype)
    vp = torch.randn(nb, hkv, bs, d, generator=g, device="cuda").to(dtype)
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:T].contiguous()
    if T > 4:
        slots[3] = -1
    pos = torch.randint(0, 9999, (T,), generator=g, device="cuda", dtype=torch.int32)
    f, _ = pkv.rope_frequencies(d if T != 37 else 32)
    for interleaved in (False, True):
        kp1, vp1, kp2, vp2 = kp.clone(), vp.clone(), kp.clone(), vp.clone()
        out = pkv.rope_append(q, k, v, kp1, vp1, slots, pos, f, interleaved=interleaved,
                              attn_scale=1.1)
        check(out, q, pos, f, dtype, interleaved=interleaved, attn_scale=1.1)
        turned = pkv.rope(k, pos, f, interleaved=interleaved, attn_scale=1.1)
        check(turned, k, pos, f, dtype, interleaved=interleaved, attn_scale=1.1)
        pkv.kv_append(kp2, vp2, slots, turned, v.contiguous())
        assert torch.equal(kp1, kp2) and torch.equal(vp1, vp2)
        assert torch.equal(out, pkv.rope(q, pos, f, interleaved=interleaved, attn_scale=1.1))
    assert pkv.read_device_status() == 0


def test_rope_append_bad_slot(pkv):
    kp = torch.zeros(2, 2, 16, 64, device="cuda")
    vp = torch.zeros_like(kp)
    x = torch.ones(3, 2, 64, device="cuda")
    slots = torch.tensor([32, 5, 1 << 40], device="cuda")          # past the pool, good, far past
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    f, _ = pkv.rope_frequencies(64)
    out = pkv.rope_append(x, x, x, kp, vp, slots, pos, f)
    assert pkv.read_device_status() == 5
    assert torch.equal(out, x)
    assert float(kp.sum()) == 2 * 64 and float(vp.sum()) == 2 * 64
    assert float(kp[0, :, 5].sum()) == 2 * 64


def test_streams_and_capture(pkv):
    """On a stream of its own, and captured and replayed over new inputs."""
    g = gen(21)
    T, hq, hkv, d = 64, 8, 2, 128
    qkv = torch.randn(T, hq + 2 * hkv, d, generator=g, device="cuda").bfloat16()
    kp = torch.zeros(8, hkv, 16, d, device="cuda", dtype=torch.bfloat16)
    vp = torch.zeros_like(kp)
    slots = torch.randperm(128, generator=g, device="cuda")[:T].contiguous()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f, _ = pkv.rope_frequencies(128)
    out = torch.empty(T, hq, d, device="cuda", dtype=torch.bfloat16)

    def call(**kw):
        return pkv.rope_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kp, vp, slots,
                               pos, f, **kw)

    eager = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        other = call(stream=stream)
        s.synchronize()
        assert torch.equal(other, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(q_out=out)
    torch.cuda.synchronize()
    qkv.mul_(-0.5)
    pos.add_(1000)
    graph.replay()
    torch.cuda.synchronize()
    replayed, pools = out.clone(), (kp.clone(), vp.clone())
    eager = call()
    assert torch.equal(replayed, eager)
    assert torch.equal(pools[0], kp) and torch.equal(pools[1], vp)
    assert pkv.read_device_status() == 0
