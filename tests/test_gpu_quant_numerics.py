"""Digits of the decode over a quantised cache, where the scores are known exactly.

q has one element and K's rows one, so that a score is one product: what is left of an output's
error is that of the softmax and of the sums, and the bounds are a few units in the last place."""
import pytest
import torch

from tests.quant_refs import held

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


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


def filled(pkv, k, v, fmt, block=16):
    """A cache of the rows k, v [S, n, Hkv, D] fp32, its table [S, blocks], and the rows as held,
    float64 on the CPU."""
    S, n, hkv, d = k.shape
    per = -(-n // block)
    c = pkv.QuantCache.empty(S * per, hkv, d, block_size=block, format=fmt)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        t.fill_(0xFF)
    table = torch.randperm(S * per, generator=gen(99), device="cuda").view(S, per)
    t = torch.arange(n, device="cuda")
    slots = (table[:, t // block] * block + t % block).flatten()
    pkv.kv_append_quant(c, slots, k.flatten(0, 1), v.flatten(0, 1))
    kk, vv = pkv.kv_read_quant(c, slots, dtype=torch.float32)
    return c, table.int().contiguous(), kk.view(k.shape), vv.view(k.shape)


def weights(x):
    """Softmax of the scores x [..., n], float64; scores of -inf among them have none."""
    return torch.softmax(x - x.amax(-1, keepdim=True), -1)


def half_step(x, dtype):
    """Half the distance between neighbouring values of `dtype` about x."""
    e = torch.floor(torch.log2(x.abs().clamp(min=1e-300)))
    return 2.0 ** (e - (8 if dtype == torch.bfloat16 else 24))


def check(out, ref, off, dtype):
    """`off`: how far the output may be before it is rounded to its type."""
    off = off + 1e-37
    off = off + half_step(ref.abs() + off, dtype)
    err = (out.double() - ref).abs()
    assert bool((err <= off).all()), (float((err - off).max()), float((err / ref.abs()).max()))


def run(pkv, q, c, table, n, scale, parts=0):
    lens = torch.full((len(q),), n, dtype=torch.int32, device="cuda")
    out = pkv.paged_decode_quant(q, c, table, lens, scale, max_context=n, partition_blocks=parts)
    assert pkv.read_device_status() == 0
    return out


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_token_comes_back(pkv, fmt, dtype):
    """One token has all the weight: its V comes back, whatever its exponent and score.

    The weight's argument is below 8 in magnitude and rounded (2^-22, ln 2 times that of the
    weight), exp2 is off by 2^-22 in weight and denominator, the weight's two parts by U, the two
    sums by U each, the quotients by 3 U: 12 U in all.  (bf16: a code's value is one of bf16.)"""
    S, G, d = 512, 8, 64
    g = gen(1)
    k = torch.zeros(S, 1, 1, d, device="cuda")
    k[..., 0] = (1 + torch.randint(0, 8, (S, 1, 1), generator=g, device="cuda") / 8) \
        * 2.0 ** -torch.randint(0, 2, (S, 1, 1), generator=g, device="cuda")
    size = torch.randint(-85, 86, (S, 1, 1, 1), generator=g, device="cuda").double()
    v = (torch.randn(S, 1, 1, d, generator=g, device="cuda").double() * 2.0 ** size).float()
    c, table, kk, vv = filled(pkv, k, v, fmt)
    q = torch.zeros(S, G, d, device="cuda", dtype=dtype)
    q[..., 0] = 1 + torch.arange(G, device="cuda") / 8
    q[::2] *= -1
    out = run(pkv, q, c, table, 1, 0.5).double()
    want = vv.double()[:, 0].expand(S, G, d)
    if dtype == torch.bfloat16:
        assert torch.equal(out, want)
    else:
        assert bool(((out - want).abs() <= 12 * U * want.abs()).all()), \
            float(((out - want).abs() / want.abs().clamp(min=1e-300)).max() / U)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("size", [2, 20, 25, 40, 110, 120])
def test_scores_of_any_size(pkv, fmt, dtype, sign, size):
    """Two levels of scores of about 2^size (and, at 120, keys whose scores are -inf), V rows whose
    sizes differ by 2^40: the tokens of the higher level share the weight.

    Scores of a level are equal to the bit; at size 2, where both count, they are off by 2 U of
    8.  exp2 by 2^-22 in each weight and denominator.  Up to 2 n + 64 roundings of sums.  What is
    below 2^-31 of the largest contribution may be lost, of n tokens."""
    n, hkv, G, d = 100, 2, 4, 64
    g = gen(size + 2 * sign + 7)
    kexp = min(90, size // 2)
    k = torch.zeros(2, n, hkv, d, device="cuda")
    high = torch.rand(2, n, hkv, generator=g, device="cuda") < 0.5
    high[:, 50] = True
    k[..., 0] = torch.where(high, 1.0 if sign < 0 else 1.5, 1.5 if sign < 0 else 1.0) * 2.0 ** kexp
    if size == 120 and sign < 0:
        k[:, ::7, :, 0] = 2.0 ** 90
    e = torch.randint(-20, 21, (2, n, hkv, 1), generator=g, device="cuda").float()
    v = torch.randn(2, n, hkv, d, generator=g, device="cuda") * 2.0 ** e
    c, table, kk, vv = filled(pkv, k, v, fmt)
    q = torch.zeros(2, hkv * G, d, device="cuda", dtype=dtype)
    q[..., 0] = sign * 2.0 ** (size - kexp)
    x = torch.einsum("shgd,snhd->shgn", q.double().view(2, hkv, G, d), kk.double()) * 0.5
    x = torch.where(x.abs() > 3.4e38, torch.full_like(x, sign * torch.inf), x)
    p = weights(x)
    ref = torch.einsum("shgn,snhd->shgd", p, vv.double()).reshape(2, hkv * G, d)
    mag = torch.einsum("shgn,snhd->shgd", p, vv.double().abs()).reshape(ref.shape)
    rel = (2 * n + 64) * U + 2.0 ** -20 + (2 * 2 * 8 * U if size == 2 else 0)
    top = vv.double().abs().amax(-1).transpose(1, 2)[:, :, None]       # [S, Hkv, 1, n]
    small = ((p * top).amax(-1) * n * 2.0 ** -30).reshape(2, hkv * G, 1)
    for parts in (0, 1):
        check(run(pkv, q, c, table, n, 0.5, parts), ref, mag * rel + small, dtype)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_keys_beside_large_queries(pkv, fmt, dtype):
    """Keys of 2^97 in dimensions where a query of 2^60 in another one is zero: scores of zero,
    so that the output is the mean of V (n + 64 roundings, exp2's 2^-22 twice)."""
    n, d = 40, 64
    g = gen(3)
    k = torch.randn(1, n, 1, d, generator=g, device="cuda") * 2.0 ** 95
    k[..., :2] = 0
    v = torch.randn(1, n, 1, d, generator=g, device="cuda")
    c, table, kk, vv = filled(pkv, k, v, fmt)
    q = torch.zeros(1, 2, d, device="cuda", dtype=dtype)
    q[..., 0] = 2.0 ** 60
    q[:, 1, 1] = -(2.0 ** 100)
    out = run(pkv, q, c, table, n, 1.0)
    ref, mag = (x.double()[:, :, 0].mean(1, keepdim=True).expand(1, 2, d) for x in (vv, vv.abs()))
    check(out, ref, mag * ((n + 64) * U + 2.0 ** -21), dtype)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("how", ["equal", "mixed"])
def test_weights_keep_their_digits(pkv, fmt, dtype, group, how):
    """Equal scores have one weight, and what is cut off it is cut off each: with V's of one sign
    the errors add up.  Mixed ones weigh by scores up to 4.

    Scores are off by 2 U of 4, twice; arguments of exp2 (up to 16) by 2^-21, its values by 2^-22,
    twice each; n + 64 roundings of sums; the weights' two parts by U."""
    S, n, hkv, d = 8, 48, 2, 128
    g = gen(group)
    k = torch.zeros(S, n, hkv, d, device="cuda")
    count = n if how == "mixed" else 1
    k[..., 0] = (1 + torch.randint(0, 8, (S, count, hkv), generator=g, device="cuda") / 8) \
        * 2.0 ** -torch.randint(0, 3, (S, count, hkv), generator=g, device="cuda")
    v = 1 + torch.randn(S, n, hkv, d, generator=g, device="cuda").abs()
    c, table, kk, vv = filled(pkv, k, v, fmt)
    q = torch.zeros(S, hkv * group, d, device="cuda", dtype=dtype)
    q[..., 0] = 1 + torch.arange(hkv * group, device="cuda") / 16
    x = torch.einsum("shgd,snhd->shgn", q.double().view(S, hkv, group, d), kk.double()) * 0.75
    p = weights(x)
    ref = torch.einsum("shgn,snhd->shgd", p, vv.double()).reshape(q.shape)
    rel = (2 * 2 * 4 + n + 64 + 1) * U + 2 * (2.0 ** -21 + 2.0 ** -22)
    for parts in (0, 1):
        check(run(pkv, q, c, table, n, 0.75, parts), ref, ref * rel, dtype)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [4, 8])
@pytest.mark.parametrize("how", ["equal", "mixed"])
def test_digits_at_length(pkv, fmt, dtype, group, how):
    """70 001 tokens in partitions of 4096, so that a warp sums 64 chunks: bounds by the order in
    which the sums are taken, below what one of the weights' two parts would cost (2^-12).

    An accumulator takes two products a chunk, rounded or cut, each a sum of 16 tokens that loses
    16 U / 2 at most; a denominator 2 x 64 additions of half a unit; 64 more for the merges of
    lanes, warps and 18 partitions.  The rest as above."""
    n, d = 70001, 64
    g = gen(group + 20)
    k = torch.zeros(1, n, 1, d, device="cuda")
    count = n if how == "mixed" else 1
    k[..., 0] = (1 + torch.randint(0, 8, (1, count, 1), generator=g, device="cuda") / 8) \
        * 2.0 ** -torch.randint(0, 3, (1, count, 1), generator=g, device="cuda")
    v = 1 + torch.randn(1, n, 1, d, generator=g, device="cuda").abs()
    c, table, kk, vv = filled(pkv, k, v, fmt)
    q = torch.zeros(1, group, d, device="cuda", dtype=dtype)
    q[..., 0] = 1 + torch.arange(group, device="cuda") / 16
    x = (q.double()[0] @ kk.double()[0, :, 0].T) * 0.75
    ref = (weights(x) @ vv.double()[0, :, 0])[None]
    rel = (2 * 64 + 8 + 64 + 64 + 2 * 2 * 4 + 1) * U + 2 * (2.0 ** -21 + 2.0 ** -22)
    assert rel < 2.0 ** -14
    check(run(pkv, q, c, table, n, 0.75, 256), ref, ref * rel, dtype)


def test_reading_back_is_exact(pkv):
    """`filled` takes the rows as held from kv_read_quant: in fp32 they are the cache's bytes."""
    for fmt in ("fp8", "fp4"):
        k, v = (torch.randn(1, 40, 2, 64, generator=gen(s), device="cuda") for s in (1, 2))
        c, table, kk, vv = filled(pkv, k, v, fmt)
        t = torch.arange(40)
        ids = table[0].cpu().long()[t // 16]
        for got, codes, side, is_v in ((kk, c.k, c.k_scales, False), (vv, c.v, c.v_scales, True)):
            assert torch.equal(got[0].double().cpu(), held(codes, side, fmt, is_v)[ids, :, t % 16])
