"""The quantised cache as a server uses it: prompts appended and prefilled through blocks read
back, a fork with copy-on-write, decode steps with their appends, finished blocks frozen from a
pool; and long contexts."""
import pytest
import torch

from tests.quant_refs import decode_bound, held, kept
from tests.shrink_refs import attention

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Rows:
    """The rows that a sequence should hold, float64 on the CPU."""

    def __init__(self, fmt, hkv, d):
        self.fmt, self.k, self.v = fmt, torch.zeros(0, hkv, d).double(), None
        self.v = self.k.clone()

    def add(self, k, v):
        self.k = torch.cat((self.k, kept(k, self.fmt)))
        self.v = torch.cat((self.v, kept(v, self.fmt)))

    def copy(self):
        r = Rows(self.fmt, *self.k.shape[1:])
        r.k, r.v = self.k.clone(), self.v.clone()
        return r


def read_back(pkv, alloc, cache, seqs, shape, dtype):
    """The sequences' blocks in a pool of their own: (K pool, V pool, table)."""
    tab = alloc.block_table(seqs, 64)
    src = sorted(set(tab[tab >= 0].tolist()))
    place = {b: i for i, b in enumerate(src)}
    kp, vp = (torch.zeros((len(src),) + shape, dtype=dtype, device="cuda") for _ in range(2))
    pkv.dequantize_blocks(cache, kp, vp, i32([[b, i] for b, i in place.items()]))
    return kp, vp, i32([[place.get(int(b), -1) for b in row] for row in tab])


def check_prefill(out, q, rows, first, scale):
    """Prefill over up to 1023 keys: weights in two bf16 parts (2^-14), scores as the decode's
    (decode_bound), the output rounded once."""
    want, _, _ = attention(q.double().cpu(), rows.k, rows.v, scale, first)
    got, qc = out.double().cpu(), q.double().cpu()
    for m in range(len(q)):
        n = first + m + 1
        x = torch.einsum("hgd,nhd->hgn", qc[m].view(rows.k.shape[1], -1, q.shape[-1]),
                         rows.k[:n]) * scale
        bound = decode_bound(qc[m], rows.k[:n], rows.v[:n], torch.softmax(x, -1), want[m], scale,
                             q.dtype)
        assert bool(((got[m] - want[m]).abs() <= bound).all()), m


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block,d", [(16, 128), (32, 64)])
def test_prompts_fork_decode(pkv, fmt, dtype, block, d):
    g = torch.Generator(device="cuda").manual_seed(block + d)
    hq, hkv, scale = 8, 2, d ** -0.5

    def draw(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    alloc = pkv.BlockAllocator(40, block_size=block, seed=7)
    cache = pkv.QuantCache.empty(40, hkv, d, block_size=block, format=fmt)
    for t in (cache.k, cache.v, cache.k_scales, cache.v_scales):
        t.fill_(0xFF)
    rows = {}
    freq, _ = pkv.rope_frequencies(d)
    # two prompts in chunks: the rows go into the cache, the blocks come back for the prefill
    for s in (0, 1):
        alloc.add_seq(s, 0)
        rows[s] = Rows(fmt, hkv, d)
    for news in ((50, 9), (21, 40)):
        qs, first, offs = [], [], [0]
        for s, n in enumerate(news):
            q, k, v = draw(n, hq, d), draw(n, hkv, d), draw(n, hkv, d)
            pos = torch.arange(alloc.seq_len(s), alloc.seq_len(s) + n, dtype=torch.int32,
                               device="cuda")
            q, k = pkv.rope(q, pos, freq), pkv.rope(k, pos, freq)
            first.append(alloc.seq_len(s))
            slots, cow = alloc.append(s, n)
            assert cow is None
            pkv.kv_append_quant(cache, torch.tensor(slots, device="cuda"), k, v)
            rows[s].add(k, v)
            qs.append(q)
            offs.append(offs[-1] + n)
        kp, vp, table = read_back(pkv, alloc, cache, [0, 1], (hkv, block, d), dtype)
        out = pkv.paged_prefill(torch.cat(qs), kp, vp, table, i32(first), i32(list(news)),
                                i32(offs), scale, max_new=max(news))
        assert pkv.read_device_status() == 0
        if dtype == torch.bfloat16:
            for s in (0, 1):
                check_prefill(out[offs[s]:offs[s + 1]], qs[s], rows[s], first[s], scale)
    # a third sequence forks from the first; all three decode, the fork's block is copied first
    alloc.fork(0, 2)
    rows[2] = rows[0].copy()
    copied = 0
    for _ in range(3):
        pairs, lens = [], []
        for s in (0, 1, 2):
            _, cow = alloc.append(s, 1)
            if cow is not None:
                pairs.append(list(cow))
            lens.append(alloc.seq_len(s))
        if pairs:
            pkv.copy_blocks_quant(cache, i32(pairs))
            copied += len(pairs)
        q, kn, vn = draw(3, hq, d), draw(3, hkv, d), draw(3, hkv, d)
        out = pkv.paged_decode_quant(q, cache, alloc.block_table([0, 1, 2], 64).cuda(), i32(lens),
                                     scale, max_context=max(lens), k_new=kn, v_new=vn)
        assert pkv.read_device_status() == 0
        for s in (0, 1, 2):
            rows[s].add(kn[s:s + 1], vn[s:s + 1])
            x = torch.einsum("hgd,nhd->hgn", q[s].cpu().double().view(hkv, -1, d),
                             rows[s].k) * scale
            p = torch.softmax(x, -1)
            ref = torch.einsum("hgn,nhd->hgd", p, rows[s].v).reshape(hq, d)
            bound = decode_bound(q[s].cpu().double(), rows[s].k, rows[s].v, p, ref, scale, dtype)
            assert bool(((out[s].double().cpu() - ref).abs() <= bound).all()), s
    assert copied == 1
    # what the cache holds is what was written, sequence by sequence
    ks, vs = (held(cache.k, cache.k_scales, fmt, False), held(cache.v, cache.v_scales, fmt, True))
    for s in (0, 1, 2):
        tab = alloc.block_table([s], 64)[0]
        ids = tab[tab >= 0].long()
        for val, want in ((ks, rows[s].k), (vs, rows[s].v)):
            assert torch.equal(val[ids].transpose(1, 2).reshape(-1, hkv, d)[:len(want)], want)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_frozen_blocks_decode_as_appended_ones(pkv, fmt):
    """A prompt kept in a pool and frozen gives the bytes, and the decode's bits, of one whose
    rows were quantised as they came."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n, hkv, d = 77, 3, 128
    k, v = (torch.randn(n, hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    kp, vp = (torch.zeros(9, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = torch.tensor([7, 2, 0, 5, 8], device="cuda")
    t = torch.arange(n, device="cuda")
    pkv.kv_append(kp, vp, ids[t // 16] * 16 + t % 16, k, v)
    frozen, appended = (pkv.QuantCache.empty(6, hkv, d, format=fmt) for _ in range(2))
    for c in (frozen, appended):
        for x in (c.k, c.v, c.k_scales, c.v_scales):
            x.zero_()
    to = torch.tensor([1, 4, 0, 3, 5], device="cuda")
    pkv.quantize_blocks(frozen, kp, vp, torch.stack((ids, to), 1).int().contiguous())
    pkv.kv_append_quant(appended, to[t // 16] * 16 + t % 16, k, v)
    q = torch.randn(1, 12, d, generator=g, device="cuda").bfloat16()
    outs = [pkv.paged_decode_quant(q, c, to[None].int().contiguous(), i32([n]), 0.09,
                                   max_context=80) for c in (frozen, appended)]
    assert torch.equal(outs[0], outs[1])
    a, b = (pkv.kv_read_quant(c, to[t // 16] * 16 + t % 16) for c in (frozen, appended))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert pkv.read_device_status() == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_long_context(pkv, fmt, dtype):
    """300 000 tokens, a few of which hold most of the weight: the many small weights count."""
    g = torch.Generator(device="cuda").manual_seed(9)
    n, d = 300_000, 64
    nb = -(-n // 16)
    cache = pkv.QuantCache.empty(nb, 1, d, format=fmt)
    k, v = (torch.randn(n, 1, d, generator=g, device="cuda") for _ in range(2))
    v += 0.5
    q = torch.randn(1, 8, d, generator=g, device="cuda").to(dtype)
    k[5] = q[0].float().mean(0) * 6
    perm = torch.randperm(nb, generator=g, device="cuda")
    t = torch.arange(n, device="cuda")
    slots = perm[t // 16] * 16 + t % 16
    pkv.kv_append_quant(cache, slots, k.bfloat16(), v.bfloat16())
    out = pkv.paged_decode_quant(q, cache, perm[None].int().contiguous(), i32([n]), d ** -0.5,
                                 max_context=n)
    assert pkv.read_device_status() == 0
    kk, vv = pkv.kv_read_quant(cache, slots)                 # exact in bf16
    x = torch.einsum("gd,nd->gn", q[0].double(), kk[:, 0].double()) * d ** -0.5
    p = torch.softmax(x, -1)
    ref = p @ vv[:, 0].double()
    # decode_bound, on the GPU: scores of `size`, n terms
    size = float((q[0].double().abs() @ kk[:, 0].double().abs().T).max()) * d ** -0.5
    rel = 2 * ((d + 12) * 2.0 ** -23 * size + (2 * size + 181) * 2.0 ** -24 + 2.0 ** -22)
    rel += (n / 2 ** 4) * 2.0 ** -23 + (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21)
    bound = ref.abs() * torch.finfo(dtype).eps / 2 * 1.01 + p @ vv[:, 0].double().abs() * rel
    assert bool(((out[0].double() - ref).abs() <= bound).all())
