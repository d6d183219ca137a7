"""Prompts over a quantised cache in fp32: their blocks come back into a pool and are attended
there, in chunks over a cached prefix."""
import pytest
import torch

from tests.test_gpu_quant_serving import Rows, check_prefill, i32, read_back

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


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("block,d", [(16, 128), (32, 64)])
def test_fp32_prompts_in_chunks(pkv, fmt, block, d):
    """Against 64-bit attention over the rows as held, within an fp32 decode's bound."""
    g = torch.Generator(device="cuda").manual_seed(block)
    hq, hkv, scale = 8, 2, d ** -0.5
    alloc = pkv.BlockAllocator(30, block_size=block, seed=3)
    cache = pkv.QuantCache.empty(30, hkv, d, block_size=block, format=fmt)
    for t in (cache.k, cache.v, cache.k_scales, cache.v_scales):
        t.fill_(0xFF)
    rows = {}
    for s in (0, 1):
        alloc.add_seq(s, 0)
        rows[s] = Rows(fmt, hkv, d)
    for news in ((37, 1), (1, 70), (33, 16)):
        qs, first, offs = [], [], [0]
        for s, n in enumerate(news):
            q, k, v = (torch.randn(n, h, d, generator=g, device="cuda") for h in (hq, hkv, hkv))
            first.append(alloc.seq_len(s))
            slots, _ = alloc.append(s, n)
            pkv.kv_append_quant(cache, torch.tensor(slots, device="cuda"), k, v)
            rows[s].add(k, v)
            qs.append(q)
            offs.append(offs[-1] + n)
        kp, vp, table = read_back(pkv, alloc, cache, [0, 1], (hkv, block, d), torch.float32)
        out = pkv.paged_prefill(torch.cat(qs), kp, vp, table, i32(first), i32(list(news)),
                                i32(offs), scale, max_new=max(news))
        assert pkv.read_device_status() == 0
        for s in (0, 1):
            check_prefill(out[offs[s]:offs[s + 1]], qs[s], rows[s], first[s], scale)
