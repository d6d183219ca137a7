"""Corners of the operators around a shrinking cache that their own files do not reach: wide
clusters over short rows."""
import pytest
import torch

from tests.test_gpu_evict import bits, expect, gen, i32, same_positions, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_58_gb300 import build
    build.build()
    import paged_kv_cache_58_gb300 as m
    return m


@pytest.mark.parametrize("kind", ["spread", "zeros"])
def test_evict_wide_clusters_over_short_rows(pkv, kind):
    """A bound that gives every row eight CTAs, and rows of which most of them have no entry:
    those reach the exchange through shared memory at once, the others after a scan."""
    lens = [1, 31, 33, 64, 257, 600, 9000, 0, 2049, 40]
    budgets = [0, 30, 1, 32, 256, 10, 512, 4, 2048, 40]
    hkv, bs, bound = 2, 16, 9008
    kp, vp, table, g = setup(lens, hkv, bs, 64, torch.bfloat16, 31)
    w = torch.rand(len(lens), hkv, bound, generator=gen(32), device="cuda")
    if kind == "zeros":
        w.zero_()
    pos = torch.zeros(w.shape, dtype=torch.int32, device="cuda")
    rows = list(range(len(lens)))
    want = expect(kp, vp, table, lens, budgets, w, pos, 3, 8, lens, [0] * len(lens), rows)
    left = pkv.evict(kp, vp, table, i32(lens), i32(budgets), w, pos, max_context=bound, sinks=3,
                     recent=8)
    assert pkv.read_device_status() == 0
    assert left.tolist() == want[4]
    assert torch.equal(bits(kp), bits(want[0])) and torch.equal(bits(vp), bits(want[1]))
    assert torch.equal(w.cpu(), want[2])
    assert same_positions(pos, want[3], rows, want[4])
