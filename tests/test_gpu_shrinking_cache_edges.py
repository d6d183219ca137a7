"""Corners of the operators around a shrinking cache that their own files do not reach: wide
clusters over short rows, the rotation inside a differentiated program,
decode steps that follow each other without a pause, prompt
weights whose bits must not depend on what ran before, and whose waits run out."""
import pytest
import torch

from tests.shrink_refs import rotate, rotate_bound
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved,inverse", [(False, False), (True, True)])
def test_rope_in_a_differentiated_program(pkv, dtype, interleaved, inverse):
    """The output carries a gradient: the opposite turn of the output's, for gradients of any
    layout (expanded, strided, off the 16-byte grid); and it has one itself."""
    g = gen(41)
    f, _ = pkv.rope_frequencies(48)
    pos = torch.tensor([5, 77777, 3], dtype=torch.int32, device="cuda")
    leaf = torch.randn(3, 6, 64, generator=g, device="cuda").to(dtype).requires_grad_()
    x = leaf[:, 2:4]                                        # a slice of a fused projection
    kw = dict(interleaved=interleaved, attn_scale=1.5)
    y = pkv.rope(x, pos, f, inverse=inverse, **kw)
    assert y.requires_grad
    with torch.no_grad():
        plain = pkv.rope(x, pos, f, inverse=inverse, **kw)
    assert not plain.requires_grad and torch.equal(plain, y.detach())
    w = torch.randn(3, 2, 64, generator=g, device="cuda").to(dtype)
    flat = torch.randn(3 * 2 * 64 + 1, generator=g, device="cuda").to(dtype)
    for out_grad in (w, w[:, :1].expand(3, 2, 64), w.transpose(0, 1).contiguous().transpose(0, 1),
                     flat[1:].view(3, 2, 64)):
        got, = torch.autograd.grad(y, leaf, out_grad, retain_graph=True)
        ref = rotate(out_grad, pos, f, inverse=not inverse, **kw)
        bound = rotate_bound(out_grad, pos, f, ref, dtype, **kw)
        assert got.dtype == dtype
        assert bool(((got[:, 2:4].cpu().double() - ref).abs() <= bound).all())
        assert not got[:, :2].any() and not got[:, 4:].any()
    # the gradient is linear in the output's gradient: its own is the turn again
    v = w.clone().requires_grad_()
    gx, = torch.autograd.grad(y, x, v, create_graph=True)
    again, = torch.autograd.grad(gx, v, w)
    assert torch.equal(again, pkv.rope(w, pos, f, inverse=inverse, **kw))
    # a lost gradient is refused, not passed over
    for out in (torch.empty_like(w), x):
        with pytest.raises(ValueError):
            pkv.rope(x, pos, f, out=out)
    with torch.no_grad():
        assert torch.equal(pkv.rope(x, pos, f, inverse=inverse, out=torch.empty_like(w), **kw), plain)
    # positions that changed since would give another gradient: torch refuses
    pos.add_(1)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, leaf, w)


def test_rope_gradient_captured(pkv):
    """Forward and backward captured on a side stream and replayed over new inputs."""
    g = gen(42)
    f, _ = pkv.rope_frequencies(64)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    x = torch.randn(9, 4, 64, generator=g, device="cuda").bfloat16()
    w = torch.randn(9, 4, 64, generator=g, device="cuda").bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        leaf = x.detach().requires_grad_()
        y = pkv.rope(leaf, pos, f)
        grad, = torch.autograd.grad(y, leaf, w)
    torch.cuda.synchronize()
    w.mul_(-2.0)
    pos.add_(70)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y.detach(), pkv.rope(x, pos, f))
    assert torch.equal(grad, pkv.rope(w, pos, f, inverse=True))
    assert pkv.read_device_status() == 0


@pytest.mark.parametrize("S,hkv,group,d,n,pb", [(3, 3, 4, 128, 700, 8), (16, 2, 8, 64, 2000, 16),
                                                (2, 1, 1, 64, 5000, 4), (5, 4, 2, 128, 90, 0)])
def test_decode_weights_steps_back_to_back(pkv, S, hkv, group, d, n, pb):
    """Steps that start before the one before them has ended, over growing contexts and rows
    whose ends share cache lines, against the same steps one at a time: the same bits."""
    g = gen(n)
    blocks, W = -(-n // 16), n + 7
    kp = torch.randn(S * blocks, hkv, 16, d, generator=g, device="cuda").bfloat16()
    vp = torch.randn(S * blocks, hkv, 16, d, generator=g, device="cuda").bfloat16()
    table = torch.randperm(S * blocks, generator=g, device="cuda").view(S, -1).to(torch.int32)
    lens = torch.randint(n // 2, n - 24, (S,), generator=g, device="cuda", dtype=torch.int32)
    w0 = torch.rand(S, hkv, W, generator=g, device="cuda")
    q = torch.randn(24, S, hkv * group, d, generator=g, device="cuda").bfloat16()
    kn = torch.randn(24, S, hkv, d, generator=g, device="cuda").bfloat16()
    ids = torch.randperm(S, generator=g, device="cuda").to(torch.int32)
    need = pkv.decode_weights_workspace_bytes(kp, S, hkv * group, n, pb)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def steps(pause):
        k, v, w, cl = kp.clone(), vp.clone(), w0.clone(), lens.clone()
        out = torch.empty_like(q)
        for i in range(24):
            cl.add_(1)
            for new, decay in ((kn[i], 0.9), (None, 0.99)):
                pkv.paged_decode_weights(q[i], k, v, table, cl, d ** -0.5, w, max_context=n,
                                         k_new=new, v_new=new, row_ids=ids, decay=decay,
                                         partition_blocks=pb, out=out[i], workspace=ws)
                if pause:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return out, w, k

    want = steps(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(steps(False), want))
    assert pkv.read_device_status() == 0


@pytest.mark.parametrize("reqs,d,hkv,group,new,n", [(50, 64, 4, 2, 40, 300), (50, 128, 4, 2, 40, 300),
                                                    (2, 128, 4, 2, 40, 300), (70, 64, 2, 8, 9, 130),
                                                    (9, 128, 8, 1, 200, 1000)])
def test_prefill_weights_give_the_same_bits(pkv, reqs, d, hkv, group, new, n):
    """Query and key tiles that end inside, so that rows and keys beyond them are whatever shared
    memory held: the same call gives the same bits, whatever ran before it and whatever the
    padding is."""
    g = gen(52)
    blocks = -(-n // 16)
    kp = torch.randn(reqs * blocks, hkv, 16, d, generator=g, device="cuda").bfloat16()
    table = torch.randperm(reqs * blocks, generator=g, device="cuda").view(reqs, -1).to(torch.int32)
    q = torch.randn(reqs * new, hkv * group, d, generator=g, device="cuda").bfloat16()
    cached, news = i32([n - new] * reqs), i32([new] * reqs)
    off = i32([new * i for i in range(reqs + 1)])

    def call(q, kp):
        w = torch.zeros(reqs, hkv, n, device="cuda")
        pkv.paged_prefill_weights(q, kp, table, cached, news, off, d ** -0.5, w, max_new=new,
                                  max_context=n)
        return w

    want = call(q, kp)
    # wild values in tiles of another call, which stay behind in shared memory
    wild = torch.where(torch.rand(kp.shape, generator=g, device="cuda") < 0.5, 1e30, -1e30).bfloat16()
    for other in (None, wild, kp):
        if other is not None:
            call(q * 100, other)
        for _ in range(8):
            assert torch.equal(call(q, kp), want)
    # the last request's neighbours are not its own: longer arrays, wild rows behind them
    longer = torch.cat([q, torch.full_like(q[:new], 1e30)])
    assert torch.equal(call(longer, kp), want)
    assert pkv.read_device_status() == 0


@pytest.mark.parametrize("stall", ["1", "2"])
@pytest.mark.parametrize("reqs,d", [(2, 128), (50, 64)])   # an item a CTA; items from the counter
def test_prefill_weights_after_a_timeout(pkv, monkeypatch, stall, reqs, d):
    """A wait of either pass that runs out (its copies all land, but its barrier waits for 16
    bytes more) is reported within a few seconds, and the next call is right."""
    g = gen(51)
    hkv, group, new, n = 4, 2, 40, 300
    blocks = -(-n // 16)
    kp = torch.randn(reqs * blocks, hkv, 16, d, generator=g, device="cuda").bfloat16()
    table = torch.randperm(reqs * blocks, generator=g, device="cuda").view(reqs, -1).to(torch.int32)
    q = torch.randn(reqs * new, hkv * group, d, generator=g, device="cuda").bfloat16()
    cached, news = i32([n - new] * reqs), i32([new] * reqs)
    off = i32([new * i for i in range(reqs + 1)])
    need = pkv.prefill_weights_workspace_bytes(kp, reqs, hkv * group, new, n)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def call():
        w = torch.zeros(reqs, hkv, n, device="cuda")
        pkv.paged_prefill_weights(q, kp, table, cached, news, off, d ** -0.5, w, max_new=new,
                                  max_context=n, workspace=ws)
        return w

    want = call()
    assert pkv.read_device_status() == 0
    total = want.double().sum(-1)                       # each row's probabilities add up to 1
    assert float((total - new * group).abs().max()) < 1e-3 * new * group
    monkeypatch.setenv("PKV_TEST_PREFILL_WEIGHTS_STALL", stall)
    call()
    assert pkv.read_device_status() == 4
    monkeypatch.delenv("PKV_TEST_PREFILL_WEIGHTS_STALL")
    assert torch.equal(call(), want)
    assert pkv.read_device_status() == 0
