"""Calls of the quantised cache that its documentation allows and the other tests do not make:
rows 16 bytes off, the same block twice, captured moves, other streams, many heads."""
import threading

import pytest
import torch

from tests.quant_refs import decode_bound, held, kept, rows_of

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("off", ["rows", "tokens"])
def test_rows_16_bytes_off(pkv, fmt, dtype, off):
    """Rows that begin at odd multiples of 16 bytes, all of them or every other token."""
    T, hkv, d = 37, 3, 64
    unit = 16 // dtype.itemsize
    step = 2 * hkv * d + (unit if off == "tokens" else 2 * unit)

    def rows(x):
        return x[unit if off == "rows" else 0:].as_strided((T, 2 * hkv, d), (step, d, 1))

    flat = torch.randn((T + 1) * step, generator=gen(1), device="cuda").to(dtype)
    x = rows(flat)
    c = pkv.QuantCache.empty(4, hkv, d, format=fmt)
    slots = torch.randperm(64, generator=gen(2), device="cuda")[:T]
    pkv.kv_append_quant(c, slots, x[:, :hkv], x[:, hkv:])
    assert torch.equal(rows_of(held(c.k, c.k_scales, fmt, False), slots), kept(x[:, :hkv], fmt))
    assert torch.equal(rows_of(held(c.v, c.v_scales, fmt, True), slots), kept(x[:, hkv:], fmt))
    back = torch.full_like(flat, 5.0)
    y = rows(back)
    pkv.kv_read_quant(c, slots, k_out=y[:, :hkv], v_out=y[:, hkv:])
    assert torch.equal(y.double().cpu(), torch.cat((kept(x[:, :hkv], fmt), kept(x[:, hkv:], fmt)),
                                                   1).to(dtype).double())
    y.fill_(5.0)
    assert bool((back == 5.0).all())              # nothing between the rows was written
    # pools 16 bytes off
    pool = torch.zeros(2 * hkv * 16 * d + unit, device="cuda", dtype=dtype)[unit:].view(2, hkv, 16,
                                                                                       d)
    pool.copy_(torch.randn(pool.shape, generator=gen(3), device="cuda"))
    out = torch.zeros_like(pool)
    outk = torch.zeros(pool.numel() + unit, device="cuda", dtype=dtype)[unit:].view_as(pool)
    pkv.quantize_blocks(c, pool, pool, i32([[0, 3], [1, 2]]))
    pkv.dequantize_blocks(c, outk, out, i32([[3, 0], [2, 1]]))
    assert torch.equal(out, outk) and torch.equal(out.double().cpu(),
                                                  kept(pool, fmt).to(dtype).double())
    assert pkv.read_device_status() == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_types_write_the_same_bytes(pkv, fmt):
    """bf16 rows, and the same values as fp32."""
    x = torch.randn(50, 4, 128, generator=gen(4), device="cuda").bfloat16()
    x[7] *= 1e20
    a, b = (pkv.QuantCache.empty(4, 2, 128, format=fmt) for _ in range(2))
    for c in (a, b):
        for t in (c.k, c.v, c.k_scales, c.v_scales):
            t.zero_()
    slots = torch.arange(50, device="cuda")
    pkv.kv_append_quant(a, slots, x[:, :2], x[:, 2:])
    y = x.float()
    pkv.kv_append_quant(b, slots, y[:, :2], y[:, 2:])
    for name in ("k", "v", "k_scales", "v_scales"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_same_block_twice(pkv, fmt):
    """A source block for two destinations, and a table that names a block three times."""
    hkv, d = 2, 128
    c = pkv.QuantCache.empty(5, hkv, d, format=fmt)
    k, v = (torch.randn(16, hkv, d, generator=gen(s), device="cuda").bfloat16() for s in (5, 6))
    slots = 2 * 16 + torch.arange(16, device="cuda")
    pkv.kv_append_quant(c, slots, k, v)
    pkv.copy_blocks_quant(c, i32([[2, 0], [2, 4]]))
    kp = torch.zeros(3, hkv, 16, d, device="cuda", dtype=torch.bfloat16)
    vp = torch.zeros_like(kp)
    pkv.dequantize_blocks(c, kp, vp, i32([[2, 0], [2, 1], [4, 2]]))
    assert torch.equal(kp[0], kp[1]) and torch.equal(vp[0], vp[2])
    q = torch.randn(2, 8, d, generator=gen(7), device="cuda").bfloat16()
    out = pkv.paged_decode_quant(q, c, i32([[2, 2, 2], [0, 4, 2]]), i32([48, 48]), 0.1,
                                 max_context=48)
    one = pkv.paged_decode_quant(q[:1], c, i32([[2]]), i32([16]), 0.1, max_context=16)
    kk, vv = kept(k, fmt), kept(v, fmt)
    x = torch.einsum("hgd,nhd->hgn", q[0].cpu().double().view(hkv, -1, d), kk) * 0.1
    p = torch.softmax(x, -1)
    ref = torch.einsum("hgn,nhd->hgd", p, vv).reshape(8, d)
    bound = decode_bound(q[0].cpu().double(), kk, vv, p, ref, 0.1, torch.bfloat16)
    for got in (out[0], one[0]):
        assert bool(((got.double().cpu() - ref).abs() <= bound).all())
    assert pkv.read_device_status() == 0


def test_moves_captured_and_on_other_streams(pkv):
    """Append, freeze, copy and thaw recorded once and replayed with other rows; the same on a
    stream of its own while the default one is busy; and from two host threads."""
    hkv, d = 3, 64
    for fmt in ("fp8", "fp4"):
        c = pkv.QuantCache.empty(8, hkv, d, format=fmt)
        k = torch.zeros(20, hkv, d, device="cuda")
        v, pool = torch.zeros_like(k), torch.zeros(2, hkv, 16, d, device="cuda")
        out = torch.zeros(4, hkv, 16, d, device="cuda")
        out2 = torch.zeros_like(out)
        slots = torch.arange(20, device="cuda")
        to, copy, back = i32([[0, 4], [1, 5]]), i32([[4, 6]]), i32([[0, 0], [1, 1], [6, 2], [5, 3]])

        def step(stream=None):
            pkv.kv_append_quant(c, slots, k, v, stream=stream)
            pkv.quantize_blocks(c, pool, pool, to, stream=stream)
            pkv.copy_blocks_quant(c, copy, stream=stream)
            pkv.dequantize_blocks(c, out, out2, back, stream=stream)

        def right():
            want = torch.cat((kept(k, fmt), torch.zeros(12, hkv, d).double())).view(2, 16, hkv, d)
            got = out.double().cpu()
            return torch.equal(got[:2].transpose(1, 2).reshape(32, hkv, d)[:20],
                               want.reshape(32, hkv, d)[:20]) and \
                torch.equal(got[2:], kept(pool, fmt))

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        for seed in (1, 2, 3):
            for t in (k, v, pool):
                t.copy_(torch.randn(t.shape, generator=gen(seed), device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            assert right()
        k.copy_(torch.randn(k.shape, generator=gen(9), device="cuda"))
        s.wait_stream(torch.cuda.current_stream())
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(4):
            busy = busy @ busy * 1e-4
        step(stream=s)
        torch.cuda.synchronize()
        assert right()
        errors = []

        def host():
            try:
                st = torch.cuda.Stream()
                mine = pkv.QuantCache.empty(2, hkv, d, format=fmt)
                table, n = i32([[0, 1]]), i32([20])
                q = torch.randn(1, hkv, d, generator=gen(2), device="cuda")
                torch.cuda.synchronize()
                outs = []
                for _ in range(20):
                    pkv.kv_append_quant(mine, slots, k, v, stream=st)
                    outs.append(pkv.paged_decode_quant(q, mine, table, n, 0.1, max_context=32,
                                                       partition_blocks=1, stream=st))
                torch.cuda.synchronize()
                if not all(torch.equal(o, outs[0]) for o in outs):
                    errors.append("outputs differ")
            except Exception as e:   # noqa: BLE001 - shown by the assertion below
                errors.append(repr(e))

        threads = [threading.Thread(target=host) for _ in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not errors
        assert pkv.read_device_status() == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_many_heads_and_sequences(pkv, fmt):
    """40 kv heads of one query head each, 150 sequences, lengths from 1 on, tables wider than
    needed."""
    hkv, d, S = 40, 64, 150
    lens = [1 + (7 * i) % 45 for i in range(S)]
    c = pkv.QuantCache.empty(3 * S, hkv, d, format=fmt)
    table = torch.randperm(3 * S, generator=gen(1), device="cuda").int().view(S, 3)
    table = torch.cat((table, torch.full((S, 5), -1, device="cuda", dtype=torch.int32)),
                      1).contiguous()
    t = torch.arange(48, device="cuda")
    slots = torch.cat([table[i].long()[t[:n] // 16] * 16 + t[:n] % 16 for i, n in
                       enumerate(lens)])
    k, v = (torch.randn(sum(lens), hkv, d, generator=gen(s), device="cuda").bfloat16()
            for s in (2, 3))
    pkv.kv_append_quant(c, slots, k, v)
    q = torch.randn(S, hkv, d, generator=gen(4), device="cuda").bfloat16()
    out = pkv.paged_decode_quant(q, c, table, i32(lens), 0.125, max_context=45)
    assert pkv.read_device_status() == 0
    kk, vv = kept(k, fmt), kept(v, fmt)
    at = 0
    for i, n in enumerate(lens):
        ki, vi = kk[at:at + n], vv[at:at + n]
        at += n
        if i % 10:
            continue
        x = torch.einsum("hgd,nhd->hgn", q[i].cpu().double().view(hkv, 1, d), ki) * 0.125
        p = torch.softmax(x, -1)
        ref = torch.einsum("hgn,nhd->hgd", p, vi).reshape(hkv, d)
        bound = decode_bound(q[i].cpu().double(), ki, vi, p, ref, 0.125, torch.bfloat16)
        assert bool(((out[i].double().cpu() - ref).abs() <= bound).all()), i
