"""Host side of the operators around a shrinking cache: rotary frequencies against their
formulas, private copies and truncation in the block allocator, and the argument checks of
the device calls (fake pointers: nothing may be launched)."""
import ctypes
import math

import pytest
import torch

OK, INVALID, UNSUPPORTED, NOMEM, NOT_FOUND = 0, 1, 2, 6, 7
A, A2 = 0x10000, 0x4000000
U = 0x10008


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_58_gb300 import build
    build.build()
    import paged_kv_cache_58_gb300 as m
    return m


# ------------------------------------------------------------------ frequencies

def plain(r, theta):
    return [theta ** (-2 * i / r) for i in range(r // 2)]


def close(got, want):
    assert len(got) == len(want)
    for g, w in zip(got.tolist(), want):
        assert abs(g - w) <= 1e-14 * abs(w), (g, w)


@pytest.mark.parametrize("r,theta", [(16, 10000.0), (64, 10000.0), (96, 1e6), (128, 500000.0)])
def test_plain_and_scaled_frequencies(pkv, r, theta):
    f, s = pkv.rope_frequencies(r, theta, device="cpu")
    assert s == 1.0 and f.dtype == torch.float64
    close(f, plain(r, theta))
    f, s = pkv.rope_frequencies(r, theta, scaling="linear", factor=4, device="cpu")
    assert s == 1.0
    close(f, [x / 4 for x in plain(r, theta)])
    f, _ = pkv.rope_frequencies(r, theta, scaling="ntk", factor=4, device="cpu")
    close(f, plain(r, theta * 4 ** (r / (r - 2))))
    # the highest frequency is kept, the lowest divided by the factor
    assert abs(float(f[-1]) * 4 / plain(r, theta)[-1] - 1) < 1e-12 and float(f[0]) == 1.0


@pytest.mark.parametrize("kind,low,high", [("llama3", 1, 4), ("yarn", 1, 32), ("yarn", 2, 20)])
def test_banded_frequencies(pkv, kind, low, high):
    r, theta, factor, trained = 128, 500000.0, 8.0, 8192
    kw = {} if (kind, low, high) in (("llama3", 1, 4), ("yarn", 1, 32)) else dict(low=low, high=high)
    f, s = pkv.rope_frequencies(r, theta, scaling=kind, factor=factor,
                                original_context=trained, device="cpu", **kw)
    want = []
    for x in plain(r, theta):
        wavelength = 2 * math.pi / x
        if wavelength < trained / high:
            want.append(x)
        elif wavelength > trained / low:
            want.append(x / factor)
        else:
            t = (trained / wavelength - low) / (high - low)
            want.append((1 - t) * x / factor + t * x)
    for g, w in zip(f.tolist(), want):
        assert abs(g - w) <= 1e-12 * w
    assert s == (pytest.approx(0.1 * math.log(factor) + 1, rel=1e-7) if kind == "yarn" else 1.0)


def test_frequency_refusals(pkv):
    def code(*a, **k):
        with pytest.raises(pkv.PkvError) as e:
            pkv.rope_frequencies(*a, device="cpu", **k)
        return e.value.status

    assert code(0) == INVALID and code(7) == INVALID and code(-2) == INVALID
    assert code(64, 0.0) == INVALID and code(64, float("nan")) == INVALID
    assert code(64, scaling="linear", factor=0.5) == INVALID
    assert code(2, scaling="ntk", factor=2) == INVALID
    assert code(64, scaling="llama3", factor=8) == INVALID                  # no trained context
    assert code(64, scaling="yarn", factor=8, original_context=4096, low=4, high=4) == INVALID
    with pytest.raises(ValueError):
        pkv.rope_frequencies(64, scaling="other", device="cpu")
    out = (ctypes.c_double * 32)()
    sc = pkv.RopeScaling(9, 1.0, 1.0, 4.0, 1.0)
    assert pkv.lib().pkv_rope_frequencies(out, None, 64, 1e4, ctypes.byref(sc)) == UNSUPPORTED
    assert pkv.lib().pkv_rope_frequencies(out, None, 64, 1e4, None) == OK    # plain, no scale asked


# ------------------------------------------------------------------ allocator

@pytest.mark.parametrize("bs", [16, 32])
def test_privatize_and_truncate(pkv, bs):
    a = pkv.BlockAllocator(16, bs)
    a.add_seq(1, 4 * bs + 3)
    a.fork(1, 2)
    t1 = a.block_table([1], 5)[0].tolist()
    assert a.num_free == 11
    assert a.privatize(2, 0) == []
    pairs = a.privatize(2, 2 * bs + 1)           # the first three blocks
    assert [p[0] for p in pairs] == t1[:3]
    t2 = a.block_table([2], 5)[0].tolist()
    assert [p[1] for p in pairs] == t2[:3] and t2[3:] == t1[3:]
    assert a.block_table([1], 5)[0].tolist() == t1          # the sibling keeps its blocks
    assert a.num_free == 8
    assert a.privatize(2, 2 * bs + 1) == []                 # private already
    a.truncate(2, 2 * bs + 1)
    assert a.seq_len(2) == 2 * bs + 1 and a.seq_num_blocks(2) == 3
    assert a.num_free == 8 and all(a.refcount(b) == 1 for b in t1)
    a.truncate(1, 0)
    assert a.seq_len(1) == 0 and a.num_free == 13
    slots, cow = a.append(2, 1)                             # the next token follows
    assert cow is None and slots == [t2[2] * bs + 1]
    a.free_seq(1), a.free_seq(2)
    assert a.num_free == 16


def test_privatize_and_truncate_refusals(pkv):
    a = pkv.BlockAllocator(6, 16)
    a.add_seq(1, 64)
    a.fork(1, 2)
    before = a.block_table([1, 2], 4)

    def code(f, *x):
        with pytest.raises(pkv.PkvError) as e:
            f(*x)
        return e.value.status

    assert code(a.privatize, 2, 65) == INVALID
    assert code(a.privatize, 2, -1) == INVALID
    assert code(a.privatize, 9, 1) == NOT_FOUND
    assert code(a.privatize, 2, 64) == NOMEM                # 4 shared, 2 free
    n = ctypes.c_int(7)
    pairs = (ctypes.c_int32 * 2)()
    assert pkv.lib().pkv_alloc_privatize(a._h, 2, 32, pairs, 1, ctypes.byref(n)) == INVALID
    assert code(a.truncate, 2, 65) == INVALID
    assert code(a.truncate, 2, -1) == INVALID
    assert code(a.truncate, 9, 0) == NOT_FOUND
    assert torch.equal(a.block_table([1, 2], 4), before) and a.num_free == 2


def test_privatize_of_absurd_lengths(pkv):
    """Lengths no sequence has are refused without room being made for their pairs."""
    a = pkv.BlockAllocator(6, 16)
    a.add_seq(1, 64)
    for n in (2 ** 40, 2 ** 62):
        with pytest.raises(pkv.PkvError) as e:
            a.privatize(1, n)
        assert e.value.status == INVALID
    a.fork(1, 2)
    a.truncate(1, 16)
    assert len(a.privatize(2, 64)) == 1   # what the other still holds
    assert a.num_free == 1


def test_truncate_and_privatize_respect_the_prefix_cache(pkv):
    """Blocks that a prefix cache holds are shared: an eviction copies them first, and a
    truncation leaves them cached."""
    a = pkv.BlockAllocator(8, 16)
    pc = pkv.PrefixCache(a)
    toks = list(range(48))
    a.add_seq(1, 48)
    assert pc.insert(1, toks) == 3
    old = a.block_table([1], 3)[0].tolist()
    assert [p[0] for p in a.privatize(1, 20)] == old[:2]
    a.truncate(1, 20)
    assert pc.match(toks) == old
    assert [a.refcount(b) for b in old] == [1, 1, 1]
    pc.close()


# ------------------------------------------------------------------ argument checks

fake = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers")


def desc(pkv, nb=64, bs=16, hkv=8, d=128, dtype=1):
    return pkv.PoolDesc(nb, bs, hkv, d, dtype)


@fake
def test_rope_checks(pkv):
    def r(dtype=1, out=A2, os=1024, x=A, xs=1024, pos=A, f=A, rot=128, T=4, H=8, d=128):
        return pkv.lib().pkv_rope(dtype, out, os, x, xs, pos, f, rot, 0, 0, 1.0, T, H, d, None)

    assert r(T=0) == OK
    assert r(T=-1) == INVALID and r(H=0) == INVALID and r(rot=0) == INVALID
    assert r(dtype=2) == UNSUPPORTED
    assert r(d=96, rot=96) == UNSUPPORTED
    assert r(rot=24) == UNSUPPORTED           # not a multiple of 16
    assert r(rot=144) == INVALID              # more than the head
    assert r(out=None) == INVALID and r(x=None) == INVALID and r(pos=None) == INVALID
    assert r(f=None) == INVALID
    assert r(out=U) == INVALID and r(x=U) == INVALID
    assert r(os=1016) == INVALID              # tokens of the output overlap
    assert r(os=1028) == INVALID              # not whole 16-byte chunks
    assert r(xs=1028) == INVALID and r(xs=-1024) == INVALID
    assert r(T=1 << 31) == UNSUPPORTED
    assert r(pos=0x10002) == INVALID and r(f=0x10004) == INVALID


@fake
def test_rope_append_checks(pkv):
    def r(d=None, kp=A, vp=A, sl=A, qo=A2, qos=4096, q=A, qs=6144, k=A, ks=6144, v=A, vs=6144,
          pos=A, f=A, rot=64, T=4, hq=32):
        return pkv.lib().pkv_rope_append(ctypes.byref(d or desc(pkv)), kp, vp, sl, qo, qos, q, qs,
                                         k, ks, v, vs, pos, f, rot, 0, 1.0, T, hq, None)

    assert r(T=0) == OK
    assert r(d=desc(pkv, bs=8)) == UNSUPPORTED
    assert r(rot=8) == UNSUPPORTED and r(rot=256) == INVALID
    for name in ("kp", "vp", "sl", "qo", "q", "k", "v", "pos", "f"):
        assert r(**{name: None}) == INVALID, name
    for name in ("kp", "vp", "qo", "q", "k", "v"):
        assert r(**{name: U}) == INVALID, name
    assert r(qos=4088) == INVALID
    for name in ("qs", "ks", "vs"):
        assert r(**{name: 6148}) == INVALID, name
    assert r(T=-1) == INVALID and r(hq=0) == INVALID


@fake
def test_decode_weights_checks(pkv):
    lib = pkv.lib()

    def w(d=None, kn=None, vn=None, mbs=8, max_ctx=100, S=2, hq=32, wt=A, stride=128, rows=2,
          ids=None, decay=1.0, ws=A, wsb=1 << 24, pb=0):
        return lib.pkv_paged_decode_weights(ctypes.byref(d or desc(pkv)), A, A, A, A, kn, vn, A,
                                            mbs, A, max_ctx, S, hq, 0.1, pb, wt, stride, ids, rows,
                                            decay, ws, wsb, None)

    assert w(S=0) == OK
    assert w(kn=A) == INVALID and w(vn=A) == INVALID          # both or neither
    assert w(kn=U, vn=A) == INVALID
    assert w(wt=None) == INVALID
    assert w(stride=99) == INVALID                            # shorter than the context
    assert w(rows=1) == INVALID                               # fewer rows than sequences
    assert w(rows=0, ids=A) == INVALID
    assert w(decay=-0.1) == INVALID and w(decay=1.5) == INVALID
    assert w(decay=float("nan")) == INVALID
    assert w(hq=24) == UNSUPPORTED and w(d=desc(pkv, d=96)) == UNSUPPORTED
    need = lib.pkv_paged_decode_weights_workspace_bytes(ctypes.byref(desc(pkv)), 2, 32, 100, 0)
    assert need >= 2 * 32 * 100 * 4
    assert w(wsb=need - 1) == NOMEM and w(ws=None) == NOMEM and w(ws=U) == NOMEM
    # one partition needs a workspace too: the scores go there
    one = lib.pkv_paged_decode_weights_workspace_bytes(ctypes.byref(desc(pkv)), 2, 32, 100, 7)
    assert w(pb=7, wsb=one - 1) == NOMEM
    # a partition longer than the context needs no more than one of the context
    assert lib.pkv_paged_decode_weights_workspace_bytes(ctypes.byref(desc(pkv)), 2, 32, 100,
                                                        1 << 30) == one
    ask = lib.pkv_paged_decode_weights_workspace_bytes
    assert ask(ctypes.byref(desc(pkv)), 0, 32, 100, 0) == 0
    assert ask(ctypes.byref(desc(pkv, d=96)), 2, 32, 100, 0) == 0


@fake
def test_prefill_weights_checks(pkv):
    lib = pkv.lib()

    def p(d=None, q=A, kp=A, bt=A, mbs=8, cl=A, nl=A, qo=A, R=2, N=10, max_new=5, max_ctx=100,
          hq=32, scale=0.1, window=0, wt=A, stride=128, rows=2, ids=None, decay=1.0, ws=A,
          wsb=1 << 24):
        return lib.pkv_paged_prefill_weights(ctypes.byref(d or desc(pkv)), q, kp, bt, mbs, cl, nl,
                                             qo, R, N, max_new, max_ctx, hq, scale, window, wt,
                                             stride, ids, rows, decay, ws, wsb, None)

    assert p(R=0) == OK and p(N=0) == OK and p(max_new=0) == OK
    assert p(R=-1) == INVALID and p(window=-1) == INVALID and p(scale=0.0) == INVALID
    for name in ("q", "kp", "bt", "cl", "nl", "qo", "wt"):
        assert p(**{name: None}) == INVALID, name
    assert p(q=U) == INVALID and p(kp=U) == INVALID
    assert p(max_ctx=129) == INVALID                          # beyond the table
    assert p(stride=99) == INVALID and p(rows=1) == INVALID and p(decay=2.0) == INVALID
    assert p(hq=20) == INVALID and p(hq=24) == UNSUPPORTED
    need = lib.pkv_paged_prefill_weights_workspace_bytes(ctypes.byref(desc(pkv)), 2, 32, 5, 100, 0)
    assert need >= 2 * 8 * 5 * 4 * 8
    assert p(wsb=need - 1) == NOMEM and p(ws=None) == NOMEM and p(ws=U) == NOMEM


@fake
def test_evict_checks(pkv):
    lib = pkv.lib()

    def e(d=None, kp=A, vp=A, bt=A, mbs=8, cl=A, max_ctx=100, S=2, bu=A, sinks=0, recent=0,
          seen=None, tracked=None, w=A, wo=A, po=A, poo=A, stride=128, ids=None, rows=2, nl=A2,
          ws=A, wsb=1 << 24):
        return lib.pkv_evict(ctypes.byref(d or desc(pkv)), kp, vp, bt, mbs, cl, max_ctx, S, bu,
                             sinks, recent, seen, tracked, w, wo, po, poo, stride, ids, rows, nl,
                             ws, wsb, None)

    assert e(S=0) == OK
    assert e(S=-1) == INVALID and e(sinks=-1) == INVALID and e(recent=-1) == INVALID
    for name in ("kp", "vp", "bt", "cl", "bu", "w", "wo", "po", "poo", "nl"):
        assert e(**{name: None}) == INVALID, name
    assert e(kp=U) == INVALID and e(max_ctx=129) == INVALID and e(stride=99) == INVALID
    assert e(rows=1) == INVALID
    assert e(wo=A + 16) == INVALID and e(poo=A + 4096) == INVALID   # overlap, not the same
    for name in ("cl", "bu", "seen", "tracked", "ids"):
        assert e(**{name: A2}) == INVALID, name                     # new_lens is an input
        assert e(**{name: A2 + 4}) == INVALID, name                 # overlaps one by a value
    for name in ("cl", "bu", "seen", "tracked", "ids", "nl", "po", "poo", "wo", "bt"):
        assert e(**{name: 0x9000002}) == INVALID, name              # not on 4 bytes
    assert e(max_ctx=(1 << 20) + 1, mbs=1 << 17, stride=1 << 21) == UNSUPPORTED
    need = lib.pkv_evict_workspace_bytes(ctypes.byref(desc(pkv)), 2, 100)
    assert need > 0
    assert e(wsb=need - 1) == NOMEM and e(ws=None) == NOMEM and e(ws=U) == NOMEM
    assert e(S=70000, rows=70000) == UNSUPPORTED


def test_python_refusals_before_the_library(pkv):
    """Shapes, types and devices are checked on the host before any address is passed on."""
    q = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        pkv.rope(q, torch.zeros(2, dtype=torch.int32), torch.ones(32, dtype=torch.float64))
    pool = torch.zeros(4, 4, 16, 64)
    with pytest.raises(ValueError):
        pkv.evict(pool, pool, torch.zeros(2, 1, dtype=torch.int32), None, None, q, q,
                  max_context=4)
