"""Host side of the quantised cache: sizes of its arrays, the argument checks of the device calls
(fake pointers: nothing may be launched), and the 64-bit rounding that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

from tests.quant_refs import e4m3_values, held, kept

OK, INVALID, UNSUPPORTED, NOMEM = 0, 1, 2, 6
A, U = 0x10000, 0x10008


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_58_gb300 import build
    build.build()
    import paged_kv_cache_58_gb300 as m
    return m


def cache(pkv, nb=64, bs=16, hkv=8, d=128, fmt=0, k=A, v=A, ks=A, vs=A):
    return pkv.QuantCacheDesc(nb, bs, hkv, d, fmt, k, v, ks, vs)


def test_sizes(pkv):
    lib = pkv.lib()

    def both(**kw):
        c = ctypes.byref(cache(pkv, **kw))
        return lib.pkv_quant_codes_bytes(c), lib.pkv_quant_scales_bytes(c)

    assert both() == (64 * 8 * 16 * 128, 64 * 8 * 16)
    assert both(bs=32, d=64) == (64 * 8 * 32 * 64, 64 * 8 * 32)
    assert both(fmt=1) == (64 * 8 * 16 * 64, 64 * 8 * (128 + 16))
    assert both(fmt=1, bs=32, d=64, hkv=3) == (64 * 3 * 32 * 32, 64 * 3 * 2 * (64 + 16))
    assert both(k=0, v=0, ks=0, vs=0) == both()             # the pointers are not looked at
    for wrong in (dict(nb=0), dict(nb=-1), dict(bs=8), dict(bs=48), dict(hkv=0), dict(d=96),
                  dict(fmt=2), dict(fmt=-1), dict(hkv=70000), dict(nb=1 << 40),
                  dict(nb=(1 << 31) // 128 + 1)):
        assert both(**wrong) == (0, 0), wrong
    assert lib.pkv_quant_codes_bytes(None) == 0
    assert both(nb=((1 << 31) - 1) // 128)[0] > 0           # the largest


fake = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers")


@fake
@pytest.mark.parametrize("name", ["append", "read"])
def test_rows_checks(pkv, name):
    fn = getattr(pkv.lib(), f"pkv_kv_{name}_quant")
    B = 1 << 30

    def r(c=None, sl=A, dt=1, k=A, ks=1024, v=B, vs=1024, T=4, none=False):
        return fn(None if none else ctypes.byref(c or cache(pkv)), sl, dt, k, ks, v, vs, T, None)

    assert r(T=0) == OK and r(T=0, k=None, v=None, sl=None) == OK
    assert r(T=-1) == INVALID and r(none=True) == INVALID
    assert r(c=cache(pkv, fmt=5)) == UNSUPPORTED and r(c=cache(pkv, d=80)) == UNSUPPORTED
    assert r(c=cache(pkv, bs=64)) == UNSUPPORTED and r(c=cache(pkv, nb=0)) == INVALID
    assert r(dt=2) == UNSUPPORTED
    for what in ("sl", "k", "v"):
        assert r(**{what: None}) == INVALID, what
    for what in ("k", "v", "ks", "vs"):
        assert r(c=cache(pkv, **{what: 0})) == INVALID, what
        assert r(c=cache(pkv, **{what: U})) == INVALID, what
    assert r(k=U) == INVALID and r(v=U) == INVALID and r(sl=0x10004) == INVALID
    for what in ("ks", "vs"):
        assert r(**{what: 1028}) == INVALID, what           # not whole 16 bytes
        assert r(**{what: -1024}) == INVALID, what
    assert r(T=1 << 28) == UNSUPPORTED                      # 2^31 rows
    if name == "read":
        assert r(ks=1016) == INVALID and r(vs=512) == INVALID       # tokens in one another
        assert r(v=A) == INVALID and r(v=A + 1024) == INVALID       # K's rows in V's
        assert r(ks=2048, vs=2048, v=A + 1024) == INVALID           # half a row


@fake
@pytest.mark.parametrize("name", ["quantize", "dequantize"])
def test_blocks_checks(pkv, name):
    fn = getattr(pkv.lib(), f"pkv_{name}_blocks")

    def r(c=None, p=None, k=A, v=A, pairs=A, n=4, **pool):
        d = pkv.PoolDesc(*[{**dict(nb=64, bs=16, hkv=8, d=128, dt=1), **pool}[x]
                           for x in ("nb", "bs", "hkv", "d", "dt")])
        return fn(ctypes.byref(c or cache(pkv)), ctypes.byref(d), k, v, pairs, n, None)

    assert r(n=0) == OK and r(n=0, pairs=None) == OK
    assert r(n=-1) == INVALID
    assert r(bs=32) == INVALID and r(hkv=4) == INVALID and r(d=64) == INVALID
    assert r(dt=3) == UNSUPPORTED and r(c=cache(pkv, fmt=9)) == UNSUPPORTED
    assert r(k=None) == INVALID and r(v=None) == INVALID and r(pairs=None) == INVALID
    assert r(k=U) == INVALID and r(pairs=0x10002) == INVALID
    assert r(c=cache(pkv, ks=U)) == INVALID and r(c=cache(pkv, v=0)) == INVALID
    assert r(n=1 << 24) == UNSUPPORTED                      # 2^31 rows


@fake
def test_copy_checks(pkv):
    def r(c=None, pairs=A, n=3):
        return pkv.lib().pkv_copy_blocks_quant(ctypes.byref(c or cache(pkv)), pairs, n, None)

    assert r(n=0) == OK and r(n=0, pairs=None) == OK
    assert r(n=-1) == INVALID and r(pairs=None) == INVALID and r(pairs=0x10002) == INVALID
    assert r(c=cache(pkv, k=U)) == INVALID and r(c=cache(pkv, bs=24)) == UNSUPPORTED


@fake
def test_decode_checks(pkv):
    lib = pkv.lib()

    def r(c=None, dt=1, out=A, q=A, kn=None, vn=None, bt=A, mbs=64, cl=A, ctx=1000, S=2, hq=32,
          pb=0, ws=A, wsb=1 << 30):
        return lib.pkv_paged_decode_quant(ctypes.byref(c or cache(pkv)), dt, out, q, kn, vn, bt,
                                          mbs, cl, ctx, S, hq, 0.1, pb, ws, wsb, None)

    assert r(S=0) == OK
    assert r(S=-1) == INVALID and r(hq=0) == INVALID and r(pb=-1) == INVALID
    assert r(dt=2) == UNSUPPORTED and r(c=cache(pkv, fmt=3)) == UNSUPPORTED
    for what in ("out", "q", "bt", "cl"):
        assert r(**{what: None}) == INVALID, what
    for what in ("out", "q"):
        assert r(**{what: U}) == INVALID, what
    assert r(bt=0x10002) == INVALID and r(cl=0x10001) == INVALID
    assert r(kn=A) == INVALID and r(vn=A) == INVALID        # both or neither
    assert r(kn=A, vn=U) == INVALID
    assert r(c=cache(pkv, vs=0)) == INVALID
    assert r(ctx=0) == INVALID and r(ctx=64 * 16 + 1) == INVALID and r(mbs=0) == INVALID
    assert r(hq=20) == INVALID                              # not a multiple of the kv heads
    assert r(hq=24) == UNSUPPORTED and r(hq=128) == UNSUPPORTED     # groups of 3 and of 16
    assert r(S=65536) == UNSUPPORTED
    assert r(mbs=1 << 26) == UNSUPPORTED and r(pb=1 << 30, mbs=64) != OK
    ask = lib.pkv_paged_decode_quant_workspace_bytes
    c = ctypes.byref(cache(pkv))
    need = ask(c, 2, 32, 1000, 8)
    assert need > 0
    assert r(pb=8, wsb=need - 1) == NOMEM and r(pb=8, ws=None) == NOMEM and r(pb=8, ws=U) == NOMEM
    assert ask(c, 2, 32, 1000, 63) == 0                     # one partition: no workspace
    assert ask(c, 0, 32, 1000, 0) == 0 and ask(ctypes.byref(cache(pkv, d=96)), 2, 32, 1000, 0) == 0
    assert r(pb=1, ctx=20000, mbs=2000) == UNSUPPORTED      # more than 1024 partitions
    # the library's own choice stays within them, whatever the length
    for S in (1, 3, 64, 4096):
        for hkv in (1, 2, 8, 64):
            for ctx in (1, 17, 4096, 131072, 1 << 20, 1 << 28):
                d = ctypes.byref(cache(pkv, hkv=hkv))
                rows = S * hkv
                assert ask(d, S, hkv, ctx, 0) <= rows * 512 * (128 + 3) * 4 + 64


def test_python_checks(pkv):
    cpu = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        pkv.QuantCache(cpu, cpu, cpu, cpu)                  # not on a GPU
    with pytest.raises(ValueError):
        pkv.QuantCache(cpu, cpu, cpu, cpu, format="fp6")
    with pytest.raises(ValueError):
        pkv.QuantCache(cpu[0], cpu, cpu, cpu)
    with pytest.raises(ValueError):
        pkv.QuantCache.empty(2, 2, 64, format="int4", device="cpu")


# ------------------------------------------------------------------ the reference itself

def test_reference_rounding():
    """The tests' own form, at values worked out by hand."""
    v = e4m3_values()
    assert v[0x7e] == 448 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and v[0xbc] == -1.5
    assert math.isnan(v[0x7f]) and math.isnan(v[0xff])

    def row(*x):
        r = torch.zeros(64)
        r[:len(x)] = torch.tensor(x)
        return r

    # largest 448: unit 1.  17 lies between 16 and 18 (tie to 16's even code), 19 between 18 and 20
    got = kept(row(448.0, 17.0, 19.0, -17.1, 0.001, 0.00097, 2.0 ** -10), "fp8")
    assert got[:7].tolist() == [448, 16, 20, -18, 2.0 ** -9 * 1, 0, 0]
    # one more than 448 doubles the unit
    assert kept(row(449.0, 17.0), "fp8")[:2].tolist() == [448, 16]
    assert kept(row(449.0, 3.0 * 2 ** -9), "fp8")[1] == 2.0 ** -8 * 2   # 1.5 units: to the even
    # fp4: largest 6 -> unit 2^-8 (2688 2^-9 < 6 <= 2688 2^-8), scale 256, codes 6 3 ...
    got = kept(row(6.0, 3.0, 2.5, 3.5, 5.0, 0.25, 0.75, -1.25), "fp4")
    assert got[:8].tolist() == [6, 3, 2, 4, 4, 0, 1, -1]
    nan = kept(row(1.0, float("nan"), 2.0), "fp4")
    assert nan[:16].isnan().all() and not nan[16:].isnan().any()
    nan = kept(row(1.0, float("nan"), 2.0), "fp8")
    assert nan[1].isnan() and nan[0] == 1 and nan[2] == 2
    inf = kept(row(float("inf"), -float("inf"), 1.0), "fp8")
    assert inf[:3].tolist() == [448 * 2.0 ** 90, -448 * 2.0 ** 90, 0]
    assert kept(row(2.0 ** -105), "fp8")[0] == 0 and kept(row(), "fp4").abs().sum() == 0


def test_reference_layout():
    """A block whose bytes say where they lie."""
    codes = torch.zeros(1, 1, 32, 32, dtype=torch.uint8)
    codes[0, 0, 17, 3] = 0x52                               # elements 6 (code 2: 1.0) and 7 (3.0)
    scales = torch.zeros(1, 1, 160, dtype=torch.uint8)
    scales[0, 0, 80 + 64 + 1] = 127 + 3                     # token 17's exponent
    one = 0x38
    k = scales.clone()
    k[0, 0, 80 + 1 * 4 + 0] = one                           # K: [token 1][group 0] of the second run
    assert held(codes, k, "fp4", False)[0, 0, 17, 5:9].tolist() == [0, 8, 24, 0]
    v = scales.clone()
    v[0, 0, 80 + 0 * 16 + 0 * 4 + 1] = one                  # V: [0][group 0][token 1]
    assert held(codes, v, "fp4", True)[0, 0, 17, 5:9].tolist() == [0, 8, 24, 0]
