"""Arrays of a quantised cache and of a pool that share bytes, refused on the host (fake pointers:
nothing may be launched)."""
import ctypes

import pytest
import torch

INVALID = 1
G = 1 << 30

fake = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers")


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_58_gb300 import build
    build.build()
    import paged_kv_cache_58_gb300 as m
    return m


CODES = 64 * 8 * 16 * 128          # bytes of k_codes
SIDE = 64 * 8 * 16                 # of k_scales


def calls(pkv, k=1 * G, v=2 * G, ks=3 * G, vs=4 * G):
    """Every device call over a cache whose arrays lie there, with all else in order."""
    lib = pkv.lib()
    c = ctypes.byref(pkv.QuantCacheDesc(64, 16, 8, 128, 0, k, v, ks, vs))
    p = ctypes.byref(pkv.PoolDesc(64, 16, 8, 128, 1))
    A, B, C = 10 * G, 20 * G, 30 * G
    return {
        "append": lib.pkv_kv_append_quant(c, C, 1, A, 1024, B, 1024, 4, None),
        "read": lib.pkv_kv_read_quant(c, C, 1, A, 1024, B, 1024, 4, None),
        "quantize": lib.pkv_quantize_blocks(c, p, A, B, C, 4, None),
        "dequantize": lib.pkv_dequantize_blocks(c, p, A, B, C, 4, None),
        "copy": lib.pkv_copy_blocks_quant(c, C, 4, None),
        "decode": lib.pkv_paged_decode_quant(c, 1, A, B, None, None, C, 64, C, 1000, 2, 32, 0.1, 0,
                                             40 * G, G, None),
    }


@fake
def test_cache_arrays(pkv):
    for name, st in calls(pkv).items():
        assert st != INVALID, name
    # side by side, to the byte
    for name, st in calls(pkv, v=G + CODES, ks=G + 2 * CODES, vs=G + 2 * CODES + SIDE).items():
        assert st != INVALID, name
    for wrong in (dict(v=G), dict(vs=3 * G), dict(v=G + CODES - 16), dict(v=G - CODES + 16),
                  dict(ks=2 * G + CODES - 16), dict(vs=G), dict(vs=3 * G + SIDE - 16),
                  dict(ks=G - SIDE + 16)):
        for name, st in calls(pkv, **wrong).items():
            assert st == INVALID, (name, wrong)


@fake
def test_pools_read_into(pkv):
    lib = pkv.lib()
    c = ctypes.byref(pkv.QuantCacheDesc(64, 16, 8, 128, 0, 1 * G, 2 * G, 3 * G, 4 * G))
    p = ctypes.byref(pkv.PoolDesc(64, 16, 8, 128, 1))
    n = 2 * CODES                                             # bytes of a bf16 pool

    def r(fn, k, v):
        return fn(c, p, k, v, 30 * G, 4, None)

    for k, v in ((10 * G, 10 * G), (10 * G, 10 * G + n - 16), (10 * G + n - 16, 10 * G)):
        assert r(lib.pkv_dequantize_blocks, k, v) == INVALID
        assert r(lib.pkv_quantize_blocks, k, v) != INVALID    # only read
    assert r(lib.pkv_dequantize_blocks, 10 * G, 10 * G + n) != INVALID
    assert r(lib.pkv_dequantize_blocks, 10 * G + n, 10 * G) != INVALID
    # a pool in the cache's own arrays
    for at in (1 * G, 2 * G + CODES - 16, 3 * G - n + 16, 4 * G):
        for k, v in ((at, 20 * G), (20 * G, at)):
            assert r(lib.pkv_dequantize_blocks, k, v) == INVALID
            assert r(lib.pkv_quantize_blocks, k, v) == INVALID
