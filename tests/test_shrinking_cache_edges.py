"""Host side of the corners of the operators around a shrinking cache."""
import ctypes
import math
import os
import random
import re

import pytest
import torch

INVALID = 1
A = 0x1000000
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_58_gb300", "csrc")


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_58_gb300 import build
    build.build()
    import paged_kv_cache_58_gb300 as m
    return m


def test_evict_waits_for_its_cluster_before_it_touches_it():
    """Another CTA's shared memory may be accessed only once all CTAs of the cluster are known
    to have started.  An access too early does not show in results, so the kernel's text is
    looked at: a cluster barrier is complete ahead of the first remote address."""
    with open(os.path.join(CSRC, "evict.cu")) as f:
        kernel = f.read().split("evict_kernel(const EvictArgs", 1)[1]
    kernel = re.sub(r"//[^\n]*", "", kernel)
    barrier = min(kernel.index(x) for x in ("cluster.barrier_wait()", "cluster.sync()"))
    assert barrier < kernel.index("map_shared_rank")
    if kernel.index("cluster.barrier_wait()") == barrier:
        assert kernel.index("cluster.barrier_arrive()") < barrier


# ------------------------------------------------------------------ frequencies

def test_frequencies_under_another_default_device(pkv):
    """They are computed on the host: torch's default device must not name where."""
    want, _ = pkv.rope_frequencies(64, device="cpu")
    with torch.device("meta"):
        got, _ = pkv.rope_frequencies(64, device="cpu")
    assert got.device.type == "cpu" and torch.equal(got, want)


@pytest.mark.parametrize("r,theta,factor,trained,low,high", [
    (128, 1e6, 4.0, 32768, 1, 32), (64, 1e4, 40.0, 4096, 1, 32), (128, 500000.0, 8.0, 8192, 2, 20),
    (16, 150000.0, 32.0, 4096, 1, 32), (64, 1e4, 16.0, 4096, 0, 32), (32, 1e4, 2.0, 40, 1, 4)])
def test_yarn_by_pair_index(pkv, r, theta, factor, trained, low, high):
    """The blend that released models use: linear in the pair index, from the last whole index
    with at least `high` turns over the trained context to the first with at most `low`."""
    f, s = pkv.rope_frequencies(r, theta, scaling="yarn_pairs", factor=factor, low=low, high=high,
                                original_context=trained, device="cpu")
    assert s == pytest.approx(0.1 * math.log(factor) + 1, rel=1e-7)
    plain = [theta ** (-2 * i / r) for i in range(r)]          # past r / 2 as well: the borders
    turns = [trained * x / (2 * math.pi) for x in plain]
    first = max([i for i in range(r) if turns[i] >= high], default=0)
    last = min([i for i in range(r) if turns[i] <= low], default=r - 1)
    assert last > first
    for i, got in enumerate(f.tolist()):
        stretched = min(max((i - first) / (last - first), 0.0), 1.0)
        want = stretched * plain[i] / factor + (1 - stretched) * plain[i]
        assert abs(got - want) <= 1e-12 * want, i


def test_yarn_ramps_differ(pkv):
    """Base 1e6, 32768 trained tokens, factor 4, 128 dimensions: pair 32 by index, worked out by
    hand (between pairs 23 and 40: 8/17 kept), and by turns."""
    kw = dict(factor=4, original_context=32768, device="cpu")
    by_pair, _ = pkv.rope_frequencies(128, 1e6, scaling="yarn_pairs", **kw)
    by_turns, _ = pkv.rope_frequencies(128, 1e6, scaling="yarn", **kw)
    assert float(by_pair[32]) == pytest.approx(1e-3 * (8 / 17 + 9 / 17 / 4), rel=1e-12)
    assert float(by_turns[32]) == pytest.approx(3.52e-4, rel=1e-2)
    assert torch.equal(by_pair[:18], by_turns[:18]) and torch.equal(by_pair[40:], by_turns[40:])


def test_yarn_by_pair_index_refusals(pkv):
    kw = dict(scaling="yarn_pairs", device="cpu")
    for bad in (dict(factor=4), dict(factor=4, original_context=4096, theta=1.0),
                dict(factor=0.5, original_context=4096),
                dict(factor=4, original_context=4096, low=4, high=4)):
        with pytest.raises(pkv.PkvError) as e:
            pkv.rope_frequencies(64, **bad, **kw)
        assert e.value.status == INVALID
    # the whole of a head turns more than `high` times, or less than `low`
    f, _ = pkv.rope_frequencies(64, 2.0, factor=4, original_context=1 << 20, **kw)
    g, _ = pkv.rope_frequencies(64, 2.0, device="cpu")
    assert torch.equal(f, g)
    f, _ = pkv.rope_frequencies(64, 1e4, factor=4, original_context=1, **kw)
    g, _ = pkv.rope_frequencies(64, 1e4, device="cpu")
    assert torch.equal(f, g / 4)


def test_readme_passes_the_scale_on():
    """YaRN's scale goes with its frequencies: the example that takes both passes both."""
    with open(os.path.join(os.path.dirname(CSRC), "..", "README.md")) as f:
        example = f.read().split("freq, attn_scale = pkv.rope_frequencies(", 1)[1].split("```")[0]
    for call in re.findall(r"pkv\.rope(?:_append)?\(((?:[^()]|\([^()]*\))*)\)", example):
        assert "freq" in call and "attn_scale=attn_scale" in call


def test_block_table_under_another_default_device(pkv):
    a = pkv.BlockAllocator(4, 16)
    a.add_seq(1, 40)
    want = a.block_table([1], 4)
    with torch.device("meta"):
        got = a.block_table([1], 4)
    assert got.device.type == "cpu" and torch.equal(got, want)


# ------------------------------------------------------------------ rows that overlap

fake = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers")


def touch(n, a, a_step, a_bytes, b, b_step, b_bytes):
    """Whether any of n rows at a has a byte in common with any of n rows at b."""
    return any(a + i * a_step < b + j * b_step + b_bytes and b + j * b_step < a + i * a_step + a_bytes
               for i in range(n) for j in range(n))


@fake
def test_rope_refuses_rows_that_overlap(pkv):
    """The output in its input's place, between its rows and apart from them is taken, rows that
    share a byte are not; against every pair of rows looked at."""
    H, D, es = 2, 64, 2
    row = H * D * es
    r = random.Random(7)

    def taken(out, so, x, sx, n):
        # on a host without a GPU a call whose arguments are accepted ends with the CUDA error
        return pkv.lib().pkv_rope(1, out, so // es, x, sx // es, A, A, 64, 0, 0, 1.0, n, H, D,
                                  None) != INVALID

    assert taken(A, row, A, row, 5) and taken(A, 3 * row, A, 3 * row, 5)       # in place
    assert taken(A, 4 * row, A, row, 1)                                        # one token
    assert taken(A, 3 * row, A + row, 3 * row, 5)                              # a neighbour slice
    assert not taken(A, row, A + 16, row, 5) and not taken(A + 16, row, A, row, 5)
    assert not taken(A, 2 * row, A, row, 5) and not taken(A, row, A, 0, 2)
    assert not taken(A, 3 * row, A + 3 * row, 3 * row, 2)                      # a token later
    both = [0, 0]
    for _ in range(4000):
        n = r.choice([1, 2, 3, 7])
        so = row + 16 * r.choice([0, 1, 8, 16, 17, 40])
        sx = r.choice([so, 0, 16, row, row + 16 * r.randint(0, 40)])
        x = A + 16 * r.randint(-150, 150)
        want = (x == A and (so == sx or n == 1)) or not touch(n, A, so, row, x, sx, row)
        assert taken(A, so, x, sx, n) == want, (n, so, sx, x - A)
        both[want] += 1
    assert min(both) > 500


@fake
def test_rope_append_refuses_an_output_over_its_inputs(pkv):
    d, far = pkv.PoolDesc(64, 16, 2, 64, 1), A + (1 << 24)
    es, step, T = 2, 8 * 64 * 2, 4       # tokens of 4 + 2 + 2 heads

    def taken(qo, q, k, v, qos=step):
        return pkv.lib().pkv_rope_append(
            ctypes.byref(d), far, far, far, qo, qos // es, q, step // es, k, step // es, v,
            step // es, far, far, 64, 0, 1.0, T, 4, None) != INVALID

    q, k, v = A, A + 4 * 128, A + 6 * 128
    assert taken(q, q, k, v)                           # in place, in one projection
    assert taken(far + (1 << 20), q, k, v)
    assert not taken(q + 16, q, k, v) and not taken(q, q, k, v, qos=2 * step)
    assert not taken(q + 128, q, k, v)                 # its last head is k's first
    assert not taken(q, A + (1 << 20), q + 3 * 128, v) and not taken(q, q, k, q + 3 * step)
    assert taken(A + T * step, q, k, v) and not taken(A + T * step - 16, q, k, v)


# ------------------------------------------------------------------ plans

@pytest.mark.parametrize("hkv", [2, 8])
def test_prompt_weights_split_keys_by_the_ctas_of_a_launch(pkv, hkv):
    """fp32: where the scores of one kv head fill a launch's share, a launch has that head's CTAs
    alone, and its keys are cut for those as with one kv head: the statistics of a head take the
    same room."""
    ask = pkv.lib().pkv_paged_prefill_weights_workspace_bytes

    def need(heads):
        d = pkv.PoolDesc(4096, 16, heads, 64, 0)
        return ask(ctypes.byref(d), 1, 4 * heads, 512, 32768, 0)

    scores = 4 * 512 * 32768 * 4                       # one kv head's, all of the share
    one = need(1) - scores - 16                        # a counter is in every workspace
    assert one % (4 * 512 * 8) == 0 and one // (4 * 512 * 8) > 1     # parts of the keys
    assert need(hkv) - scores - 16 == hkv * one
