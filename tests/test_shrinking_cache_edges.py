"""Host side of the corners of the operators around a shrinking cache."""
import os
import re

import pytest

OK, INVALID = 0, 1
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
