"""CPU: kernels that write to other CTAs' shared memory.

A CTA of a cluster may touch another one's shared memory only once that one is known
to have started, which a barrier of the cluster guarantees and nothing else does.  A
run cannot show that it is missing, the source can."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "split_kv_mla_paged_gb300", "csrc")
BARRIER = re.compile(r"cluster\.sync\(\)|cluster_wait\(\)")


def _kernels(text):
    """The bodies of a source's __global__ functions, without comments."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__", text):
        at = text.index("{", m.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield text[at:end]


USERS = [(os.path.basename(f), body) for f in sorted(glob.glob(os.path.join(CSRC, "*.cu*")))
         for body in _kernels(open(f).read()) if "map_shared_rank" in body]


def test_the_kernels_with_distributed_shared_memory_are_found():
    assert [f for f, _ in USERS] == ["evict.cu", "verify.cu"]


@pytest.mark.parametrize("name,body", USERS, ids=[f for f, _ in USERS])
def test_a_cluster_barrier_precedes_the_first_access(name, body):
    assert BARRIER.search(body[:body.index("map_shared_rank")]), name
