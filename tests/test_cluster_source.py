"""Rules of the kernels whose CTAs form clusters, checked on their source: no run can show
them to be broken, for CTAs of a cluster nearly always start together."""
import os
import re

from tests.test_gmm_source import CSRC, code

REMOTE = r"\b(cluster_st_\w+|cluster_sum|cluster_ld_\w+|mbar_arrive_cluster)\("


def kernels():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cuh"):
            for k in code(name).split("__global__ void")[1:]:
                yield name, k


def test_no_cta_touches_another_before_it_is_known_to_run():
    """Being scheduled together does not say that a neighbour has started: a barrier of the
    cluster stands before a kernel's first access to another CTA's shared memory."""
    found = set()
    for name, k in kernels():
        first = re.search(REMOTE, k)
        if not first:
            continue
        found.add(name)
        before = k[:first.start()]
        if "cluster_sync();" in before:
            continue
        assert "cluster_wait();" in before, name
        assert before.index("cluster_arrive();") < before.index("cluster_wait();"), name
    assert found == {"f8moe.cuh", "gmm.cuh", "gmm_pair.cuh", "w4.cuh", "w4_many.cuh"}


def test_barriers_in_two_steps_are_paired():
    """Whoever arrives also waits, at once and under the same condition."""
    for name, k in kernels():
        if "cluster_arrive();" in k or "cluster_wait();" in k:
            for half in ("cluster_arrive();", "cluster_wait();"):
                assert k.count(half) == 1, name
            assert "if (ranks > 1) { cluster_arrive(); cluster_wait(); }" in k, name
