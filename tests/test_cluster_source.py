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


def test_split_barriers_are_paired_on_every_way_out():
    """Whoever arrives at a split cluster barrier also waits for it, before an early return
    too, and under the same condition."""
    for name, k in kernels():
        if "cluster_arrive();" not in k:
            continue
        assert k.count("cluster_arrive();") == 1 == k.count("if (ranks > 1) cluster_arrive();")
        body = k[k.index("cluster_arrive();"):]
        for way_out in re.findall(r"\{([^{}]*)return; \}", body):
            assert "if (ranks > 1) cluster_wait();" in way_out, (name, way_out)
        assert not re.search(r"\) return;", body), name
        # the first tile, which every cluster that stays has, waits before its first store
        assert "if (ranks > 1 && tile == cluster) cluster_wait();" in k, name
        assert k.index("tile == cluster) cluster_wait();") < re.search(REMOTE, k).start()
