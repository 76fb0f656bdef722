"""Rules of the grouped products' kernels that no run can show to be broken (a
race that is nearly always won), checked on their source."""
import os
import re

import moe_ffn_gb300 as qm

CSRC = os.path.join(os.path.dirname(qm.__file__), "csrc")


def code(name):
    """A source file without comments, white space folded."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    return re.sub(r"\s+", " ", text)


def between(text, a, b):
    i = text.index(a)
    return text[i:text.index(b, i)]


DRAIN = "drain_stages<C::NST>(empty, it, ok, p.err)"


def test_no_cta_leaves_with_a_commit_in_flight():
    """A commit's arrival comes from the tensor core, so no barrier between
    threads orders it: every barrier that a commit signals is waited for, in
    both CTAs of a pair, before the CTA ends (its shared memory may be another
    launch's at once)."""
    pair = code("gmm_pair.cuh")
    signalled = set(re.findall(r"umma::commit_pair\(&?(\w+)", pair))
    assert signalled == {"empty", "acc_full", "mma_done"}
    # stages: the weight-load warp of either CTA, at the end of its loop
    loads = between(pair, "if (warp == 0 || warp == 2) {", "else if (warp == 1 && rank == 0)")
    assert f"if (wgt && !{DRAIN}" in loads
    # accumulators: every epilogue warp of either CTA, before each use
    epilogue = pair[pair.index("regs_inc<C::REGS_EPI>()"):]
    assert epilogue.count("mbar_wait_spin(&acc_full[ab]") == 2  # one per form
    # the last commit: the first CTA's MMA warp before the closing barrier, the
    # second CTA behind it
    mma = between(pair, "else if (warp == 1 && rank == 0)", "else if (C::F8 && warp == 3)")
    assert mma.index("commit_pair(mma_done)") < mma.index("mbar_wait_spin(mma_done")
    end = pair[pair.rindex("cluster_sync();"):]
    assert re.search(r"if \(rank != 0\) mbar_wait_spin\(mma_done,.*tmem_dealloc_pair", end)

    one = code("gmm.cuh")
    assert set(re.findall(r"umma::commit\(&?(\w+)", one)) == {"empty", "acc_full", "mma_done"}
    assert DRAIN in between(one, "if (warp == 0) {", "else if (warp == 1)")
    body = between(one, "bool drain_stages(", "__global__")
    assert "mbar_wait_spin(&empty[k % NST], (k / NST) & 1" in body and "__all_sync" in body
    assert one.index("commit(mma_done)") < one.index("mbar_wait_spin(mma_done")


def test_no_read_only_loads_of_stream_ordered_data():
    """These grids may start before the launch that writes their inputs has
    ended (weight scales included: every operand is ordered by the stream).
    Loads that promise read-only data for the kernel's whole life, written out
    or allowed to the compiler by __restrict__, are not theirs to use."""
    for name in ("f8.cuh", "f8.cu", "f8moe.cuh", "gmm.cuh", "gmm_pair.cuh", "gmm_tiles.cuh"):
        text = code(name)
        for word in ("__ldg(", "ld.global.nc", "__restrict__"):
            assert word not in text, (name, word)
        # nothing is read before the dependency wait but the kernel's own control block
        for kernel in re.findall(r"__global__ void.*?pdl_wait\(\);", text):
            reads = set(re.findall(r"__ldcg\(([^)]*)\)", kernel))
            assert reads <= {"&p.err->skip_arrive_cta"}, (name, reads)
