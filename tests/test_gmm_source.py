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


def test_no_cta_leaves_with_a_commit_in_flight():
    """A commit's arrival comes from the tensor core, so no barrier between
    threads orders it: every barrier that a commit signals is waited for, in
    both CTAs of a pair, before the CTA ends (its shared memory may be another
    launch's at once)."""
    pair = code("gmm_pair.cuh")
    signalled = set(re.findall(r"umma::commit_pair\(&?(\w+)", pair))
    assert signalled == {"empty", "acc_full", "mma_done"}
    # stages: handed back only where a later load waits for them
    assert pair.count("commit_pair(&empty") == pair.count(
        "if (k0 + k < ret) umma::commit_pair(&empty[s])") == 1
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
    assert one.count("commit(&empty") == one.count("if (kb < ret) umma::commit(&empty[s])") == 1
    assert one.index("commit(mma_done)") < one.index("mbar_wait_spin(mma_done")


def test_stages_are_handed_back_exactly_where_a_load_waits():
    """The arithmetic of unreturned() over whole runs of a CTA: step i of n hands
    its stage back exactly if a load i + NST follows, which waits for it."""
    text = code("gmm.cuh")
    assert "return after < NST ? NST - static_cast<int>(after) : 0;" in text
    for name, first, last in (("gmm.cuh", "kend", "kend - kbeg"), ("gmm_pair.cuh", "p.kb", "p.kb")):
        expr = (f"const int ret = {first} - unreturned<C::NST>( "
                f"static_cast<int64_t>((tiles - 1 - t) / step) * ")
        assert expr + (f"({last}))" if "-" in last else f"{last})") in code(name)
    for nst in (5, 6, 7, 8):
        for kb in (1, 2, 3, nst - 1, nst, nst + 1, 2 * nst + 1):
            for first, step, tiles in ((0, 1, 1), (0, 1, 2), (1, 3, 2), (2, 3, 12), (0, 5, 26)):
                own = range(first, tiles, step)
                n = len(own) * kb
                i = 0
                for t in own:
                    after = (tiles - 1 - t) // step * kb
                    ret = kb - (nst - after if after < nst else 0)
                    for k in range(kb):
                        assert (k < ret) == (i + nst < n), (nst, kb, t, k)
                        i += 1


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
