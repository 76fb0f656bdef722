"""Rules of the 4-bit products' kernels that no run can show to be broken, checked on their
source (with tests/test_steps_source.py)."""
import re

from tests.test_gmm_source import between, code


def test_a_warp_that_gives_up_waits_for_its_own_products():
    """On the way out after a wait that ran out, the warp that issued MMAs waits for the last
    commit of them: their arrivals and the accumulators must not outlive the CTA's hold on
    its shared and tensor memory."""
    mma = between(code("w4_many.cuh"), "const int h = warp;", "} else if (warp == 2) {")
    end = mma[mma.index("if (ok) { for (uint32_t i = nx"):]
    assert re.search(r"\} else if \(nx > 0 \|\| db > 0 \|\| dph == 0\) \{ "
                     r"uint64_t\* last = &d_full\[\(db > 0 \? db - 1 : C::DB - 1\) \* 2 \+ h\]; "
                     r"const uint32_t done = db > 0 \? dph \^ 1 : dph; .*"
                     r"for \(int i = 0; i < 1000 && !mbar_try_wait\(last, done\); \+\+i\)", end)


def test_the_last_accumulators_phase():
    """The arithmetic of that wait, over any number of groups issued: the buffer and the parity
    of the last one, and nothing where there was none."""
    DB = 2
    for per_block in (1, 2, 4):
        db, dph = 0, 1
        for n in range(40):
            nx = n // per_block
            issued = nx > 0 or db > 0 or dph == 0
            assert issued == (n > 0)
            if issued:
                last = n - 1
                assert (db - 1 if db > 0 else DB - 1) == last % DB
                assert (dph ^ 1 if db > 0 else dph) == (last // DB) & 1
            db += 1
            if db == DB:
                db, dph = 0, dph ^ 1
