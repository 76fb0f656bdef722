"""Rules of the kernels of moe_steps.cuh and w4*.cuh that no run can show to be broken,
checked on their source (as tests/test_gmm_source.py does for the grouped products)."""
import re

from tests.test_gmm_source import between, code

FILES = ("moe_steps.cuh", "moe_steps.cu", "w4.cuh", "w4_many.cuh", "w4.cu", "rows.cuh")


def test_no_read_only_loads_of_stream_ordered_data():
    """Grids that may start before the launch that writes their inputs has ended do not
    load them as constant data, nor before the dependency wait."""
    for name in FILES:
        text = code(name)
        for word in ("__ldg(", "ld.global.nc", "__restrict__"):
            assert word not in text, (name, word)
        for kernel in re.findall(r"__global__ void.*?pdl_wait\(\);", text):
            reads = set(re.findall(r"__ldcg\(([^)]*)\)", kernel))
            assert reads <= {"&p.err->skip_arrive_cta"}, (name, reads)


def test_every_kernel_waits_and_triggers_in_this_order():
    for name in ("moe_steps.cuh", "w4.cuh", "w4_many.cuh"):
        text = code(name)
        kernels = text.split("__global__ void")[1:]
        assert kernels
        for k in kernels:
            assert 0 < k.index("pdl_wait();") < k.index("pdl_trigger();"), name


def test_no_cta_leaves_with_an_arrival_of_the_tensor_core_in_flight():
    """Each barrier that a commit of the many-rows kernel signals is waited for before the
    CTA ends: accumulators by the warps that read them, the others by the MMA warps."""
    text = code("w4_many.cuh")
    assert set(re.findall(r"umma::commit\(&(\w+)", text)) == {"d_full", "a_empty", "x_empty"}
    mma = between(text, "const int h = warp;", "} else if (warp == 2) {")
    end = mma[mma.index("if (ok) { for (uint32_t i = nx"):]
    assert "wait(&x_empty[i % C::XS], (i / C::XS) & 1)" in end
    assert "if (na0 > 0) wait(&a_empty[h], (na0 - 1) & 1)" in end
    assert "if (na1 > 0) wait(&a_empty[2 + h], (na1 - 1) & 1)" in end
    sums = text[text.index("regs_inc<C::REGS_SUMS>()"):]
    assert sums.count("wait(&d_full[db * 2 + h]") == 1


def test_register_shares_add_up():
    """setmaxnreg draws on what the launch was given: 64 registers for each of 1024
    threads."""
    text = code("w4_many.cuh")
    for tma in (True, False):
        env = {}
        for name, expr in re.findall(r"(REGS_\w+) = ([^,;]+)[,;]", text):
            m = re.match(r"TMA_X \? (\S+) : (\S+)", expr.strip())
            v = (m.group(1) if tma else m.group(2)) if m else expr.strip()
            env[name] = env[v] if v in env else int(v)
        assert set(env) == {"REGS_AUX", "REGS_X", "REGS_CODES", "REGS_SUMS"}
        assert all(v % 8 == 0 and 24 <= v <= 256 for v in env.values())
        total = env["REGS_AUX"] + env["REGS_X"] + 4 * env["REGS_CODES"] + 2 * env["REGS_SUMS"]
        assert total <= 8 * 64
    assert "regs_inc<C::REGS_X>()" in text and "regs_dec<C::REGS_CODES>()" in text
