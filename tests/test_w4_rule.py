"""Which of the two kernels a 4-bit product takes: the library's own rule, compiled for the
host, against measured times of both kernels (profiles/w4_kernel_times.json)."""
import ctypes
import json
import os
import subprocess
import tempfile

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def many():
    so = os.path.join(tempfile.mkdtemp(prefix="w4_rule_"), "libw4_rule.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-x", "c++", "-o", so,
                    os.path.join(HERE, "host", "w4_rule.cpp")], check=True)
    f = ctypes.CDLL(so).many_rows_host
    f.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong, ctypes.c_longlong,
                  ctypes.c_int]
    return lambda m, e, n, k, kind: bool(f(m, e, n, k, kind == "f32"))


@pytest.fixture(scope="module")
def times():
    with open(os.path.join(os.path.dirname(HERE), "profiles", "w4_kernel_times.json")) as f:
        return json.load(f)["times"]


def lost(many, times):
    """(share of the faster kernel's time that the rule loses, case) of every case."""
    out = []
    for kind, s, e, n, k, rows, few, big in times:
        taken = big if many(rows * e, e, n, k, kind) else few
        out.append((taken / min(few, big) - 1, (kind, s, e, n, k, rows, few, big)))
    return sorted(out, reverse=True)


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_the_rule_takes_the_faster_kernel(many, times, grouped, f32):
    """Nearly always, and otherwise not a much slower one: a twentieth of the cases may lose
    more than a tenth, none more than what the rule's comment says (0.6, once), and on
    average a call loses less than 2.5%."""
    some = lost(many, [t for t in times if (t[2] > 1) == grouped and (t[0] == "f32") == f32])
    assert len(some) >= 50
    assert some[0][0] <= 0.61, some[:5]
    assert sum(v > 0.10 for v, _ in some) <= max(4, len(some) // 20), some[:20]
    assert sum(v for v, _ in some) / len(some) < 0.025


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_more_rows_never_go_back(many, kind):
    """The choice changes once as rows are added."""
    for e in (1, 8, 100):
        for n, k in ((300, 640), (4096, 4096), (14336, 4096), (1024, 128), (1 << 20, 32)):
            picks = [many(m * e, e, n, k, kind) for m in range(1, 600)]
            assert picks == sorted(picks)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gpu_tests_reach_the_kernel_they_are_for(many, kind):
    """The shapes by which tests/test_gpu_w4*.py mean one kernel or the other."""
    from tests.test_gpu_w4 import MANY
    for m, n, k, _ in MANY + [(500, 1280, 1024, 64), (500, 2048, 1024, 128), (64, 4096, 4096, 128),
                              (600, 8000, 1024, 128), (300, 9000, 1024, 128)]:
        assert many(m, 1, n, k, kind), (m, n, k)
    uneven = 3 + sum([150, 1, 64, 65, 129, 7, 300, 63, 2, 200]) + 5
    assert many(uneven, 14, 520, 1024, kind) and many(uneven, 14, 768, 672, kind)
    for m, n, k in ((1, 4096, 4096), (5, 48, 14336), (64, 16, 4096),
                    (4 if kind == "f32" else 8, 4096, 14336), (16, 4096, 4096), (13, 1000, 5120),
                    (70, 200, 512)):
        assert not many(m, 1, n, k, kind), (m, n, k)
    for m, e, n, k in ((8, 128, 768, 2048), (12, 4, 200, 6144), (9, 9, 100, 256)):
        assert not many(m, e, n, k, kind), (m, e, n, k)
