"""build(): the library does not depend on the binding's C module, which belongs to one
interpreter.  With stand-ins for the compilers that write their output file and a log."""
import os
import stat
import sysconfig

import pytest

import moe_ffn_gb300 as qm


@pytest.fixture
def tree(tmp_path, monkeypatch):
    def tool(name, status=0):
        p = tmp_path / name
        p.write_text(f"""#!/bin/sh
echo "$@" >> {tmp_path}/{name}.log
[ {status} = 0 ] || exit {status}
while [ $# -gt 0 ]; do [ "$1" = -o ] && echo {name} > "$2"; shift; done
exit 0
""")
        p.chmod(p.stat().st_mode | stat.S_IXUSR)
        return str(p)

    class Tree:
        lib, calls = str(tmp_path / "lib.so"), str(tmp_path / ("_calls" + os.path.basename(
            qm.CALLS_PATH)[6:]))

        def compilers(self, nvcc=0, cc=0):
            monkeypatch.setenv("NVCC", tool("nvcc", nvcc))
            monkeypatch.setenv("CC", tool("cc", cc) if cc is not None else str(tmp_path / "none"))

        def runs(self, name):
            log = tmp_path / f"{name}.log"
            return len(log.read_text().splitlines()) if log.exists() else 0

    monkeypatch.setattr(qm, "_HERE", str(tmp_path))
    monkeypatch.setattr(qm, "LIB_PATH", Tree.lib)
    monkeypatch.setattr(qm, "CALLS_PATH", Tree.calls)
    monkeypatch.setattr(qm, "_calls", None)
    return Tree()


def test_the_module_is_named_for_its_interpreter():
    tag = sysconfig.get_config_var("EXT_SUFFIX")
    assert qm.CALLS_PATH.endswith(tag) and "cpython" in tag


@pytest.mark.parametrize("cc", [1, None], ids=["fails", "missing"])
def test_the_library_builds_without_the_module(tree, cc):
    tree.compilers(cc=cc)
    with pytest.warns(RuntimeWarning, match="calls.c"):
        assert qm.build() == tree.lib
    assert os.path.exists(tree.lib) and not os.path.exists(tree.calls)
    assert tree.runs("nvcc") == len(qm.UNITS) + 1
    # what could not be built is tried again, alone
    with pytest.warns(RuntimeWarning):
        qm.build()
    assert tree.runs("nvcc") == len(qm.UNITS) + 1
    tree.compilers()
    qm.build()
    assert os.path.exists(tree.calls) and tree.runs("nvcc") == len(qm.UNITS) + 1
    n = tree.runs("cc")
    qm.build()
    assert tree.runs("cc") == n and sorted(os.listdir(os.path.dirname(tree.lib))) == sorted(
        {"nvcc", "nvcc.log", "cc", "cc.log", os.path.basename(tree.lib),
         os.path.basename(tree.calls)})


def test_an_outdated_module_is_not_left_behind(tree):
    tree.compilers()
    qm.build()
    os.utime(tree.calls, (1, 1))
    tree.compilers(cc=1)
    with pytest.warns(RuntimeWarning):
        qm.build()
    assert not os.path.exists(tree.calls)


def test_a_library_that_does_not_compile_raises(tree):
    import subprocess
    tree.compilers(nvcc=2)
    with pytest.raises(subprocess.CalledProcessError):
        qm.build()
    assert not os.path.exists(tree.lib)


def test_without_the_module_calls_go_the_long_way(monkeypatch, tmp_path):
    """The library's own answers, with a warning the first time."""
    qm.build()
    monkeypatch.setattr(qm, "CALLS_PATH", str(tmp_path / "missing.so"))
    monkeypatch.setattr(qm, "_calls", None)
    with pytest.warns(RuntimeWarning, match="build"):
        with pytest.raises(qm.QmoeError, match="top_k") as e:
            qm.moe_route(qm.F32, None, 4, 8, 9, None, None)
    assert e.value.status == qm.ERR_INVALID_ARGUMENT
    qm.moe_combine(qm.F32, None, 0, 8, None, None, 0, 2, qm.F32, None, None)
    with pytest.raises(qm.QmoeError, match="scale_cols"):
        qm.w4_mm(None, qm.F16, None, None, 16, 4, 64, qm.F32, None, 1, qm.F32, None)
