"""The short way from the binding into the library (csrc/calls.c): what it takes, what
it leaves to the binding's own checks, and that a refusal of the library comes through.
On CPU, with tensors that say they are on a device."""
import ctypes

import pytest

import moe_ffn_gb300 as qm
from tests.test_f8_abi import INV

torch = pytest.importorskip("torch")
F, B, H, I, U = torch.float32, torch.bfloat16, torch.float16, torch.int32, torch.uint8


class Fake:
    """A contiguous tensor on device `dev`, at a made-up address that nothing reads (every
    call here is refused by the library or not made)."""

    def __init__(self, numel, dtype, dev=0, contiguous=True, ptr=1 << 20):
        self.dtype, self._n, self._dev, self._c, self._p = dtype, numel, dev, contiguous, ptr
        self.nbytes = numel * 4

    def get_device(self):
        return self._dev

    def is_contiguous(self):
        return self._c

    def numel(self):
        return self._n

    def data_ptr(self):
        return self._p


@pytest.fixture
def calls():
    """The module with the library's functions and a made-up current device 0."""
    qm.build()
    m = qm._bind_calls()
    h = qm.lib()
    names = ("moe_route", "moe_route_backward", "moe_permute", "moe_combine",
             "moe_combine_backward", "w4_mm", "w4_mm_grouped")
    addr = tuple(ctypes.cast(getattr(h, n), ctypes.c_void_p).value for n in names)
    m.bind(addr, (F, B, H, I, U), lambda: 0, lambda dev: 0)
    yield m
    m.bind(addr, (F, B, H, I, U), torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)


def route(flags=0, **kw):
    a = dict(lt=qm.F32, x=Fake(32, F), t=4, e=8, k=2, idx=Fake(8, I), w=Fake(8, F), flags=flags,
             st=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(lt=99), dict(lt="f32"), dict(x=1 << 20), dict(x=Fake(32, B)), dict(x=Fake(31, F)),
    dict(x=Fake(32, F, dev=-1)), dict(x=Fake(32, F, dev=1)), dict(x=Fake(32, F, contiguous=False)),
    dict(x=object()), dict(t=-1), dict(t=1 << 31), dict(t=1 << 70), dict(t=4.0), dict(k=-2),
    dict(idx=Fake(8, F)), dict(idx=Fake(7, I)), dict(w=Fake(8, F, dev=1)), dict(st=0),
    dict(e=1 << 40), dict(flags=-1)])
def test_what_is_left_to_the_binding(calls, kw):
    assert calls.route(*route(flags=2)) == INV     # (as it stands the library refuses it)
    assert "route_flags" in qm.last_error()
    assert calls.route(*route(**{"flags": 2, **kw})) is None


def test_null_arrays_reach_the_library(calls):
    """None is a null pointer, which the library refuses where it needs one."""
    assert calls.route(*route(x=None)) == INV
    assert calls.route(*route(idx=None)) == INV


def test_another_current_device_is_left_to_the_binding(calls):
    def dev1():
        return 1

    def broken():
        raise RuntimeError("no device")
    h = qm.lib()
    addr = tuple(ctypes.cast(h.moe_route, ctypes.c_void_p).value for _ in range(7))
    for get in (dev1, broken):
        calls.bind(addr, (F, B, H, I, U), get, lambda dev: 0)
        assert calls.route(*route(flags=2)) is None


def test_every_call_is_refused_as_the_library_refuses_it(calls):
    f, i, u = Fake(1 << 20, F), Fake(1 << 20, I), Fake(1 << 20, U)
    assert calls.route_backward(qm.F32, f, 4, 8, 9, i, f, f, f, 0, None) == INV   # k > E
    assert "top_k" in qm.last_error()
    small = Fake(10, U)
    small.nbytes = 10
    assert calls.permute(qm.F32, f, 4, 8, i, 8, 2, f, i, i, small, None) == INV
    assert "workspace 10" in qm.last_error()
    odd = Fake(1 << 20, F, ptr=(1 << 20) + 2)
    assert calls.combine(qm.F32, odd, 8, 8, i, None, 4, 2, qm.F32, None, f, None) == INV
    assert calls.combine_backward(qm.F32, f, 8, 8, i, f, 4, 2, qm.F32, f, None, None, None) == INV
    assert "grad_y" in qm.last_error()
    w4 = [u, qm.F32, f, None, 32, -1, 4, 48, qm.F32, f, 1, None, qm.F32, f, None]
    assert calls.w4(*w4) == INV and "w4_mm:" in qm.last_error()          # 48 % 32
    w4[5], w4[11] = 3, i
    assert calls.w4(*w4) == INV and "w4_mm_grouped:" in qm.last_error()
    for groups in (0, -2, 1 << 20):
        w4[5] = groups
        assert calls.w4(*w4) is None
    w4[5], w4[4] = 3, 0
    assert calls.w4(*w4) is None


def test_binding_raises_what_the_short_way_answers(calls):
    with pytest.raises(qm.QmoeError) as e:
        qm.moe_route(qm.F32, Fake(32, F), 4, 8, 9, Fake(36, I), Fake(36, F))
    assert e.value.status == INV and "top_k" in str(e.value)


@pytest.mark.parametrize("name,n", [("route", 9), ("route_backward", 11), ("permute", 12),
                                    ("combine", 12), ("combine_backward", 13), ("w4", 15)])
def test_argument_counts(calls, name, n):
    for k in (0, n - 1, n + 1):
        with pytest.raises(TypeError):
            getattr(calls, name)(*[None] * k)
    with pytest.raises((TypeError, ValueError)):
        calls.bind((), (), None, None)


def test_missing_module_fails_loudly(monkeypatch, tmp_path):
    monkeypatch.setattr(qm, "CALLS_PATH", str(tmp_path / "missing.so"))
    monkeypatch.setattr(qm, "_calls", None)
    with pytest.raises(qm.QmoeError, match="build"):
        qm._bind_calls()
