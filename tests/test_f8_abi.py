"""Argument checks of the e4m3 and grouped products: every refusal happens on
the host, before any CUDA work, with a status and a message."""
import ctypes

import pytest

import moe_ffn_gb300 as qm

FAKE = 1 << 20  # a 16-byte-aligned non-null address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    qm.build()
    return qm.lib()


INV, UNS = qm.ERR_INVALID_ARGUMENT, qm.ERR_UNSUPPORTED


def refused(lib, status, want):
    assert status == want, (status, qm.last_error())
    assert qm.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(xtype=qm.E4M3), UNS), (dict(xtype=qm.Q8_0), UNS), (dict(x=None), INV),
    (dict(q=None), INV), (dict(scale=None), INV), (dict(rows=-1), INV), (dict(cols=0), INV),
    (dict(ldx=63), INV), (dict(cols=(1 << 20) + 1, ldx=1 << 21), UNS), (dict(x=FAKE + 1), INV),
    (dict(scale=FAKE + 2), INV), (dict(rows=1 << 31), UNS),
    (dict(rows=0x7fffff00, cols=1 << 20, ldx=1 << 20), UNS),
])
def test_quantize_refusals(lib, kw, want):
    a = dict(xtype=qm.BF16, x=FAKE, rows=2, cols=64, ldx=64, q=FAKE, scale=FAKE)
    a.update(kw)
    refused(lib, lib.f8_quantize(a["xtype"], a["x"], a["rows"], a["cols"], a["ldx"], a["q"],
                                 a["scale"], None), want)


MM_BAD = [
    (dict(W=None), INV), (dict(w_scale=None), INV), (dict(x=None), INV),
    (dict(x_scale=None), INV), (dict(y=None), INV), (dict(rows=0), INV), (dict(cols=0), INV),
    (dict(n=-1), INV), (dict(cols=72), UNS), (dict(ldx=264), UNS), (dict(ldx=128), INV),
    (dict(ldy=99), INV), (dict(ytype=qm.E4M3), UNS), (dict(ytype=3), UNS),
    (dict(W=FAKE + 8), INV), (dict(x=FAKE + 8), INV), (dict(y=FAKE + 1), INV),
    (dict(w_scale=FAKE + 2), INV), (dict(x_scale=FAKE + 1), INV),
    (dict(cols=(1 << 20) + 16, ldx=1 << 21), UNS), (dict(n=1 << 31), UNS),
    (dict(rows=1 << 31, ldy=1 << 31), UNS),
]


@pytest.mark.parametrize("kw,want", MM_BAD)
def test_f8_mm_refusals(lib, kw, want):
    a = dict(W=FAKE, w_scale=FAKE, rows=100, cols=256, x=FAKE, x_scale=FAKE, n=3, ldx=256,
             ytype=qm.BF16, y=FAKE, ldy=100)
    a.update(kw)
    refused(lib, lib.f8_mm(a["W"], a["w_scale"], a["rows"], a["cols"], a["x"], a["x_scale"],
                           a["n"], a["ldx"], a["ytype"], a["y"], a["ldy"], None), want)


@pytest.mark.parametrize("kw,want", MM_BAD + [
    (dict(offsets=None), INV), (dict(offsets=FAKE + 2), INV), (dict(groups=0), INV),
    (dict(groups=1025), UNS), (dict(wtype=qm.F32), UNS), (dict(wtype=qm.Q4_K), UNS),
    (dict(wtype=qm.BF16), INV),                                  # scales with a 16-bit type
    (dict(wtype=qm.F16, w_scale=None, x_scale=None, cols=100, ldx=104), UNS),
])
def test_mm_grouped_refusals(lib, kw, want):
    a = dict(wtype=qm.E4M3, W=FAKE, w_scale=FAKE, groups=4, rows=100, cols=256, x=FAKE,
             x_scale=FAKE, n=3, ldx=256, offsets=FAKE, ytype=qm.F16, y=FAKE, ldy=100)
    a.update(kw)
    refused(lib, lib.mm_grouped(a["wtype"], a["W"], a["w_scale"], a["groups"], a["rows"],
                                a["cols"], a["x"], a["x_scale"], a["n"], a["ldx"], a["offsets"],
                                a["ytype"], a["y"], a["ldy"], None), want)


def shape(**kw):
    d = dict(hidden=256, expert_dim=128, num_experts=8, top_k=2, n_tokens=3, gate_qtype=qm.E4M3,
             up_qtype=qm.E4M3, down_qtype=qm.E4M3)
    d.update(kw)
    return qm.moe_shape(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(hidden=0), INV), (dict(expert_dim=-1), INV), (dict(num_experts=0), INV),
    (dict(top_k=0), INV), (dict(n_tokens=-1), INV), (dict(renormalize=False), INV),
    (dict(gate_qtype=qm.Q4_K), UNS), (dict(down_qtype=qm.BF16), UNS),
    (dict(num_experts=257), UNS), (dict(top_k=17), UNS), (dict(hidden=192), UNS),
    (dict(expert_dim=96), UNS), (dict(n_tokens=1 << 28), UNS),
])
def test_moe_shape_refusals(lib, kw, want):
    s = shape(**kw)
    assert lib.moe_experts_f8_workspace_size(ctypes.byref(s)) == 0
    assert qm.last_error()
    with pytest.raises(qm.QmoeError):
        qm.moe_experts_f8_workspace_size(s)
    refused(lib, lib.moe_experts_f8(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.byref(s), qm.BF16,
                                    FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None), want)


@pytest.mark.parametrize("pos", [0, 1, 2, 3, 4, 5, 8, 9, 10, 12, 13])
def test_moe_null_and_alignment(lib, pos):
    s = shape()
    need = qm.moe_experts_f8_workspace_size(s)

    def call(args, ws_bytes=need):
        return lib.moe_experts_f8(*args, ws_bytes, None)
    base = [FAKE] * 6 + [ctypes.byref(s), qm.BF16] + [FAKE] * 6
    null, off = list(base), list(base)
    null[pos] = None
    off[pos] = FAKE + 2
    refused(lib, call(null), INV)
    refused(lib, call(off), INV)
    refused(lib, call(base, need - 1), INV)
    bad = list(base)
    bad[7] = qm.E4M3
    refused(lib, call(bad), UNS)
    residual = list(base)
    residual[11] = FAKE + 4
    refused(lib, call(residual), INV)


def test_moe_workspace_covers_its_arrays(lib):
    s = shape(hidden=2048, expert_dim=768, num_experts=128, top_k=8, n_tokens=5)
    P = 40
    need = 129 * 4 + P * 4 + P * 2048 + P * 16 * 4 + P * 768 + P * 6 * 4 + P * 2048 * 4
    got = qm.moe_experts_f8_workspace_size(s)
    assert need <= got <= need + 7 * 256 and got % 256 == 0


def test_no_rows_is_ok_without_a_device(lib):
    """A call with no rows returns before any pointer or device is looked at."""
    assert lib.f8_quantize(qm.F32, None, 0, 64, 64, None, None, None) == qm.OK
    assert lib.f8_mm(None, None, 5, 64, None, None, 0, 64, qm.F32, None, 5, None) == qm.OK
    assert lib.mm_grouped(qm.BF16, None, None, 3, 5, 64, None, None, 0, 64, None, qm.F32, None,
                          5, None) == qm.OK
    s = shape(n_tokens=0)
    assert lib.moe_experts_f8(None, None, None, None, None, None, ctypes.byref(s), qm.F32, None,
                              None, None, None, None, None, 0, None) == qm.OK


def test_binding_refuses_host_and_mistyped_tensors(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 128)
    with pytest.raises(qm.QmoeError) as ei:
        qm.f8_quantize(qm.F32, x, 2, 128, x, x, stream=0)
    assert ei.value.status == INV and "current CUDA device" in str(ei.value)


class OnDevice:
    """A host tensor that says it is on the current CUDA device: for refusals
    that come before anything is launched."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def get_device(self):
        import torch
        return torch.cuda.current_device() if torch.cuda.is_initialized() else -1

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refuses_layouts_it_would_misread(lib):
    """Arrays are read by address, row after row: a transposed tensor, rows
    with gaps where no stride is given, or another stride than the one given
    would be read in the wrong order."""
    torch = pytest.importorskip("torch")
    d = OnDevice
    n, k, m = 64, 128, 4
    w = torch.zeros(n, k, dtype=torch.uint8)
    ws, xs, y = torch.zeros(1, 1), torch.zeros(m, 1), torch.zeros(m, n)
    x = torch.zeros(m, k, dtype=torch.uint8)
    gaps = torch.zeros(2 * m, 2 * k, dtype=torch.uint8)

    def f8(w=w, ws=ws, x=x, xs=xs, y=y, **kw):
        qm.f8_mm(d(w), d(ws), n, k, d(x), d(xs), m, qm.F32, d(y), stream=0, **kw)

    wide = torch.zeros(n, 2 * k, dtype=torch.uint8)
    for name, call in [
            ("W", lambda: f8(w=torch.zeros(k, n, dtype=torch.uint8).t())),
            ("W", lambda: f8(w=wide[:, :k])),
            ("x", lambda: f8(x=torch.zeros(k, m, dtype=torch.uint8).t())),
            ("x", lambda: f8(x=gaps[:m, :k])),
            ("x", lambda: f8(x=gaps[::2, :k], ldx=2 * k)),
            ("x_scale", lambda: f8(xs=torch.zeros(m, 2)[:, :1])),
            ("y", lambda: f8(y=torch.zeros(m, 2 * n)[:, :n])),
            ("y", lambda: f8(y=torch.zeros(n, m).t()))]:
        with pytest.raises(qm.QmoeError) as ei:
            call()
        assert ei.value.status == INV and f"f8_mm: {name} " in str(ei.value)
        assert "stride" in str(ei.value)


def test_binding_takes_rows_with_the_given_stride(lib):
    torch = pytest.importorskip("torch")
    qm._context(0)
    big = torch.zeros(3, 4, 256)
    dev = OnDevice(big).get_device()
    for t, ld in [(big[0, :, :128], 256), (big[0, ::2, :128], 512), (big[:, :, :128], 256),
                  (big[0], 256), (big[0], 128), (big.view(-1), 256), (big[1, 2:3, 5:133], 128)]:
        assert qm._arg("f", "x", OnDevice(t), qm.F32, 1, dev, ld) == t.data_ptr()


def test_type_numbers_match_header():
    text = open(qm.HEADER).read()
    for name in ("BF16", "F16", "E4M3"):
        assert f"#define QMOE_{name} {getattr(qm, name)}\n" in text
