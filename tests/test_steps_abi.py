"""Argument checks of routing, sorting by expert, weighted sums and 4-bit products:
every refusal happens on the host, before any CUDA work."""
import pytest

import moe_ffn_gb300 as qm
from tests import steps_ref as ref
from tests.test_f8_abi import FAKE, INV, UNS, OnDevice, lib, refused  # noqa: F401


ROUTE_BAD = [
    (dict(ltype=qm.E4M3), UNS), (dict(ltype=qm.Q4_K), UNS), (dict(logits=None), INV),
    (dict(idx=None), INV), (dict(w=None), INV), (dict(n=-1), INV), (dict(E=0), INV),
    (dict(k=0), INV), (dict(k=9), INV), (dict(ldl=7), INV), (dict(flags=2), INV),
    (dict(E=1025, ldl=1025), UNS), (dict(E=64, ldl=64, k=17), UNS), (dict(n=1 << 25), UNS),
    (dict(logits=FAKE + 1), INV), (dict(idx=FAKE + 2), INV), (dict(w=FAKE + 1), INV),
]


@pytest.mark.parametrize("kw,want", ROUTE_BAD)
def test_route_refusals(lib, kw, want):  # noqa: F811
    a = dict(ltype=qm.BF16, logits=FAKE, n=3, E=8, ldl=8, k=2, flags=0, idx=FAKE, w=FAKE)
    a.update(kw)
    refused(lib, lib.moe_route(a["ltype"], a["logits"], a["n"], a["E"], a["ldl"], a["k"],
                               a["flags"], a["idx"], a["w"], None), want)


@pytest.mark.parametrize("kw,want", ROUTE_BAD + [
    (dict(dw=None), INV), (dict(g=None), INV), (dict(ldg=7), INV), (dict(g=FAKE + 1), INV),
    (dict(dw=FAKE + 2), INV)])
def test_route_backward_refusals(lib, kw, want):  # noqa: F811
    a = dict(ltype=qm.BF16, logits=FAKE, n=3, E=8, ldl=8, k=2, flags=1, idx=FAKE, w=FAKE, dw=FAKE,
             g=FAKE, ldg=8)
    a.update(kw)
    refused(lib, lib.moe_route_backward(a["ltype"], a["logits"], a["n"], a["E"], a["ldl"], a["k"],
                                        a["flags"], a["idx"], a["w"], a["dw"], a["g"], a["ldg"],
                                        None), want)


@pytest.mark.parametrize("kw,want", [
    (dict(xtype=qm.E4M3), UNS), (dict(x=None), INV), (dict(idx=None), INV), (dict(rows=None), INV),
    (dict(offsets=None), INV), (dict(pos=None), INV), (dict(ws=None), INV), (dict(n=-1), INV),
    (dict(cols=0), INV), (dict(ldx=63), INV), (dict(ldr=63), INV), (dict(E=0), INV),
    (dict(k=0), INV), (dict(E=1025), UNS), (dict(k=17), UNS), (dict(n=1 << 25), UNS),
    (dict(cols=(1 << 20) + 1, ldx=1 << 21, ldr=1 << 21), UNS), (dict(x=FAKE + 1), INV),
    (dict(rows=FAKE + 1), INV), (dict(idx=FAKE + 2), INV), (dict(pos=FAKE + 2), INV),
    (dict(offsets=FAKE + 2), INV), (dict(ws=FAKE + 8), INV), (dict(bytes=0), INV),
    (dict(n=1 << 20, bytes=256), INV),
])
def test_permute_refusals(lib, kw, want):  # noqa: F811
    a = dict(xtype=qm.BF16, x=FAKE, n=3, cols=64, ldx=64, idx=FAKE, E=8, k=2, rows=FAKE, ldr=64,
             offsets=FAKE, pos=FAKE, ws=FAKE, bytes=1 << 12)
    a.update(kw)
    refused(lib, lib.moe_permute(a["xtype"], a["x"], a["n"], a["cols"], a["ldx"], a["idx"], a["E"],
                                 a["k"], a["rows"], a["ldr"], a["offsets"], a["pos"], a["ws"],
                                 a["bytes"], None), want)


@pytest.mark.parametrize("args", [(-1, 8, 2), (3, 0, 2), (3, 8, 0), (3, 1025, 2), (3, 8, 17),
                                  (1 << 25, 8, 2)])
def test_permute_workspace_refusals(lib, args):  # noqa: F811
    with pytest.raises(qm.QmoeError):
        qm.moe_permute_workspace_size(*args)


@pytest.mark.parametrize("t,e,k", [(0, 1, 1), (1, 128, 8), (4096, 128, 8), (1 << 21, 1024, 16),
                                   (1 << 25, 1, 1), (1 << 25, 3, 1)])
def test_permute_workspace_sizes(lib, t, e, k):  # noqa: F811
    """Counts of 16 bits for every run of at least 16 tokens: never more than an
    eighth of a kilobyte an expert and token run, and whole 256-byte units."""
    n = qm.moe_permute_workspace_size(t, e, k)
    assert n % 256 == 0 and 256 <= n <= 256 + 2 * e * max(-(-t // 16), 1)


COMBINE_BAD = [
    (dict(ytype=qm.E4M3), UNS), (dict(otype=qm.Q8_0), UNS), (dict(y=None), INV),
    (dict(pos=None), INV), (dict(n=-1), INV), (dict(n_rows=-1), INV), (dict(cols=0), INV),
    (dict(k=0), INV), (dict(k=17), UNS), (dict(ldy=63), INV), (dict(ldo=63), INV),
    (dict(n=1 << 25), UNS), (dict(n_rows=1 << 31), UNS), (dict(pos=FAKE + 2), INV),
    (dict(w=FAKE + 2), INV), (dict(y=FAKE + 1), INV),
    (dict(cols=(1 << 20) + 1, ldy=1 << 21, ldo=1 << 21), UNS),
]


@pytest.mark.parametrize("kw,want", COMBINE_BAD + [
    (dict(out=None), INV), (dict(out=FAKE + 1), INV), (dict(residual=FAKE + 1), INV)])
def test_combine_refusals(lib, kw, want):  # noqa: F811
    a = dict(ytype=qm.BF16, y=FAKE, n_rows=6, cols=64, ldy=64, pos=FAKE, w=FAKE, n=3, k=2,
             otype=qm.BF16, residual=FAKE, out=FAKE, ldo=64)
    a.update(kw)
    refused(lib, lib.moe_combine(a["ytype"], a["y"], a["n_rows"], a["cols"], a["ldy"], a["pos"],
                                 a["w"], a["n"], a["k"], a["otype"], a["residual"], a["out"],
                                 a["ldo"], None), want)


@pytest.mark.parametrize("kw,want", COMBINE_BAD + [
    (dict(g=None), INV), (dict(gy=None, gw=None), INV), (dict(ldg=63), INV),
    (dict(g=FAKE + 1), INV), (dict(gy=FAKE + 1), INV), (dict(gw=FAKE + 2), INV)])
def test_combine_backward_refusals(lib, kw, want):  # noqa: F811
    a = dict(ytype=qm.BF16, y=FAKE, n_rows=6, cols=64, ldy=64, pos=FAKE, w=FAKE, n=3, k=2,
             otype=qm.BF16, g=FAKE, ldo=64, gy=FAKE, ldg=64, gw=FAKE)
    a.update(kw)
    refused(lib, lib.moe_combine_backward(a["ytype"], a["y"], a["n_rows"], a["cols"], a["ldy"],
                                          a["pos"], a["w"], a["n"], a["k"], a["otype"], a["g"],
                                          a["ldo"], a["gy"], a["ldg"], a["gw"], None), want)


W4_BAD = [
    (dict(W=None), INV), (dict(scale=None), INV), (dict(x=None), INV), (dict(y=None), INV),
    (dict(stype=qm.E4M3), UNS), (dict(xtype=qm.Q4_0), UNS), (dict(ytype=qm.E4M3), UNS),
    (dict(S=16), UNS), (dict(S=256), UNS), (dict(S=0), UNS), (dict(cols=96, S=64), INV),
    (dict(cols=100, S=32), INV), (dict(rows=0), INV), (dict(cols=0), INV), (dict(n=-1), INV),
    (dict(ldx=255), INV), (dict(ldy=99), INV), (dict(W=FAKE + 8), INV), (dict(scale=FAKE + 1), INV),
    (dict(x=FAKE + 1), INV), (dict(y=FAKE + 1), INV), (dict(n=1 << 31), UNS),
    (dict(rows=1 << 31, ldy=1 << 31), UNS), (dict(cols=1 << 21, ldx=1 << 21), UNS),
]


@pytest.mark.parametrize("kw,want", W4_BAD)
def test_w4_mm_refusals(lib, kw, want):  # noqa: F811
    a = dict(W=FAKE, stype=qm.F16, scale=FAKE, zero=None, S=128, rows=100, cols=256, xtype=qm.BF16,
             x=FAKE, n=3, ldx=256, ytype=qm.BF16, y=FAKE, ldy=100)
    a.update(kw)
    refused(lib, lib.w4_mm(a["W"], a["stype"], a["scale"], a["zero"], a["S"], a["rows"], a["cols"],
                           a["xtype"], a["x"], a["n"], a["ldx"], a["ytype"], a["y"], a["ldy"],
                           None), want)


@pytest.mark.parametrize("kw,want", W4_BAD + [
    (dict(E=0), INV), (dict(E=1025), UNS), (dict(offsets=None), INV), (dict(offsets=FAKE + 2), INV)])
def test_w4_mm_grouped_refusals(lib, kw, want):  # noqa: F811
    a = dict(W=FAKE, stype=qm.F16, scale=FAKE, zero=FAKE, S=128, E=4, rows=100, cols=256,
             xtype=qm.BF16, x=FAKE, n=3, ldx=256, offsets=FAKE, ytype=qm.BF16, y=FAKE, ldy=100)
    a.update(kw)
    refused(lib, lib.w4_mm_grouped(a["W"], a["stype"], a["scale"], a["zero"], a["S"], a["E"],
                                   a["rows"], a["cols"], a["xtype"], a["x"], a["n"], a["ldx"],
                                   a["offsets"], a["ytype"], a["y"], a["ldy"], None), want)


def test_no_rows_is_ok_without_a_device(lib):  # noqa: F811
    assert lib.moe_route(qm.F32, None, 0, 8, 8, 2, 0, None, None, None) == qm.OK
    assert lib.moe_route_backward(qm.F32, None, 0, 8, 8, 2, 0, None, None, None, None, 8,
                                  None) == qm.OK
    assert lib.moe_combine(qm.F32, None, 0, 8, 8, None, None, 0, 2, qm.F32, None, None, 8,
                           None) == qm.OK
    assert lib.moe_combine_backward(qm.F32, None, 0, 8, 8, None, None, 0, 2, qm.F32, None, 8, None,
                                    8, FAKE, None) == qm.OK
    assert lib.w4_mm(None, qm.F16, None, None, 32, 5, 64, qm.F32, None, 0, 64, qm.F32, None, 5,
                     None) == qm.OK
    assert lib.w4_mm_grouped(None, qm.F16, None, None, 32, 3, 5, 64, qm.F32, None, 0, 64, None,
                             qm.F32, None, 5, None) == qm.OK


def test_binding_refuses_wrong_tensors(lib):  # noqa: F811
    """Host tensors, other types, other strides and too few elements."""
    torch = pytest.importorskip("torch")
    d = OnDevice
    f, i, b = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.bfloat16

    def route(x=d(f), idx=d(i), w=d(torch.zeros(4, 2)), **kw):
        qm.moe_route(qm.F32, x, 4, 8, 2, idx, w, stream=0, **kw)

    def permute(x=d(f), rows=d(torch.zeros(8, 8)), offsets=d(torch.zeros(9, dtype=torch.int32)),
                ws=d(torch.zeros(256, dtype=torch.uint8)), **kw):
        qm.moe_permute(qm.F32, x, 4, 8, d(i), 8, 2, rows, offsets, d(i), ws, stream=0, **kw)

    def w4(W=d(torch.zeros(4, 16, dtype=torch.uint8)), s=d(torch.zeros(4, 1, dtype=torch.half)),
           z=None, x=d(torch.zeros(1, 32))):
        qm.w4_mm(W, qm.F16, s, z, 32, 4, 32, qm.F32, x, 1, qm.F32, d(torch.zeros(1, 4)), stream=0)

    def combine(y=d(torch.zeros(8, 8)), out=d(f), **kw):
        qm.moe_combine(qm.F32, y, 8, 8, d(i), None, 4, 2, qm.F32, None, out, stream=0, **kw)

    for name, call in [
            ("logits", lambda: route(x=f)), ("logits", lambda: route(x=d(f.to(b)))),
            ("logits", lambda: route(x=d(f), ldl=9)),
            ("topk_idx", lambda: route(idx=d(i.long()))),
            ("topk_w", lambda: route(w=d(torch.zeros(4, 1)))),
            ("x", lambda: permute(x=d(f.t()))), ("rows", lambda: permute(rows=d(f))),
            ("offsets", lambda: permute(offsets=d(torch.zeros(8, dtype=torch.int32)))),
            ("ws", lambda: permute(ws_bytes=512)),
            ("y", lambda: combine(y=d(f))), ("out", lambda: combine(out=d(f.to(b)))),
            ("W", lambda: w4(W=d(torch.zeros(4, 15, dtype=torch.uint8)))),
            ("W", lambda: w4(W=d(torch.zeros(4, 16, dtype=torch.int8)))),
            ("scale", lambda: w4(s=d(torch.zeros(4, 1)))),
            ("zero", lambda: w4(z=d(torch.zeros(3, 1, dtype=torch.uint8)))),
            ("x", lambda: w4(x=d(torch.zeros(1, 31))))]:
        with pytest.raises(qm.QmoeError) as ei:
            call()
        assert ei.value.status == INV and f": {name} " in str(ei.value), name


def test_reference_rule_of_routing():
    """The 64-bit form that the GPU tests use, on cases worked out by hand."""
    import numpy as np
    nan, inf = np.nan, np.inf
    idx, w, _ = ref.route([[0, 1, 1, -inf], [nan, 0, 1, 2], [-inf] * 4, [-inf, -inf, 3, -inf]], 2,
                          True)
    assert idx.tolist() == [[1, 2], [0, 1], [0, 1], [2, 0]]
    assert w[0].tolist() == [0.5, 0.5] and np.isnan(w[1:3]).all() and w[3].tolist() == [1.0, 0.0]
    off, pos = ref.permute(np.array([[2, 0], [0, -1], [2, 2]]), 3)
    assert off.tolist() == [0, 2, 2, 5] and pos.tolist() == [[2, 0], [1, -1], [3, 4]]
