"""The binding refuses integers that the library's C types would cut to other ones: a type,
size or byte count that then passes the checks here and means another array there."""
import pytest

import moe_ffn_gb300 as qm
from tests.test_f8_abi import INV, OnDevice, lib, shape  # noqa: F401  (lib is a fixture)

torch = pytest.importorskip("torch")
W32, W64 = 1 << 32, 1 << 64


def f(*s):
    return OnDevice(torch.zeros(*s))


def i(*s):
    return OnDevice(torch.zeros(*s, dtype=torch.int32))


def u(*s):
    return OnDevice(torch.zeros(*s, dtype=torch.uint8))


CALLS = {  # name: (call, arguments of 32 bits, arguments of 64)
    "moe_route": (lambda **a: qm.moe_route(**{**dict(
        ltype=0, logits=f(4, 8), n_tokens=4, num_experts=8, top_k=2, topk_idx=i(4, 2),
        topk_w=f(4, 2), ldl=8, stream=0), **a}),
        ("ltype", "num_experts", "top_k"), ("n_tokens", "ldl")),
    "moe_route_backward": (lambda **a: qm.moe_route_backward(**{**dict(
        ltype=0, logits=f(4, 8), n_tokens=4, num_experts=8, top_k=2, topk_idx=i(4, 2),
        topk_w=f(4, 2), grad_w=f(4, 2), grad_logits=f(4, 8), ldl=8, ldg=8, stream=0), **a}),
        ("ltype", "num_experts", "top_k"), ("n_tokens", "ldl", "ldg")),
    "moe_permute": (lambda **a: qm.moe_permute(**{**dict(
        xtype=0, x=f(4, 8), n_tokens=4, cols=8, topk_idx=i(4, 2), num_experts=8, top_k=2,
        rows=f(8, 8), offsets=i(9), pos=i(4, 2), ws=u(256), ldx=8, ldr=8, ws_bytes=256, stream=0),
        **a}), ("xtype", "num_experts", "top_k"), ("n_tokens", "cols", "ldx", "ldr")),
    "moe_permute_workspace_size": (lambda **a: qm.moe_permute_workspace_size(**{**dict(
        n_tokens=4, num_experts=8, top_k=2), **a}), ("num_experts", "top_k"), ("n_tokens",)),
    "moe_combine": (lambda **a: qm.moe_combine(**{**dict(
        ytype=0, y=f(8, 8), n_rows=8, cols=8, pos=i(4, 2), topk_w=None, n_tokens=4, top_k=2,
        otype=0, residual=None, out=f(4, 8), ldy=8, ldo=8, stream=0), **a}),
        ("ytype", "otype", "top_k"), ("n_rows", "cols", "n_tokens", "ldy", "ldo")),
    "moe_combine_backward": (lambda **a: qm.moe_combine_backward(**{**dict(
        ytype=0, y=f(8, 8), n_rows=8, cols=8, pos=i(4, 2), topk_w=None, n_tokens=4, top_k=2,
        otype=0, grad_out=f(4, 8), grad_y=f(8, 8), grad_w=f(4, 2), ldy=8, ldo=8, ldg=8, stream=0),
        **a}), ("ytype", "otype", "top_k"), ("n_rows", "cols", "n_tokens", "ldy", "ldo", "ldg")),
    "w4_mm": (lambda **a: qm.w4_mm(**{**dict(
        W=u(4, 32), stype=0, scale=f(4, 2), zero=None, scale_cols=32, rows=4, cols=64, xtype=0,
        x=f(1, 64), n_tokens=1, ytype=0, y=f(1, 4), ldx=64, ldy=4, stream=0), **a}),
        ("stype", "scale_cols", "xtype", "ytype"), ("rows", "cols", "n_tokens", "ldx", "ldy")),
    "w4_mm_grouped": (lambda **a: qm.w4_mm_grouped(**{**dict(
        W=u(2, 4, 32), stype=0, scale=f(2, 4, 2), zero=None, scale_cols=32, num_groups=2, rows=4,
        cols=64, xtype=0, x=f(1, 64), n_rows=1, offsets=i(3), ytype=0, y=f(1, 4), ldx=64, ldy=4,
        stream=0), **a}), ("stype", "scale_cols", "num_groups", "xtype", "ytype"),
        ("rows", "cols", "n_rows", "ldx", "ldy")),
    "f8_quantize": (lambda **a: qm.f8_quantize(**{**dict(
        xtype=0, x=f(2, 128), rows=2, cols=128, q=u(2, 128), scale=f(2, 1), ldx=128, stream=0),
        **a}), ("xtype",), ("rows", "cols", "ldx")),
    "f8_mm": (lambda **a: qm.f8_mm(**{**dict(
        W=u(128, 128), w_scale=f(1, 1), rows=128, cols=128, x=u(1, 128), x_scale=f(1, 1),
        n_tokens=1, ytype=0, y=f(1, 128), ldx=128, ldy=128, stream=0), **a}),
        ("ytype",), ("rows", "cols", "n_tokens", "ldx", "ldy")),
    "mm_grouped": (lambda **a: qm.mm_grouped(**{**dict(
        wtype=qm.E4M3, W=u(2, 128, 128), w_scale=f(2, 1), num_groups=2, rows=128, cols=128,
        x=u(1, 128), x_scale=f(1, 1), n_rows=1, offsets=i(3), ytype=0, y=f(1, 128), ldx=128,
        ldy=128, stream=0), **a}),
        ("wtype", "num_groups", "ytype"), ("rows", "cols", "n_rows", "ldx", "ldy")),
}


@pytest.mark.parametrize("name,arg,wide", [
    (n, a, w) for n, (_, small, large) in CALLS.items()
    for a, ws in [(a, (W32, -W32)) for a in small] + [(a, (W64, -W64)) for a in large]
    for w in ws])
def test_wide_integers_are_refused(lib, name, arg, wide):  # noqa: F811
    """The value 2^32 (2^64) from the right one, which the library would take for it."""
    call = CALLS[name][0]
    right = {"scale_cols": 32, "num_groups": 2, "num_experts": 8, "top_k": 2, "wtype": qm.E4M3}
    with pytest.raises(qm.QmoeError) as e:
        call(**{arg: wide + right.get(arg, 1 if arg in ("n_tokens", "n_rows", "rows") else
                                      0 if "type" in arg else 128)})
    assert e.value.status == INV and "does not fit" in str(e.value)
    assert str(e.value).startswith(f"INVALID_ARGUMENT: {name}: ")


@pytest.mark.parametrize("n", [-1, -257, W64 + 256])
def test_byte_counts_are_not_cut_either(lib, n):  # noqa: F811
    for call in (lambda: CALLS["moe_permute"][0](ws_bytes=n),
                 lambda: qm.moe_experts_f8(*[None] * 6, shape(n_tokens=0), qm.BF16, *[None] * 5,
                                           u(256), ws_bytes=n, stream=0)):
        with pytest.raises(qm.QmoeError) as e:
            call()
        assert e.value.status == INV and "does not fit" in str(e.value)


def test_xtype_of_the_e4m3_layer(lib):  # noqa: F811
    with pytest.raises(qm.QmoeError, match="does not fit"):
        qm.moe_experts_f8(*[None] * 6, shape(n_tokens=0), W32, *[None] * 5, u(4096), stream=0)


def test_calls_as_they_stand_pass_the_binding(lib):  # noqa: F811
    """Without a device the library's answer is that there is none."""
    if torch.cuda.is_available():
        pytest.skip("host tensors must not reach a kernel")
    for name, (call, _, _) in CALLS.items():
        if name == "moe_permute_workspace_size":
            assert call() == 256
            continue
        with pytest.raises(qm.QmoeError) as e:
            call()
        assert e.value.status != INV and "does not fit" not in str(e.value), name
