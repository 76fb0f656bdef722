"""GPU tests of single properties of the e4m3 and grouped products, against the
64-bit forms of tests/f8_ref.py."""
import numpy as np
import pytest

from tests import f8_ref as ref
from tests.test_gpu_f8 import check, dev, f64, f8_operands, out_tensor, wide_operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f8", "bf16"])
@pytest.mark.parametrize("m,n", [(40, 100), (700, 2048)], ids=["few_rows", "pairs"])
def test_bad_offsets_compute_nothing(qm, kind, m, n):
    """Groups whose offsets decrease, overlap or leave x are not computed in
    part: y stays as it was, whatever the other groups hold.  (Clamped, the
    overlapping ones would race for the same rows, and 512 such groups of 2^29
    rows make 2^32 tiles of 64.)"""
    import torch
    g = np.random.default_rng(81)
    k, e = 128, 6
    if kind == "f8":
        xq, xs, wq, ws, xv, wv = f8_operands(g, m, n, k, e)
        args = (qm.E4M3, dev(wq), dev(ws), e, n, k, dev(xq), dev(xs), m)
        terms = ref.f8_terms(k)
    else:
        x, w, xv, wv = wide_operands(g, m, n, k, e, "bf16")
        args = (qm.BF16, w.cuda(), None, e, n, k, x.cuda(), None, m)
        terms = ref.wide_terms(k)
    y = out_tensor(m, n, torch.float32)
    for off in ([0, m, 0, m, 0, m, 0],          # every other group the whole of x
                [0, 9, 5, m, m, m, m],          # one decrease
                [0, 4, 8, 9, 20, 30, m + 1],    # the last row outside
                [-1, 4, 8, 9, 20, 30, m],
                [2**31 - 1, -2**31, 2**31 - 1, 0, 1, 2, 3]):
        qm.mm_grouped(*args, dev(np.array(off, dtype=np.int64).astype(np.int32)), qm.F32, y)
        assert qm.device_status() == qm.ERR_INVALID_ARGUMENT
        assert "offsets" in qm.last_error()
        assert (y == 77.0).all(), off
    good = [0, 7, 7, 20, 21, 30, m]
    qm.mm_grouped(*args, dev(np.int32(good)), qm.F32, y)
    assert qm.device_status() == qm.OK
    for i in range(e):
        r = slice(good[i], good[i + 1])
        if good[i] == good[i + 1]:
            continue
        want, err = ref.product(xv[r], wv[i], terms)
        check(f64(y[r]), want, ref.rounded(want, err, "f32"), f"group {i}")


def test_bad_offsets_past_the_first_scan(qm):
    """1024 groups are scanned in several steps of one CTA's threads: a bad
    offset in the first or the last step stops the call all the same."""
    import torch
    g = np.random.default_rng(82)
    m, n, k, e = 1024, 64, 128, 1024
    x, w, xv, wv = wide_operands(g, m, n, k, 1, "bf16")
    W, X = w.cuda().expand(e, n, k).contiguous(), x.cuda()
    good = np.arange(e + 1, dtype=np.int32)
    for i in (0, 100, 500, 1023, 1024):
        off = good.copy()
        off[i] = -3 if i == 0 else 2000
        y = out_tensor(m, n, torch.float32)
        qm.mm_grouped(qm.BF16, W, None, e, n, k, X, None, m, dev(off), qm.F32, y)
        assert qm.device_status() == qm.ERR_INVALID_ARGUMENT
        assert (y == 77.0).all(), i
    qm.mm_grouped(qm.BF16, W, None, e, n, k, X, None, m, dev(good), qm.F32, y)
    assert qm.device_status() == qm.OK
    want, err = ref.product(xv, wv[0], ref.wide_terms(k))
    check(f64(y), want, ref.rounded(want, err, "f32"), "1024 groups")


# SwiGLU alone: with x = 1, one code per weight row and a down matrix that copies
# one 128-block of the activations into the output, out is the activation after its
# e4m3 rounding.  Every product is exact (powers of two times a four-bit
# significand), so |out - a| is at most half a step of a: 2^-4 |a|, or 2^-10 of the
# block's scale where that is more, and SwiGLU's own error, stated as 2^-20 |a|.
def swiglu_case(qm, tokens, blocks, probe, gates, up):
    import torch
    H, F = 128, 128 * blocks
    table = np.abs(ref.TABLE[:127])
    codes = np.array([int(np.argmin(np.abs(table - abs(v)))) for v in gates], np.uint8)
    gq = np.repeat(codes[:, None], H, axis=1)
    G = np.zeros((1, F, H), np.uint8)
    G[0, probe * 128:probe * 128 + 128] = gq
    U = np.full((1, F, H), 0x38, np.uint8)  # 1.0
    D = np.zeros((1, H, F), np.uint8)
    D[0, np.arange(H), probe * 128 + np.arange(H)] = 0x38
    one = lambda v, *s: dev(np.full((1,) + s, v, np.float32))
    sign = np.float32(np.sign(gates[0]))
    shape = qm.moe_shape(H, F, 1, 1, tokens, qm.E4M3, qm.E4M3, qm.E4M3)
    ws = torch.empty(qm.moe_experts_f8_workspace_size(shape), dtype=torch.uint8, device="cuda")
    out = out_tensor(tokens, H, torch.float32)
    qm.moe_experts_f8(dev(G), one(sign / 128, blocks, 1), dev(U), one(up / 128, blocks, 1), dev(D),
                      one(1.0, 1, blocks), shape, qm.F32, torch.ones(tokens, H, device="cuda"),
                      torch.zeros(tokens, 1, dtype=torch.int32, device="cuda"),
                      torch.ones(tokens, 1, device="cuda"), None, out, ws)
    assert qm.device_status() == qm.OK
    g = float(sign) * table[codes]
    a = g / (1.0 + np.exp(-g)) * up
    scale = float(ref.block_scale(np.abs(a).max()))
    tol = np.maximum(2.0 ** -4 * np.abs(a), 2.0 ** -10 * scale) + 2.0 ** -20 * np.abs(a)
    check(f64(out), np.broadcast_to(a, (tokens, H)), tol, f"SwiGLU of {gates[0]}..{gates[-1]}")


@pytest.mark.parametrize("tokens,blocks,probe", [(1, 1, 0), (20, 3, 1), (600, 10, 3), (600, 11, 10)],
                         ids=["one", "few_rows", "pairs", "pairs_odd"])
@pytest.mark.parametrize("gates,up", [
    (np.linspace(0.01, 20.0, 128), 1.0), (-np.linspace(0.01, 20.0, 128), 1.0),
    (np.linspace(20.0, 448.0, 128), 2.0 ** -3), (-np.linspace(20.0, 87.0, 128), 2.0 ** 20),
    # far below zero: silu is 2^-120 and smaller, and up brings it back
    (-np.full(128, 88.0), 2.0 ** 100), (-np.linspace(80.0, 88.0, 128), 2.0 ** 90)],
    ids=["positive", "negative", "large", "small", "far", "far_mixed"])
def test_swiglu_over_its_range(qm, tokens, blocks, probe, gates, up):
    swiglu_case(qm, tokens, blocks, probe, gates, up)


@pytest.mark.parametrize("m,n", [(3, 200), (300, 2100)], ids=["few_rows", "pairs"])
def test_scale_products_below_the_normal_range(qm, m, n):
    """The product of two scales is an f32 of its own: below 2^-126 it is a
    subnormal with fewer bits, and 0 below 2^-150.  y is the sum with that product,
    not with the exact one.  One block of K, so the inner sum times one product."""
    import torch
    g = np.random.default_rng(83)
    k = 128
    xq, _, wq, _, _, _ = f8_operands(g, m, n, k)
    xs = np.exp2(g.uniform(-90, -60, (m, 1))).astype(np.float32)
    ws = np.exp2(g.uniform(-75, -40, (1, -(-n // 128), 1))).astype(np.float32)
    xs[0], xs[1] = np.float32(2.0 ** -80), np.float32(2.0 ** -126)
    ws[0, 0] = np.float32(1.7 * 2.0 ** -60)  # row 0: 1.7 x 2^-140; row 1: 0
    y = out_tensor(m, n, torch.float32)
    qm.f8_mm(dev(wq[0]), dev(ws[0]), n, k, dev(xq), dev(xs), m, qm.F32, y)
    assert qm.device_status() == qm.OK
    with np.errstate(under="ignore"):
        sp = (xs * np.repeat(ws[0], 128, axis=0)[:n, 0][None, :]).astype(np.float32)
    sp = sp.astype(np.float64)
    assert (sp[1, :128] == 0).all() and ((sp > 0) & (sp < 2.0 ** -126)).any()
    xv, wv = ref.TABLE[xq], ref.TABLE[wq[0]]
    s, err = ref.product(xv, wv, ref.f8_terms(k))
    check(f64(y), s * sp, ref.rounded(s * sp, err * sp, "f32"), "subnormal scale products")
