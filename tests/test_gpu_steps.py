"""GPU tests of moe_route, moe_permute, moe_combine and their gradients against the
64-bit forms of tests/steps_ref.py, whose header derives the tolerances."""
import numpy as np
import pytest

from tests import steps_ref as ref
from tests.test_gpu_f8 import check, dev, f64, kinds

pytestmark = pytest.mark.gpu
TYPES = ["f32", "bf16", "f16"]


def strided(values, kind, qm, ld=None, offset=0, fill=77.0):
    """A device array of rows `ld` apart, `offset` elements into its storage;
    (the rows' view, the whole store)."""
    import torch
    code, dt = kinds(qm)[kind]
    n, k = values.shape
    ld = ld or k
    store = torch.full((offset + n * ld + 8,), fill, dtype=dt, device="cuda")
    view = store[offset:offset + n * ld].view(n, ld)
    view[:, :k] = torch.from_numpy(np.ascontiguousarray(values)).to(dt).cuda()
    return view, store


# ------------------------------------------------------------------- routing
def run_route(qm, logits, kind, k, renorm, ld=None, offset=0):
    import torch
    code, _ = kinds(qm)[kind]
    t, e = logits.shape
    x, _ = strided(logits, kind, qm, ld, offset)
    idx = torch.full((t * k + 4,), -7, dtype=torch.int32, device="cuda")
    w = torch.full((t * k + 4,), -7.0, device="cuda")
    qm.moe_route(code, x, t, e, k, idx, w, renormalize=renorm, ldl=ld)
    torch.cuda.synchronize()
    assert (idx[t * k:] == -7).all() and (w[t * k:] == -7).all()
    return f64(x[:, :e]), idx[:t * k].view(t, k), w[:t * k].view(t, k), x


def check_route(qm, logits, kind, k, renorm, **kw):
    xv, idx, w, _ = run_route(qm, logits, kind, k, renorm, **kw)
    want_idx, want_w, tol = ref.route(xv, k, renorm)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    check(f64(w), want_w, tol, "weights")


ROUTE_SHAPES = [(1, 128, 8), (1, 1, 1), (3, 2, 2), (5, 31, 7), (4, 33, 16), (2, 64, 8), (7, 100, 3),
                (9, 129, 8), (6, 200, 10), (33, 256, 8), (5, 500, 16), (3, 1000, 16), (2, 1024, 1)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t,e,k", ROUTE_SHAPES)
def test_route(qm, kind, renorm, t, e, k):
    g = np.random.default_rng(t + 3 * e + 5 * k)
    check_route(qm, 2 * g.standard_normal((t, e)), kind, k, renorm)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ld,offset", [(64, 0), (72, 8), (65, 0), (66, 1), (64, 2), (68, 4)])
def test_route_strides(qm, kind, ld, offset):
    g = np.random.default_rng(ld + offset)
    check_route(qm, g.standard_normal((9, 64)), kind, 6, False, ld=ld, offset=offset)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("renorm", [True, False])
def test_route_ties_masks_and_non_finite_logits(qm, kind, renorm):
    inf, nan = np.inf, np.nan
    low = {"f32": -3.4028235e38, "bf16": -3.3895314e38, "f16": -65504.0}[kind]
    e = 40
    rows = [np.zeros(e), np.full(e, low), np.full(e, -inf), np.full(e, nan)]
    r = np.arange(e) % 3.0
    rows += [r, -r, np.where(np.arange(e) % 2, 0.0, -0.0)]
    for at, v in [(0, nan), (39, nan), (17, inf), (5, -inf), (20, -low), (31, low)]:
        r = np.linspace(-1, 1, e)
        r[at] = v
        rows.append(r)
    r = np.full(e, -inf)
    r[33] = 2.0
    rows.append(r)                       # one expert left
    rows.append(np.where(np.arange(e) < 38, low, 1.0))   # two left, by the lowest value
    rows.append(np.linspace(-80, 0, e))
    check_route(qm, np.stack(rows), kind, 8, renorm)


def run_route_backward(qm, logits, kind, idx, w, dw, renorm, ldl=None, ldg=None, offset=0):
    import torch
    code, dt = kinds(qm)[kind]
    t, e = logits.shape
    k = idx.shape[1]
    x, _ = strided(logits, kind, qm, ldl, offset)
    grad, store = strided(np.full((t, e), 55.0), kind, qm, ldg, offset)
    qm.moe_route_backward(code, x, t, e, k, dev(idx.astype(np.int32)), dev(w.astype(np.float32)),
                          dev(dw.astype(np.float32)), grad, renormalize=renorm, ldl=ldl, ldg=ldg)
    torch.cuda.synchronize()
    assert (grad[:, e:] == 77.0).all() and (store[:offset] == 77.0).all()
    assert (store[offset + grad.numel():] == 77.0).all()
    want, tol = ref.route_backward(f64(x[:, :e]), idx, w.astype(np.float32), dw.astype(np.float32),
                                   renorm)
    check(f64(grad[:, :e]), want, ref.rounded(want, tol, kind), "gradient")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t,e,k", ROUTE_SHAPES)
def test_route_backward(qm, kind, renorm, t, e, k):
    g = np.random.default_rng(t + 3 * e + 5 * k)
    logits = 2 * g.standard_normal((t, e))
    _, idx, w, _ = run_route(qm, logits, kind, k, renorm)
    run_route_backward(qm, logits, kind, idx.cpu().numpy(), w.cpu().numpy(),
                       g.standard_normal((t, k)), renorm)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("ldl,ldg,offset", [(64, 72, 0), (72, 65, 8), (65, 64, 0), (66, 66, 1)])
def test_route_backward_strides_padding_and_repeats(qm, kind, renorm, ldl, ldg, offset):
    """Slots without an expert (their weights are not looked at) and experts named
    twice; a row without any."""
    g = np.random.default_rng(ldl + ldg)
    t, e, k = 6, 64, 5
    logits = g.standard_normal((t, e))
    idx = g.integers(0, e, (t, k))
    idx[0, 1] = idx[0, 4]
    idx[1, :3] = [-1, e, 2 ** 31 - 1]
    idx[2] = -1
    w = g.random((t, k))
    w[1, :3] = np.nan
    run_route_backward(qm, logits, kind, idx, w, g.standard_normal((t, k)), renorm, ldl, ldg,
                       offset)


@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_masks_and_nan(qm, renorm):
    e, k = 20, 4
    rows = np.stack([np.full(e, -np.inf), np.linspace(-3, 3, e), np.linspace(-3, 3, e)])
    rows[1, :17] = -np.inf   # three experts left for four slots
    rows[2, 4] = np.nan
    _, idx, w, _ = run_route(qm, rows, "f32", k, renorm)
    run_route_backward(qm, rows, "f32", idx.cpu().numpy(), w.cpu().numpy(),
                       np.arange(12.0).reshape(3, 4), renorm)


def test_route_gradient_against_differences(qm):
    """Both forms against central differences of the 64-bit weights (step 2^-12: the
    truncation is of the order of its square, 2^-24 of third derivatives below 4)."""
    g = np.random.default_rng(3)
    t, e, k, h = 4, 24, 5, 2.0 ** -12
    logits = g.standard_normal((t, e)).astype(np.float32).astype(np.float64)
    dw = g.standard_normal((t, k)).astype(np.float32)
    import torch
    for renorm in (True, False):
        x, idx, w, xt = run_route(qm, logits, "f32", k, renorm)
        grad = torch.empty(t, e, device="cuda")
        qm.moe_route_backward(qm.F32, xt, t, e, k, idx, w, dev(dw), grad, renormalize=renorm)
        i = idx.cpu().numpy()

        def loss(z):
            p = np.exp(z - z.max(1, keepdims=True))
            sel = np.take_along_axis(p, i, 1)
            return ((sel / (sel if renorm else p).sum(1, keepdims=True)) * dw).sum()
        for a in range(t):
            for b in range(e):
                d = np.zeros((t, e))
                d[a, b] = h
                want = (loss(x + d) - loss(x - d)) / (2 * h)
                # |third derivative| <= 6 sum |dw|; u for the f32 gradient's own error
                tol = h * h * np.abs(dw[a]).sum() + 64 * ref.U * np.abs(dw[a]).sum()
                assert abs(float(grad[a, b]) - want) <= tol, (renorm, a, b)


# ------------------------------------------------------------------- permute
def run_permute(qm, x, kind, idx, e, ldx=None, ldr=None, offset=0, stream=None):
    import torch
    code, dt = kinds(qm)[kind]
    (t, h), k = x.shape, idx.shape[1]
    xt, _ = strided(x, kind, qm, ldx, offset)
    rows, store = strided(np.full((t * k, h), 55.0), kind, qm, ldr, offset)
    off = torch.full((e + 3,), -7, dtype=torch.int32, device="cuda")
    pos = torch.full((t * k + 2,), -7, dtype=torch.int32, device="cuda")
    ws = torch.full((qm.moe_permute_workspace_size(t, e, k),), 0xEE, dtype=torch.uint8,
                    device="cuda")
    qm.moe_permute(code, xt, t, h, dev(idx.astype(np.int32)), e, k, rows, off, pos, ws, ldx=ldx,
                   ldr=ldr)
    torch.cuda.synchronize()
    want_off, want_pos = ref.permute(idx, e)
    assert np.array_equal(off[:e + 1].cpu().numpy(), want_off)
    assert np.array_equal(pos[:t * k].view(t, k).cpu().numpy(), want_pos)
    assert (off[e + 1:] == -7).all() and (pos[t * k:] == -7).all()
    n = int(want_off[-1])
    flat = want_pos.reshape(-1)
    src = np.empty(n, np.int64)
    src[flat[flat >= 0]] = np.nonzero(flat >= 0)[0] // k
    src = torch.from_numpy(src).cuda()
    assert torch.equal(rows[:n, :h], xt[src, :h])
    assert (rows[n:, :h] == 55.0).all()
    if ldr:
        assert (rows[:, h:] == 77.0).all()
    assert (store[:offset] == 77.0).all() and (store[offset + rows.numel():] == 77.0).all()


PERMUTE_SHAPES = [  # tokens, cols, experts, top_k
    (1, 2048, 128, 8), (1, 1, 1, 1), (2, 7, 3, 2), (3, 130, 5, 4), (17, 264, 64, 6),
    (100, 72, 16, 16), (300, 40, 1024, 3), (513, 96, 128, 8), (1024, 16, 8, 8),   # P = 8192
    (1025, 16, 8, 8), (2000, 33, 128, 8), (5000, 8, 1024, 2), (9000, 5, 3, 1), (700, 24, 256, 16),
    (1, 40000, 4, 2), (40, 5000, 9, 3),
]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t,h,e,k", PERMUTE_SHAPES)
def test_permute(qm, kind, t, h, e, k):
    g = np.random.default_rng(t + h + e + k)
    run_permute(qm, g.standard_normal((t, h)), kind, g.integers(0, e, (t, k)), e)


@pytest.mark.parametrize("t,e", [(20000, 128), (40000, 3)])
def test_permute_long_runs(qm, t, e):
    """More than 1024 pairs in a CTA's run (66 and 132 tokens of 16 slots): their rows do
    not all fit in its table and the rest are read back from pos."""
    g = np.random.default_rng(t)
    idx = g.integers(0, e, (t, 16))
    idx[g.random(idx.shape) < 0.05] = -1
    run_permute(qm, g.standard_normal((t, 4)), "bf16", idx, e)


@pytest.mark.parametrize("t", [1, 40, 1500])
def test_permute_padding(qm, t):
    """Slots outside [0, E), experts without rows, tokens without any, all padded, and
    more slots than experts."""
    g = np.random.default_rng(t)
    x = g.standard_normal((t, 24))
    idx = g.integers(-3, 9, (t, 7))
    idx[g.random(t) < 0.2] = -1
    idx[0, 0] = 2 ** 31 - 1
    idx[-1, -1] = -2 ** 31
    run_permute(qm, x, "bf16", idx, 5)
    run_permute(qm, x, "f32", np.full((t, 7), -1), 5)
    run_permute(qm, x, "f16", np.full((t, 7), 4), 5)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("h,ldx,ldr,offset", [(64, 72, 80, 0), (64, 65, 64, 0), (64, 64, 64, 1),
                                              (64, 66, 70, 2), (63, 63, 64, 0), (62, 64, 62, 4)])
def test_permute_strides(qm, kind, h, ldx, ldr, offset):
    g = np.random.default_rng(h + ldx + ldr)
    run_permute(qm, g.standard_normal((37, h)), kind, g.integers(0, 6, (37, 3)), 6, ldx, ldr,
                offset)


def test_permute_no_tokens(qm):
    import torch
    off = torch.full((9,), -7, dtype=torch.int32, device="cuda")
    qm.moe_permute(qm.F32, None, 0, 16, None, 8, 2, None, off, None, None)
    assert (off == 0).all()


# ------------------------------------------------------------------- combine
def routed(g, t, e, k, pad=0.0, rows=None):
    idx = g.integers(0, e, (t, k))
    idx[g.random((t, k)) < pad] = -1
    return ref.permute(idx, e)[1]


def run_combine(qm, kind, okind, t, h, k, pos, n_rows, weights=True, residual=True, ldy=None,
                ldo=None, offset=0, seed=0, alias=False):
    import torch
    g = np.random.default_rng(seed)
    (yc, _), (oc, _) = kinds(qm)[kind], kinds(qm)[okind]
    y, _ = strided(g.standard_normal((n_rows, h)), kind, qm, ldy, offset)
    w = g.standard_normal((t, k)).astype(np.float32)
    res, _ = strided(g.standard_normal((t, h)), okind, qm, ldo, offset)
    rv = f64(res[:, :h]) if residual else None
    out, store = (res, None) if alias else strided(np.full((t, h), 55.0), okind, qm, ldo, offset)
    qm.moe_combine(yc, y, n_rows, h, dev(pos.astype(np.int32)), dev(w) if weights else None, t, k,
                   oc, res if residual else None, out, ldy=ldy, ldo=ldo)
    torch.cuda.synchronize()
    want, tol = ref.combine(f64(y[:, :h]), pos, w.astype(np.float64) if weights else None, rv)
    check(f64(out[:, :h]), want, ref.rounded(want, tol, okind), "combine")
    if ldo:
        assert (out[:, h:] == 77.0).all()
    if store is not None:
        assert (store[:offset] == 77.0).all() and (store[offset + out.numel():] == 77.0).all()


COMBINE_SHAPES = [(1, 2048, 8), (1, 1, 1), (3, 130, 2), (17, 264, 6), (40, 1000, 16), (5, 7, 9),
                  (300, 96, 8), (2, 20000, 3)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("okind", TYPES)
@pytest.mark.parametrize("t,h,k", COMBINE_SHAPES)
def test_combine(qm, kind, okind, t, h, k):
    g = np.random.default_rng(t + h + k)
    run_combine(qm, kind, okind, t, h, k, routed(g, t, 11, k), t * k, seed=h)


@pytest.mark.parametrize("weights,residual,alias", [(False, True, False), (True, False, False),
                                                    (False, False, False), (True, True, True)])
def test_combine_without_weights_or_residual_and_in_place(qm, weights, residual, alias):
    g = np.random.default_rng(1)
    run_combine(qm, "bf16", "f32", 50, 72, 5, routed(g, 50, 8, 5, 0.2), 250, weights, residual,
                alias=alias)


@pytest.mark.parametrize("kind,okind", [("bf16", "bf16"), ("f32", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("h,ldy,ldo,offset", [(64, 72, 80, 0), (64, 65, 64, 0), (64, 64, 64, 1),
                                              (64, 64, 66, 8), (60, 64, 64, 0)])
def test_combine_strides(qm, kind, okind, h, ldy, ldo, offset):
    g = np.random.default_rng(h + ldy)
    run_combine(qm, kind, okind, 19, h, 4, routed(g, 19, 6, 4), 76, ldy=ldy, ldo=ldo,
                offset=offset)


def test_combine_rows_out_of_range_add_nothing(qm):
    """Positions outside [0, n_rows), a row named twice, infinities in rows that no
    slot names and NaN weights of slots without a row."""
    import torch
    g = np.random.default_rng(2)
    t, h, k, n = 6, 40, 5, 9
    pos = g.integers(0, n - 1, (t, k))
    pos[0] = [-1, n, 2 ** 31 - 1, -2 ** 31, 3]
    pos[1] = -1
    pos[2, 1] = pos[2, 2]
    y = g.standard_normal((n, h)).astype(np.float32)
    y[n - 1] = np.inf
    w = g.standard_normal((t, k)).astype(np.float32)
    w[0, :4] = np.nan
    out = torch.full((t, h), 55.0, device="cuda")
    qm.moe_combine(qm.F32, dev(y), n, h, dev(pos.astype(np.int32)), dev(w), t, k, qm.F32, None, out)
    want, tol = ref.combine(y.astype(np.float64), pos, w.astype(np.float64), None)
    check(f64(out), want, ref.rounded(want, tol, "f32"), "combine")
    qm.moe_combine(qm.F32, None, 0, h, dev(pos.astype(np.int32)), dev(w), t, k, qm.F32, None, out)
    assert (out == 0).all()


def test_combine_nan_and_infinities_stay_in_their_tokens(qm):
    import torch
    y = np.ones((8, 16), np.float32)
    y[2, 3], y[5, 7], y[6, 0] = np.nan, np.inf, np.inf
    pos = np.arange(8, dtype=np.int32).reshape(4, 2)
    w = np.array([[1, 1], [1, 1], [1, -1], [0, 1]], np.float32)
    out = torch.empty(4, 16, device="cuda")
    qm.moe_combine(qm.F32, dev(y), 8, 16, dev(pos), dev(w), 4, 2, qm.F32, None, out)
    want = np.einsum("tk,tkh->th", w, y.reshape(4, 2, 16))   # row 3: 0 inf = NaN
    assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)


def run_combine_backward(qm, kind, okind, t, h, k, pos, n_rows, weights=True, ld=None, offset=0,
                         want_y=True, want_w=True, seed=0):
    import torch
    g = np.random.default_rng(seed)
    (yc, _), (oc, _) = kinds(qm)[kind], kinds(qm)[okind]
    y, _ = strided(g.standard_normal((n_rows, h)), kind, qm, ld, offset)
    go, _ = strided(g.standard_normal((t, h)), okind, qm, ld, offset)
    gy, store = strided(np.full((n_rows, h), 55.0), kind, qm, ld, offset)
    w = g.standard_normal((t, k)).astype(np.float32)
    gw = torch.full((t * k + 2,), 55.0, device="cuda")
    qm.moe_combine_backward(yc, y if want_w else None, n_rows, h, dev(pos.astype(np.int32)),
                            dev(w) if weights else None, t, k, oc, go, gy if want_y else None,
                            gw if want_w else None, ldy=ld, ldo=ld, ldg=ld)
    torch.cuda.synchronize()
    wy, ww, tol = ref.combine_backward(f64(y[:, :h]), pos, w.astype(np.float64) if weights else None,
                                       f64(go[:, :h]), n_rows)
    wy = np.where(np.isnan(wy), 55.0, wy) if want_y else np.full((n_rows, h), 55.0)
    check(f64(gy[:, :h]), wy, ref.rounded(wy, ref.U * np.abs(wy), kind), "gradient of the rows")
    if want_w:
        check(f64(gw[:t * k]).reshape(t, k), ww, tol + ref.U * np.abs(ww), "gradient of the weights")
    else:
        assert (gw == 55.0).all()
    assert (gw[t * k:] == 55.0).all()
    if ld:
        assert (gy[:, h:] == 77.0).all()
    assert (store[:offset] == 77.0).all() and (store[offset + gy.numel():] == 77.0).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("okind", TYPES)
@pytest.mark.parametrize("t,h,k", COMBINE_SHAPES)
def test_combine_backward(qm, kind, okind, t, h, k):
    g = np.random.default_rng(t + h + k)
    run_combine_backward(qm, kind, okind, t, h, k, routed(g, t, 11, k, 0.1), t * k, seed=h)


@pytest.mark.parametrize("weights,want_y,want_w", [(False, True, True), (True, False, True),
                                                   (True, True, False)])
def test_combine_backward_parts(qm, weights, want_y, want_w):
    g = np.random.default_rng(4)
    run_combine_backward(qm, "bf16", "f32", 50, 72, 5, routed(g, 50, 8, 5, 0.2), 250, weights,
                         want_y=want_y, want_w=want_w)


@pytest.mark.parametrize("kind,okind", [("bf16", "bf16"), ("f32", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("h,ld,offset", [(64, 72, 0), (64, 65, 0), (64, 64, 1), (60, 64, 0)])
def test_combine_backward_strides(qm, kind, okind, h, ld, offset):
    g = np.random.default_rng(h + ld)
    pos = routed(g, 19, 6, 4)
    pos[3, 1] = 76
    run_combine_backward(qm, kind, okind, 19, h, 4, pos, 76, ld=ld, offset=offset)


# ------------------------------------------------------------ all in a run
def layer_inputs(g, t, h, f, e):
    import torch
    bf = torch.bfloat16

    def r(*s):
        return torch.from_numpy(g.standard_normal(s).astype(np.float32)).cuda()
    return (r(t, h).to(bf), (1.5 * r(t, e)), (r(e, f, h) * h ** -0.5).to(bf),
            (r(e, h, f) * f ** -0.5).to(bf))


def layer(qm, x, logits, up, down, k, bufs):
    """One layer through the library: routes, sort, the two products of its experts (a
    plain ReLU between them), weighted sum.  Buffers are made once, so that the
    chain can be captured."""
    import torch
    (t, h), (e, f) = x.shape, up.shape[:2]
    P = t * k
    if not bufs:
        def new(*s, dt=torch.bfloat16):
            return torch.zeros(*s, dtype=dt, device="cuda")
        bufs.update(idx=new(t, k, dt=torch.int32), w=new(t, k, dt=torch.float32), rows=new(P, h),
                    off=new(e + 1, dt=torch.int32), pos=new(t, k, dt=torch.int32), a=new(P, f),
                    y=new(P, h), out=new(t, h, dt=torch.float32),
                    ws=torch.empty(qm.moe_permute_workspace_size(t, e, k), dtype=torch.uint8,
                                   device="cuda"))
    b = bufs
    qm.moe_route(qm.F32, logits, t, e, k, b["idx"], b["w"])
    qm.moe_permute(qm.BF16, x, t, h, b["idx"], e, k, b["rows"], b["off"], b["pos"], b["ws"])
    qm.mm_grouped(qm.BF16, up, None, e, f, h, b["rows"], None, P, b["off"], qm.BF16, b["a"])
    b["a"].clamp_(min=0)
    qm.mm_grouped(qm.BF16, down, None, e, h, f, b["a"], None, P, b["off"], qm.BF16, b["y"])
    qm.moe_combine(qm.BF16, b["y"], P, h, b["pos"], b["w"], t, k, qm.F32, None, b["out"])
    return b["out"]


def layer_backward(qm, x, logits, up, down, k, b, grad):
    """Gradients of x and of the logits for given experts (their transposes are the
    backward products' stacks)."""
    import torch
    (t, h), (e, f) = x.shape, up.shape[:2]
    P = t * k
    gy, ga, gr = (torch.zeros_like(b[i]) for i in ("y", "a", "rows"))
    gw, gl = torch.zeros_like(b["w"]), torch.zeros_like(logits)
    gx = torch.zeros(t, h, device="cuda")
    qm.moe_combine_backward(qm.BF16, b["y"], P, h, b["pos"], b["w"], t, k, qm.F32, grad, gy, gw)
    qm.mm_grouped(qm.BF16, down.transpose(1, 2).contiguous(), None, e, f, h, gy, None, P, b["off"],
                  qm.BF16, ga)
    ga.mul_(b["a"] > 0)
    qm.mm_grouped(qm.BF16, up.transpose(1, 2).contiguous(), None, e, h, f, ga, None, P, b["off"],
                  qm.BF16, gr)
    qm.moe_combine(qm.BF16, gr, P, h, b["pos"], None, t, k, qm.F32, None, gx)
    qm.moe_route_backward(qm.F32, logits, t, e, k, b["idx"], b["w"], gw, gl)
    return gx, gl


def layer64(x, logits, up, down, idx):
    """The same layer in 64 bits by torch's own differentiation, routes given."""
    import torch
    p = torch.softmax(torch.gather(logits, 1, idx), -1)
    out = torch.zeros(x.shape[0], x.shape[1], dtype=torch.float64, device="cuda")
    for s in range(idx.shape[1]):
        a = torch.relu(torch.einsum("th,tfh->tf", x, up[idx[:, s]]))
        out = out + p[:, s:s + 1] * torch.einsum("tf,thf->th", a, down[idx[:, s]])
    return out


@pytest.mark.parametrize("t", [1, 37, 1100])
def test_layer_and_its_gradient(qm, t):
    """Routes, sort, products, weighted sum and all their gradients in a run.  Roundings
    to bf16: of a and of y on the way there; of gy, ga and gr on the way back.  Each is
    2^-8 of a value whose own error passes on; sums of many such grow as their square
    root, and the products add as the tests of mm_grouped bound them (2^-17 of the
    values' size for these lengths).  Checked in the 2-norm over all values: three
    roundings of 2^-8, uncorrelated or not, are at most 3 2^-8 relative to the
    sizes of what they round, which exceed the result's by at most the factor that
    cancellation in the sums costs, below 4 for these normal inputs."""
    import torch
    g = np.random.default_rng(t)
    e, k, h, f = 16, 4, 256, 128
    x, logits, up, down = layer_inputs(g, t, h, f, e)
    bufs = {}
    out = layer(qm, x, logits, up, down, k, bufs)
    assert qm.device_status() == qm.OK
    grad = torch.from_numpy(g.standard_normal((t, h)).astype(np.float32)).cuda()
    gx, gl = layer_backward(qm, x, logits, up, down, k, bufs, grad)
    assert qm.device_status() == qm.OK
    want_idx = ref.route(f64(logits), k, True)[0]
    assert np.array_equal(bufs["idx"].cpu().numpy(), want_idx)
    xd, ld = (v.double().requires_grad_() for v in (x, logits))
    want = layer64(xd, ld, up.double(), down.double(), bufs["idx"].long())
    want.backward(grad.double())
    for name, a, b in (("out", out, want.detach()), ("x", gx, xd.grad), ("logits", gl, ld.grad)):
        off = float((a.double() - b).norm() / b.norm())
        assert off <= 4 * 3 * 2.0 ** -8, (name, off)


def test_captured_layer_with_new_data_on_another_stream(qm):
    """The whole layer captured once and replayed on new data; the same bits as called."""
    import torch
    t, e, k, h, f = 1200, 16, 8, 256, 128   # (sorted by two launches)
    first = layer_inputs(np.random.default_rng(1), t, h, f, e)
    second = layer_inputs(np.random.default_rng(2), t, h, f, e)
    plain = [{}, {}]
    outs = [layer(qm, *inp, k, b).clone() for inp, b in zip((first, second), plain)]
    live = [a.clone() for a in first]
    bufs = {}
    layer(qm, *live, k, bufs)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            layer(qm, *live, k, bufs)
        for inp, want in ((second, outs[1]), (first, outs[0]), (second, outs[1])):
            for a, b in zip(live, inp):
                a.copy_(b)
            bufs["out"].zero_()
            bufs["pos"].fill_(-1)
            graph.replay()
            side.synchronize()
            assert torch.equal(bufs["out"], want)
    assert qm.device_status(side) == qm.OK


def test_two_streams_at_once(qm):
    """Sorts and sums of two streams with their own workspaces do not disturb each other."""
    import torch
    g = np.random.default_rng(9)
    t, e, k, h, f = 1500, 64, 8, 128, 64
    inputs = [layer_inputs(g, t, h, f, e) for _ in range(2)]
    want = [layer(qm, *i, k, {}).clone() for i in inputs]
    torch.cuda.synchronize()
    bufs, streams = [{}, {}], [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for i, b, s in zip(inputs, bufs, streams):
            with torch.cuda.stream(s):
                got.append(layer(qm, *i, k, b))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_beyond_2_31_elements(qm):
    """Positions whose offset in the rows passes 32 bits, there and back: 1,050,000
    rows of 2056 bf16 values.  Each token's rows come back as k times itself."""
    import torch
    t, k, h, e = 131250, 8, 2056, 64
    x = torch.randn(t, h, device="cuda").to(torch.bfloat16)
    idx = torch.randint(0, e, (t, k), device="cuda", dtype=torch.int32)
    rows = torch.empty(t * k, h, dtype=torch.bfloat16, device="cuda")
    off = torch.empty(e + 1, dtype=torch.int32, device="cuda")
    pos = torch.empty(t, k, dtype=torch.int32, device="cuda")
    ws = torch.empty(qm.moe_permute_workspace_size(t, e, k), dtype=torch.uint8, device="cuda")
    assert rows.numel() > 2 ** 31
    qm.moe_permute(qm.BF16, x, t, h, idx, e, k, rows, off, pos, ws)
    flat = idx.view(-1).long()
    order = torch.argsort(flat, stable=True)
    assert torch.equal(pos.view(-1)[order].long(), torch.arange(t * k, device="cuda"))
    for i in (0, 1, 4095, t * k // 2, t * k - 2, t * k - 1):
        assert torch.equal(rows[i], x[order[i] // k])
    out = torch.empty(t, h, device="cuda")
    qm.moe_combine(qm.BF16, rows, t * k, h, pos, None, t, k, qm.F32, None, out)
    # k times a bf16 value is exact in f32
    assert torch.equal(out, k * x.float())
    w = torch.rand(t, k, device="cuda")
    gw = torch.empty(t, k, device="cuda")
    qm.moe_combine_backward(qm.BF16, rows, t * k, h, pos, w, t, k, qm.BF16, x, rows, gw)
    for i in (0, 4095, t * k - 1):
        tok, slot = int(order[i]) // k, int(order[i]) % k
        want = (w[tok, slot] * x[tok].float()).to(torch.bfloat16)
        assert torch.equal(rows[i], want)


def test_named_streams_and_addresses(qm):
    """The checks' long way: a stream object, a stream's address, arrays by address."""
    import torch
    g = np.random.default_rng(6)
    t, e, k, h = 40, 16, 4, 72
    x, logits, _, _ = layer_inputs(g, t, h, 32, e)
    new = {"idx": (t, k), "pos": (t, k), "off": (e + 1,)}
    b = {n: torch.zeros(*s, dtype=torch.int32, device="cuda") for n, s in new.items()}
    b["w"], b["out"] = torch.zeros(t, k, device="cuda"), torch.zeros(t, h, device="cuda")
    b["rows"] = torch.zeros(t * k, h, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(qm.moe_permute_workspace_size(t, e, k), dtype=torch.uint8, device="cuda")

    def run(stream, at):
        qm.moe_route(qm.F32, at(logits), t, e, k, at(b["idx"]), at(b["w"]), stream=stream)
        qm.moe_permute(qm.BF16, at(x), t, h, at(b["idx"]), e, k, at(b["rows"]), at(b["off"]),
                       at(b["pos"]), at(ws), ws_bytes=ws.numel(), stream=stream)
        qm.moe_combine(qm.BF16, at(b["rows"]), t * k, h, at(b["pos"]), at(b["w"]), t, k, qm.F32,
                       None, at(b["out"]), stream=stream)
    run(None, lambda a: a)
    torch.cuda.synchronize()
    want = {n: a.clone() for n, a in b.items()}
    side = torch.cuda.Stream()
    for stream, at in ((side, lambda a: a), (side.cuda_stream, lambda a: a.data_ptr())):
        for a in b.values():
            a.zero_()
        torch.cuda.synchronize()
        run(stream, at)
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], b[n]) for n in b)


def test_sort_beside_an_overlapping_consumer(qm):
    """A chain in which every launch may start before its predecessor has ended, many times
    over: each sort and sum sees the routes and rows of its own turn."""
    import torch
    g = np.random.default_rng(12)
    t, e, k, h = 1300, 32, 8, 64     # (sorted by two launches)
    x, _, _, _ = layer_inputs(g, t, h, 32, e)
    logits = [torch.randn(t, e, device="cuda") for _ in range(6)]
    one = [{}, {}]
    for b in one:
        b.update(idx=torch.zeros(t, k, dtype=torch.int32, device="cuda"),
                 w=torch.zeros(t, k, device="cuda"),
                 pos=torch.zeros(t, k, dtype=torch.int32, device="cuda"),
                 off=torch.zeros(e + 1, dtype=torch.int32, device="cuda"),
                 rows=torch.zeros(t * k, h, dtype=torch.bfloat16, device="cuda"),
                 ws=torch.empty(qm.moe_permute_workspace_size(t, e, k), dtype=torch.uint8,
                                device="cuda"))

    def turn(b, lg, out):
        qm.moe_route(qm.F32, lg, t, e, k, b["idx"], b["w"])
        qm.moe_permute(qm.BF16, x, t, h, b["idx"], e, k, b["rows"], b["off"], b["pos"], b["ws"])
        qm.moe_combine(qm.BF16, b["rows"], t * k, h, b["pos"], b["w"], t, k, qm.F32, None, out)
        return out
    want = []
    for lg in logits:
        want.append(turn(one[0], lg, torch.zeros(t, h, device="cuda")))
        torch.cuda.synchronize()
    outs = [torch.zeros(t, h, device="cuda") for _ in range(60)]
    for i, out in enumerate(outs):
        turn(one[1], logits[i % 6], out)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want[i % 6]) for i, out in enumerate(outs))
    assert qm.device_status() == qm.OK
