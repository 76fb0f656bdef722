"""GPU tests of f8_quantize, f8_mm, mm_grouped and moe_experts_f8 against the
64-bit forms of tests/f8_ref.py, whose header derives the tolerances."""
import numpy as np
import pytest

from tests import f8_ref as ref

pytestmark = pytest.mark.gpu


def kinds(qm):
    import torch
    return {"f32": (qm.F32, torch.float32), "bf16": (qm.BF16, torch.bfloat16),
            "f16": (qm.F16, torch.float16)}


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def check(got, want, tol, what):
    got, want, tol = np.asarray(got), np.asarray(want), np.broadcast_to(tol, np.shape(want))
    assert got.shape == want.shape, what
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN where none is due, or none where one is"
    bad = ~nan & ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) / tol, 0)), got.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; at {i} got {got[i]!r} "
                             f"want {want[i]!r} tol {tol[i]:.3e}")


# ---------------------------------------------------------------- quantise
def run_quantize(qm, x, kind, ldx=None, offset=0):
    """Quantises [rows][cols] values held with rows ldx apart, `offset`
    elements into their storage."""
    import torch
    code, dt = kinds(qm)[kind]
    n, k = x.shape
    ldx = ldx or k
    store = torch.full((offset + n * ldx + 8,), 60000.0, dtype=dt, device="cuda")
    xt = store[offset:offset + n * ldx].view(n, ldx)
    xt[:, :k] = torch.from_numpy(x).to(dt).cuda()
    kb = qm.f8_blocks(k)
    q = torch.full((n * k + 16,), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((n * kb + 4,), -5.0, device="cuda")
    qm.f8_quantize(code, xt, n, k, q, s, ldx=ldx)
    torch.cuda.synchronize()
    assert (q[n * k:] == 0xAA).all() and (s[n * kb:] == -5.0).all()
    return (q[:n * k].view(n, k).cpu().numpy(), f64(s[:n * kb]).reshape(n, kb),
            f64(xt[:, :k]))


def check_quantize(q, s, x):
    wq, ws = ref.quantize(x)
    assert np.array_equal(s, ws)
    nan = ~np.isfinite(x)
    assert np.all((q[nan] & 0x7F) == 0x7F)
    assert np.array_equal(q[~nan], wq[~nan])


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 127), (5, 129), (2, 2048), (17, 1000),
                                   (300, 264), (1, 14336)])
def test_quantize(qm, kind, shape):
    g = np.random.default_rng(shape[0] * 7 + shape[1])
    x = g.standard_normal(shape).astype(np.float32) * np.exp(2 * g.standard_normal((shape[0], 1)))
    q, s, xv = run_quantize(qm, x.astype(np.float32), kind)
    check_quantize(q, s, xv)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ldx,offset", [(264, 0), (272, 8), (271, 0), (264, 1), (300, 3)])
def test_quantize_strides_and_alignment(qm, kind, ldx, offset):
    g = np.random.default_rng(ldx + offset)
    x = g.standard_normal((9, 264)).astype(np.float32)
    q, s, xv = run_quantize(qm, x, kind, ldx, offset)
    check_quantize(q, s, xv)


def test_quantize_edges(qm):
    """Blocks of zeros, signed zeros, NaN and infinities, f32's smallest and
    largest values, and largest values on and next to a scale's border."""
    blocks = []

    def block(*v):
        b = np.zeros(128, np.float32)
        b[:len(v)] = v
        blocks.append(b)
    f32 = np.float32
    block()
    block(-0.0, 0.0)
    block(np.nan, 1.0, -3.0)
    block(np.inf, -np.inf, 2.0)
    block(np.nan, np.inf)
    block(1e-45, 2e-45)
    block(1.1754944e-38, -1e-40)
    block(3.4028235e38, -1.0, 1e38)
    for k in (-126, -20, 0, 3, 100):
        t = f32(448.0) * f32(2.0) ** f32(k)
        block(t, -t / 3)
        block(np.nextafter(t, f32(np.inf)), t / 7)
        block(np.nextafter(t, f32(0)), t / 500, t / 30000, t / 1e6)
    # every midpoint between neighbouring codes (ties), and its neighbours
    mid = ((ref.TABLE[:126] + ref.TABLE[1:127]) / 2).astype(f32)
    for v in (mid, np.nextafter(mid, f32(0)), np.nextafter(mid, f32(1e9)), -mid):
        block(448.0, *v[:63])
        block(448.0, *v[63:])
    x = np.stack(blocks)
    q, s, xv = run_quantize(qm, x, "f32")
    check_quantize(q, s, xv)


# ------------------------------------------------------------- products
def f8_operands(g, m, n, k, e=1):
    """e4m3 rows and stacks with scales of wide range, as 64-bit values too."""
    def codes(*shape):
        c = g.integers(0, 256, shape, dtype=np.uint8)
        return np.where((c & 0x7F) == 0x7F, c ^ 1, c)
    kb, nb = -(-k // 128), -(-n // 128)
    xq, wq = codes(m, k), codes(e, n, k)
    xs = np.exp(g.uniform(-3, 1, (m, kb))).astype(np.float32)
    ws = np.exp(g.uniform(-4, 0, (e, nb, kb))).astype(np.float32)
    xv = ref.row_values(xq, xs.astype(np.float64))
    wv = np.stack([ref.matrix_values(wq[i], ws[i].astype(np.float64)) for i in range(e)])
    return xq, xs, wq, ws, xv, wv


def out_tensor(rows, ld, dt):
    import torch
    return torch.full((rows, ld), 77.0, dtype=dt, device="cuda")


MM_SHAPES = [  # (tokens, rows, cols)
    (1, 1, 16), (1, 128, 128), (1, 4096, 4096), (2, 100, 64), (3, 130, 144), (16, 100, 2048),
    (17, 257, 272), (31, 640, 1040), (32, 128, 4096), (33, 129, 640), (64, 300, 1040),
    (100, 128, 128), (256, 128, 256), (257, 384, 1152), (300, 1000, 512), (1000, 260, 528),
    (600, 2048, 256),
]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", MM_SHAPES)
def test_f8_mm(qm, m, n, k, kind):
    g = np.random.default_rng(m + 3 * n + 5 * k)
    xq, xs, wq, ws, xv, wv = f8_operands(g, m, n, k)
    if kind == "f16":  # keep y inside f16
        xs, xv = xs / 256, xv / 256
    code, dt = kinds(qm)[kind]
    y = out_tensor(m, n, dt)
    qm.f8_mm(dev(wq[0]), dev(ws[0]), n, k, dev(xq), dev(xs), m, code, y)
    assert qm.device_status() == qm.OK
    want, err = ref.product(xv, wv[0], ref.f8_terms(k))
    check(f64(y), want, ref.rounded(want, err, kind), f"f8_mm {m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k", [(5, 150, 272), (300, 260, 400)])
def test_f8_mm_strided(qm, m, n, k):
    """Rows of x and y with gaps: the gaps of y stay as they were."""
    import torch
    g = np.random.default_rng(5)
    xq, xs, wq, ws, xv, wv = f8_operands(g, m, n, k)
    x = torch.full((m, k + 48), 0x7F, dtype=torch.uint8, device="cuda")  # NaN codes between rows
    x[:, :k] = dev(xq)
    y = out_tensor(m, n + 7, torch.float32)
    qm.f8_mm(dev(wq[0]), dev(ws[0]), n, k, x, dev(xs), m, qm.F32, y, ldx=k + 48, ldy=n + 7)
    assert qm.device_status() == qm.OK
    want, err = ref.product(xv, wv[0], ref.f8_terms(k))
    check(f64(y[:, :n]), want, ref.rounded(want, err, "f32"), "strided")
    assert (y[:, n:] == 77.0).all()


@pytest.mark.parametrize("m", [3, 300])
def test_f8_mm_nan_stays_in_its_row_and_column(qm, m):
    import torch
    g = np.random.default_rng(9)
    n, k = 200, 512
    xq, xs, wq, ws, xv, wv = f8_operands(g, m, n, k)
    xq[1, 77] = 0x7F
    wq[0, 150, 300] = 0xFF
    xv[1], wv[0, 150] = 0, 0
    y = out_tensor(m, n, torch.float32)
    qm.f8_mm(dev(wq[0]), dev(ws[0]), n, k, dev(xq), dev(xs), m, qm.F32, y)
    want, err = ref.product(xv, wv[0], ref.f8_terms(k))
    tol = ref.rounded(want, err, "f32")
    want[1, :] = np.nan
    want[:, 150] = np.nan
    check(f64(y), want, tol, "NaN")


GROUPS = [
    ("one", [40]), ("single_rows", [1] * 8), ("gaps", [0, 5, 0, 0, 1, 33, 0]),
    ("uneven", [300, 0, 1, 17, 64, 2]), ("all_in_last", [0, 0, 0, 500]),
    ("many", [i % 4 for i in range(130)]), ("tiles", [256, 257, 255, 16, 512]),
    ("most", [1 if i % 100 == 7 else 0 for i in range(1024)]),
]


def wide_operands(g, m, n, k, e, kind):
    import torch
    dt = torch.bfloat16 if kind == "bf16" else torch.float16
    x = torch.from_numpy(g.standard_normal((m, k))).to(dt)
    w = torch.from_numpy(g.standard_normal((e, n, k)) * 0.1).to(dt)
    return x, w, x.double().numpy(), w.double().numpy()


@pytest.mark.parametrize("kind,out", [("f8", "f32"), ("f8", "bf16"), ("bf16", "bf16"),
                                      ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("name,sizes", GROUPS, ids=[g[0] for g in GROUPS])
@pytest.mark.parametrize("n,k", [(72, 80), (260, 400)])
def test_mm_grouped(qm, kind, out, name, sizes, n, k):
    """Every group against its matrix; rows before the first and after the
    last group stay as they were."""
    e = len(sizes)
    if e == 1024 and n > 72:
        n, k = 40, 48
    lead, tail = 2, 3
    m = lead + sum(sizes) + tail
    g = np.random.default_rng(n + k + m)
    code, dt = kinds(qm)[out]
    off = np.cumsum([lead] + sizes).astype(np.int32)
    y = out_tensor(m, n, dt)
    if kind == "f8":
        xq, xs, wq, ws, xv, wv = f8_operands(g, m, n, k, e)
        if out == "f16":
            xs, xv = xs / 256, xv / 256
        qm.mm_grouped(qm.E4M3, dev(wq), dev(ws), e, n, k, dev(xq), dev(xs), m, dev(off), code, y)
        terms = ref.f8_terms(k)
    else:
        x, w, xv, wv = wide_operands(g, m, n, k, e, kind)
        qm.mm_grouped(kinds(qm)[kind][0], w.cuda(), None, e, n, k, x.cuda(), None, m, dev(off),
                      code, y)
        terms = ref.wide_terms(k)
    assert qm.device_status() == qm.OK
    got = f64(y)
    assert (got[:off[0]] == 77.0).all() and (got[off[-1]:] == 77.0).all()
    for i in range(e):
        r = slice(off[i], off[i + 1])
        if off[i] == off[i + 1]:
            continue
        want, err = ref.product(xv[r], wv[i], terms)
        check(got[r], want, ref.rounded(want, err, out), f"{name} group {i}")


@pytest.mark.parametrize("kind,m,n", [
    # one group: narrow tiles in one pass, wide in one against narrow in two,
    # narrow in two against wide in two (152 SMs)
    ("f8", 260, 4096), ("f8", 640, 4096), ("f8", 1000, 4096), ("f8", 129, 14336),
    ("bf16", 260, 4096), ("bf16", 640, 4096), ("f16", 384, 4096), ("f16", 1030, 4096)])
def test_one_group_of_every_tile_width(qm, kind, m, n):
    import torch
    k = 400 if kind == "f8" else 200
    g = np.random.default_rng(m)
    y = out_tensor(m, n, torch.float32)
    off = dev(np.array([0, m], dtype=np.int32))
    if kind == "f8":
        xq, xs, wq, ws, xv, wv = f8_operands(g, m, n, k)
        qm.mm_grouped(qm.E4M3, dev(wq), dev(ws), 1, n, k, dev(xq), dev(xs), m, off, qm.F32, y)
        z = out_tensor(m, n, torch.float32)
        qm.f8_mm(dev(wq[0]), dev(ws[0]), n, k, dev(xq), dev(xs), m, qm.F32, z)
        assert torch.equal(y, z)
        terms = ref.f8_terms(k)
    else:
        x, w, xv, wv = wide_operands(g, m, n, k, 1, kind)
        qm.mm_grouped(kinds(qm)[kind][0], w.cuda(), None, 1, n, k, x.cuda(), None, m, off, qm.F32,
                      y)
        terms = ref.wide_terms(k)
    assert qm.device_status() == qm.OK
    want, err = ref.product(xv, wv[0], terms)
    check(f64(y), want, ref.rounded(want, err, "f32"), f"{kind} {m}x{n}")


@pytest.mark.parametrize("kind", ["f8", "bf16"])
@pytest.mark.parametrize("sizes", [[300, 90], [600, 0, 700, 1, 260, 129]])
def test_few_groups_of_every_tile_width(qm, kind, sizes):
    import torch
    e, n, k, m = len(sizes), 2048, 272, sum(sizes)
    g = np.random.default_rng(m)
    off = np.cumsum([0] + sizes).astype(np.int32)
    y = out_tensor(m, n, torch.float32)
    if kind == "f8":
        xq, xs, wq, ws, xv, wv = f8_operands(g, m, n, k, e)
        qm.mm_grouped(qm.E4M3, dev(wq), dev(ws), e, n, k, dev(xq), dev(xs), m, dev(off), qm.F32, y)
        terms = ref.f8_terms(k)
    else:
        x, w, xv, wv = wide_operands(g, m, n, k, e, kind)
        qm.mm_grouped(qm.BF16, w.cuda(), None, e, n, k, x.cuda(), None, m, dev(off), qm.F32, y)
        terms = ref.wide_terms(k)
    assert qm.device_status() == qm.OK
    got = f64(y)
    for i in range(e):
        r = slice(off[i], off[i + 1])
        want, err = ref.product(xv[r], wv[i], terms)
        check(got[r], want, ref.rounded(want, err, "f32"), f"group {i}")


@pytest.mark.parametrize("kind", ["f8", "bf16"])
def test_mm_grouped_larger(qm, kind):
    """Several token tiles a group and more tiles than SMs, K over many blocks."""
    import torch
    sizes = [700, 0, 130, 513, 1]
    n, k, e, m = 1100, 1536, 5, sum([700, 0, 130, 513, 1])
    g = np.random.default_rng(4)
    off = np.cumsum([0] + sizes).astype(np.int32)
    y = out_tensor(m, n, torch.float32)
    if kind == "f8":
        xq, xs, wq, ws, xv, wv = f8_operands(g, m, n, k, e)
        qm.mm_grouped(qm.E4M3, dev(wq), dev(ws), e, n, k, dev(xq), dev(xs), m, dev(off), qm.F32, y)
        terms = ref.f8_terms(k)
    else:
        x, w, xv, wv = wide_operands(g, m, n, k, e, kind)
        qm.mm_grouped(qm.BF16, w.cuda(), None, e, n, k, x.cuda(), None, m, dev(off), qm.F32, y)
        terms = ref.wide_terms(k)
    assert qm.device_status() == qm.OK
    for i in range(e):
        r = slice(off[i], off[i + 1])
        want, err = ref.product(xv[r], wv[i], terms)
        check(f64(y[r]), want, ref.rounded(want, err, "f32"), f"group {i}")


@pytest.mark.parametrize("m", [40, 700])
def test_mm_grouped_bad_offsets_are_reported(qm, m):
    """Offsets out of order or out of range (clamped in the kernel: the CPU
    test of the tiles covers the clamping) give a status, and nothing outside
    y is written; the next call works."""
    import torch
    g = np.random.default_rng(6)
    n, k, e = 100, 128, 3
    x, w, xv, wv = wide_operands(g, m, n, k, e, "bf16")
    x, w = x.cuda(), w.cuda()
    y = out_tensor(m + 8, n, torch.float32)
    for off in ([0, 9, 5, m], [0, 4, m + 100, m + 200], [-5, 4, 9, 12]):
        qm.mm_grouped(qm.BF16, w, None, e, n, k, x, None, m, dev(np.int32(off)), qm.F32, y)
        assert qm.device_status() == qm.ERR_INVALID_ARGUMENT
        assert "offsets" in qm.last_error()
        assert (y[m:] == 77.0).all()
    good = np.int32([0, 10, 10, m])
    qm.mm_grouped(qm.BF16, w, None, e, n, k, x, None, m, dev(good), qm.F32, y)
    assert qm.device_status() == qm.OK
    want, err = ref.product(xv[10:], wv[2], ref.wide_terms(k))
    check(f64(y[10:m]), want, ref.rounded(want, err, "f32"), "after bad offsets")


# ------------------------------------------------------------- MoE experts
def stack(g, e, n, k):
    w = g.standard_normal((e, n, k)) / np.sqrt(k)
    nb, kb = n // 128, k // 128
    t = w.reshape(e, nb, 128, kb, 128)
    s = (np.abs(t).max((2, 4)) / 448.0).astype(np.float32)
    q = ref.e4m3_codes(t / s[:, :, None, :, None].astype(np.float64)).reshape(e, n, k)
    return q, s, np.stack([ref.matrix_values(q[i], s[i].astype(np.float64)) for i in range(e)])


def silu(v):
    return v / (1.0 + np.exp(-v))


def moe_reference(x, idx, w, stacks, residual, kind="f32"):
    """(out, error bound before rounding).  The bound carries the products'
    errors through SwiGLU (|silu'| <= 1.1; the two fast f32 functions are within
    2^-20), lets an activation within its error of a rounding border take
    either code, and adds the down product's, the weighted sum's (k terms) and
    the residual addition's roundings.  In bf16 each expert's output is rounded
    to bf16 before the sum: 2^-8 of it (and of its error), half a step."""
    (G, U, D) = stacks
    T, k = idx.shape
    H, F, E = G.shape[2], G.shape[1], G.shape[0]
    xq, xs = ref.quantize(x)
    xv = ref.row_values(xq, xs)
    out = np.zeros((T, H)) if residual is None else residual.astype(np.float64).copy()
    err = np.zeros((T, H))
    mag = np.abs(out)
    for t in range(T):
        for s in range(k):
            e = idx[t, s]
            if e < 0 or e >= E:
                continue
            xt = xv[t:t + 1]
            g, eg = ref.product(xt, G[e], ref.f8_terms(H))
            u, eu = ref.product(xt, U[e], ref.f8_terms(H))
            a = silu(g) * u
            da = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + 2.0 ** -20 * np.abs(a)
            lo_q, lo_s = ref.quantize(a - da)
            hi_q, hi_s = ref.quantize(a + da)
            aq, a_s = ref.quantize(a)
            av = ref.row_values(aq, a_s)
            slack = np.maximum(np.abs(ref.row_values(hi_q, hi_s) - av),
                               np.abs(ref.row_values(lo_q, lo_s) - av))
            # a block whose largest value may cross a scale's border may use
            # the coarser subnormal step
            for b in range(F // 128):
                c = slice(b * 128, b * 128 + 128)
                near = np.abs(a[:, c]).max() * 2.0 ** -18 + da[:, c].max()
                if ref.block_scale(np.abs(a[:, c]).max() - near) != \
                        ref.block_scale(np.abs(a[:, c]).max() + near):
                    slack[:, c] += 2.0 ** -9 * 2 * a_s[:, b:b + 1]
            y, ey = ref.product(av, D[e], ref.f8_terms(F))
            ey = ey + slack @ np.abs(D[e]).T
            if kind == "bf16":
                ey = ref.rounded(y, ey, "bf16")
            out[t] += float(w[t, s]) * y[0]
            err[t] += abs(float(w[t, s])) * ey[0]
            mag[t] += np.abs(float(w[t, s]) * y[0])
    return out, err + (k + 2) * 2.0 ** -24 * mag


MOE = [  # T, H, F, E, k
    (1, 256, 128, 4, 2), (1, 2048, 768, 16, 8), (5, 256, 384, 8, 3), (40, 384, 256, 6, 2),
    (33, 128, 128, 1, 1), (70, 256, 128, 256, 4), (3, 640, 128, 5, 16), (300, 128, 256, 3, 2),
]


def moe_case(seed, T, H, F, E, k, kind):
    import torch
    g = np.random.default_rng(seed)
    dt = dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)[kind]
    x = torch.from_numpy(g.standard_normal((T, H))).to(dt)
    residual = torch.from_numpy(g.standard_normal((T, H))).to(dt)
    idx = np.stack([g.permutation(max(E, k))[:k] % E for _ in range(T)]).astype(np.int32)
    w = g.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    return g, x, residual, idx, w, [stack(g, E, F, H), stack(g, E, F, H), stack(g, E, H, F)]


def run_moe(qm, dims, kind, x, idx, w, st, residual, out=None, ws=None, stream=None):
    import torch
    T, H, F, E, k = dims
    shape = qm.moe_shape(H, F, E, k, T, qm.E4M3, qm.E4M3, qm.E4M3)
    code, dt = kinds(qm)[kind]
    if ws is None:
        ws = torch.full((qm.moe_experts_f8_workspace_size(shape),), 0xFF, dtype=torch.uint8,
                        device="cuda")
    if out is None:
        out = out_tensor(T, H, dt)
    qm.moe_experts_f8(*st, shape, code, x, idx, w, residual, out, ws, stream=stream)
    return out


def dev_stacks(stacks):
    return [t for q, s, _ in stacks for t in (dev(q), dev(s))]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dims", MOE, ids=lambda d: "T{}H{}F{}E{}k{}".format(*d))
def test_moe_experts(qm, dims, kind):
    g, x, residual, idx, w, stacks = moe_case(sum(dims), *dims, kind)
    out = run_moe(qm, dims, kind, x.cuda(), dev(idx), dev(w), dev_stacks(stacks), residual.cuda())
    assert qm.device_status() == qm.OK
    want, err = moe_reference(x.double().numpy(), idx, w, [s[2] for s in stacks],
                              residual.double().numpy(), kind)
    check(f64(out), want, ref.rounded(want, err, kind), "moe")


def test_moe_padding_duplicates_and_aliases(qm):
    """Slots outside [0, E) add nothing, a token of such slots keeps its
    residual, an expert named twice counts twice; without a residual the sum
    starts at zero; out may be the residual."""
    dims = (9, 256, 128, 5, 4)
    g, x, residual, idx, w, stacks = moe_case(3, *dims, "bf16")
    idx[0] = -1
    idx[3, 1:] = [5, -7, 2**31 - 1]
    idx[4] = 2
    idx[8] = -1
    st, X, I, W = dev_stacks(stacks), x.cuda(), dev(idx), dev(w)
    values = [s[2] for s in stacks]
    want, err = moe_reference(x.double().numpy(), idx, w, values, residual.double().numpy(), "bf16")
    R = residual.cuda()
    out = run_moe(qm, dims, "bf16", X, I, W, st, R)
    check(f64(out), want, ref.rounded(want, err, "bf16"), "padded")
    assert (out[0] == R[0]).all() and (out[8] == R[8]).all()
    run_moe(qm, dims, "bf16", X, I, W, st, R, out=R)
    assert (R == out).all()
    bare = run_moe(qm, dims, "bf16", X, I, W, st, None)
    want0, err0 = moe_reference(x.double().numpy(), idx, w, values, None, "bf16")
    check(f64(bare), want0, ref.rounded(want0, err0, "bf16"), "no residual")
    assert (bare[0] == 0).all()
    assert qm.device_status() == qm.OK


def test_moe_all_slots_padded(qm):
    dims = (4, 128, 128, 3, 2)
    g, x, residual, idx, w, stacks = moe_case(8, *dims, "f32")
    idx[:] = -1
    out = run_moe(qm, dims, "f32", x.cuda(), dev(idx), dev(w), dev_stacks(stacks),
                  residual.cuda())
    assert (out.cpu() == residual).all()
    assert qm.device_status() == qm.OK


def test_moe_nan_token_stays_alone(qm):
    dims = (6, 256, 128, 4, 2)
    g, x, residual, idx, w, stacks = moe_case(12, *dims, "bf16")
    st = dev_stacks(stacks)
    args = (dev(idx), dev(w), st, residual.cuda())
    clean = run_moe(qm, dims, "bf16", x.cuda(), *args)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[2, 33] = bad
        out = run_moe(qm, dims, "bf16", y.cuda(), *args)
        assert out[2].isnan().all()
        keep = [0, 1, 3, 4, 5]
        assert (out[keep] == clean[keep]).all()


# ------------------------------------------------- streams, graphs, repeats
def test_same_inputs_same_bits_and_shared_workspace(qm):
    """Repeated calls of several sizes over one workspace give the same bits."""
    import torch
    cases = []
    for dims in ((40, 384, 256, 6, 2), (1, 384, 256, 6, 2), (300, 384, 256, 6, 2)):
        g, x, residual, idx, w, stacks = moe_case(21, *dims, "bf16")
        cases.append((dims, x.cuda(), dev(idx), dev(w), dev_stacks(stacks), residual.cuda()))
    big = qm.moe_shape(384, 256, 6, 2, 300, qm.E4M3, qm.E4M3, qm.E4M3)
    ws = torch.full((qm.moe_experts_f8_workspace_size(big),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    first = [run_moe(qm, c[0], "bf16", c[1], c[2], c[3], c[4], c[5], ws=ws) for c in cases]
    for _ in range(3):
        for c, f in zip(cases, first):
            assert torch.equal(run_moe(qm, c[0], "bf16", c[1], c[2], c[3], c[4], c[5], ws=ws), f)
    assert qm.device_status() == qm.OK


def test_capture_and_replay_with_new_data(qm):
    """The chain quantise -> product -> experts captured into a graph on a
    side stream; replays follow their input buffers."""
    import torch
    dims = (7, 256, 128, 4, 2)
    T, H, F, E, k = dims
    g, x, residual, idx, w, stacks = moe_case(31, *dims, "bf16")
    P, PS, _ = stack(g, 1, H, H)
    P, PS = dev(P[0]), dev(PS[0])
    st = dev_stacks(stacks)
    shape = qm.moe_shape(H, F, E, k, T, qm.E4M3, qm.E4M3, qm.E4M3)
    ws = torch.empty(qm.moe_experts_f8_workspace_size(shape), dtype=torch.uint8, device="cuda")
    X, I, W, R = x.cuda(), dev(idx), dev(w), residual.cuda()
    q = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    s = torch.empty(T, H // 128, device="cuda")
    h, out = out_tensor(T, H, torch.bfloat16), out_tensor(T, H, torch.bfloat16)

    def chain():
        qm.f8_quantize(qm.BF16, X, T, H, q, s)
        qm.f8_mm(P, PS, H, H, q, s, T, qm.BF16, h)
        qm.moe_experts_f8(*st, shape, qm.BF16, h, I, W, R, out, ws)
    chain()
    torch.cuda.synchronize()
    eager = out.clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            chain()
    out.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    X.copy_(X.flip(0) * 2)
    I.copy_(I.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    chain()
    torch.cuda.synchronize()
    assert torch.equal(out, replayed) and not torch.equal(out, eager)
    assert qm.device_status() == qm.OK


def test_chain_matches_reference(qm):
    """A layer as it would be used: quantised activations through a dense
    product, then the experts on its output, one 64-bit pass beside it."""
    import torch
    dims = (11, 384, 256, 8, 2)
    T, H, F, E, k = dims
    g, x, residual, idx, w, stacks = moe_case(41, *dims, "bf16")
    P, PS, PV = stack(g, 1, H, H)
    q = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    s = torch.empty(T, H // 128, device="cuda")
    h = out_tensor(T, H, torch.bfloat16)
    qm.f8_quantize(qm.BF16, x.cuda(), T, H, q, s)
    qm.f8_mm(dev(P[0]), dev(PS[0]), H, H, q, s, T, qm.BF16, h)
    xq, xs = ref.quantize(x.double().numpy())
    want, err = ref.product(ref.row_values(xq, xs), PV[0], ref.f8_terms(H))
    check(f64(h), want, ref.rounded(want, err, "bf16"), "dense")
    out = run_moe(qm, dims, "bf16", h, dev(idx), dev(w), dev_stacks(stacks), h)
    hv = f64(h)
    want, err = moe_reference(hv, idx, w, [c[2] for c in stacks], hv, "bf16")
    check(f64(out), want, ref.rounded(want, err, "bf16"), "experts")
    assert qm.device_status() == qm.OK


def test_two_streams_at_once(qm):
    """Calls on two streams with their own workspaces overlap and agree with
    the calls one by one."""
    import torch
    dims = (64, 384, 256, 6, 2)
    cases = []
    for seed in (51, 52):
        g, x, residual, idx, w, stacks = moe_case(seed, *dims, "bf16")
        cases.append((x.cuda(), dev(idx), dev(w), dev_stacks(stacks), residual.cuda()))
    alone = [run_moe(qm, dims, "bf16", *c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    shape = qm.moe_shape(384, 256, 6, 2, 64, qm.E4M3, qm.E4M3, qm.E4M3)
    n = qm.moe_experts_f8_workspace_size(shape)
    bufs = [(torch.empty(n, dtype=torch.uint8, device="cuda"),
             out_tensor(64, 384, torch.bfloat16)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, c, (ws, out) in zip(streams, cases, bufs):
            run_moe(qm, dims, "bf16", *c, out=out, ws=ws, stream=s)
    torch.cuda.synchronize()
    for a, (_, out) in zip(alone, bufs):
        assert torch.equal(a, out)
    assert qm.device_status() == qm.OK


def test_binding_checks_tensors(qm):
    import torch
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(4, 256, dtype=torch.uint8, device="cuda")
    s = torch.zeros(4, 2, device="cuda")
    y = torch.zeros(4, 100, device="cuda")
    w, wsc = torch.zeros(100, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, device="cuda")
    with pytest.raises(qm.QmoeError, match="dtype"):
        qm.f8_quantize(qm.F32, x, 4, 256, q, s)
    with pytest.raises(qm.QmoeError, match="needed"):
        qm.f8_quantize(qm.BF16, x, 5, 256, q, s)
    with pytest.raises(qm.QmoeError, match="needed"):
        qm.f8_quantize(qm.BF16, x, 4, 256, q, s[:, 1:].contiguous())
    with pytest.raises(qm.QmoeError, match="needed"):
        qm.f8_mm(w, wsc[:1].clone(), 100, 256, q, s, 4, qm.F32, y)
    with pytest.raises(qm.QmoeError, match="current CUDA device"):
        qm.f8_mm(w.cpu(), wsc, 100, 256, q, s, 4, qm.F32, y)
    with pytest.raises(qm.QmoeError, match="dtype"):
        qm.mm_grouped(qm.E4M3, w, wsc, 1, 100, 256, q, s, 4, torch.zeros(2, device="cuda"),
                      qm.F32, y)


# ----------------------------------------------------- beyond 32-bit offsets
def test_f8_mm_output_beyond_2_31_elements(qm):
    """70,000 x 40,000 outputs (2.8e9 elements): sampled rows, the last among
    them, against the 64-bit form."""
    import torch
    m, n, k = 70000, 40000, 32
    g = np.random.default_rng(61)
    xq, xs, wq, ws, xv, wv = f8_operands(g, m, n, k)
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    qm.f8_mm(dev(wq[0]), dev(ws[0]), n, k, dev(xq), dev(xs), m, qm.BF16, y)
    assert qm.device_status() == qm.OK
    rows = [0, 1, 53686, 53687, 53688, 69998, 69999]  # 53687 * 40000 passes 2^31
    want, err = ref.product(xv[rows], wv[0], ref.f8_terms(k))
    check(f64(y[rows]), want, ref.rounded(want, err, "bf16"), "rows")


@pytest.mark.parametrize("kind", ["f8", "bf16"])
def test_mm_grouped_weights_beyond_2_31_elements(qm, kind):
    """A stack of 2.4e9 elements: only the last group's matrix is not zero."""
    import torch
    e, n, k, m = 36, 8192, 8192, 72
    g = np.random.default_rng(62)
    off = np.arange(0, 2 * e + 1, 2).astype(np.int32)
    y = out_tensor(m, n, torch.float32)
    if kind == "f8":
        xq, xs, wq, ws, xv, wv = f8_operands(g, m, 256, k)
        W = torch.zeros(e, n, k, dtype=torch.uint8, device="cuda")
        S = torch.ones(e, n // 128, k // 128, device="cuda")
        W[-1, -256:] = dev(wq[0])
        S[-1, -2:] = dev(ws[0])
        qm.mm_grouped(qm.E4M3, W, S, e, n, k, dev(xq), dev(xs), m, dev(off), qm.F32, y)
        terms, w = ref.f8_terms(k), wv[0]
    else:
        x, w16, xv, wv = wide_operands(g, m, 256, k, 1, "bf16")
        W = torch.zeros(e, n, k, dtype=torch.bfloat16, device="cuda")
        W[-1, -256:] = w16[0].cuda()
        qm.mm_grouped(qm.BF16, W, None, e, n, k, x.cuda(), None, m, dev(off), qm.F32, y)
        terms, w = ref.wide_terms(k), wv[0]
    assert qm.device_status() == qm.OK
    assert (y[:-2] == 0).all() and (y[-2:, :-256] == 0).all()
    want, err = ref.product(xv[-2:], w, terms)
    check(f64(y[-2:, -256:]), want, ref.rounded(want, err, "f32"), "last group")


def test_moe_many_tokens_repeat_the_first(qm):
    """140,000 tokens (the activations' rows pass 2^31 bytes) that repeat 64
    tokens: every repeat has the bits of the first."""
    import torch
    dims = (64, 2048, 128, 8, 8)
    g, x, residual, idx, w, stacks = moe_case(63, *dims, "bf16")
    reps = 2188
    T = 64 * reps
    st = dev_stacks(stacks)
    X, I, W, R = (t.repeat(reps, 1) for t in (x.cuda(), dev(idx), dev(w), residual.cuda()))
    out = run_moe(qm, (T,) + dims[1:], "bf16", X, I, W, st, R)
    assert qm.device_status() == qm.OK
    first = out[:64]
    assert (out.view(reps, 64, -1) == first).all()
    want, err = moe_reference(x.double().numpy()[:8], idx[:8], w[:8], [s[2] for s in stacks],
                              residual.double().numpy()[:8], "bf16")
    check(f64(first[:8]), want, ref.rounded(want, err, "bf16"), "moe")


def test_first_call_may_be_captured():
    """A process whose first call of each function is inside a capture."""
    import subprocess
    import sys
    code = """
import torch, moe_ffn_gb300 as qm
x = torch.randn(4, 256, device="cuda", dtype=torch.bfloat16)
q = torch.empty(4, 256, dtype=torch.uint8, device="cuda"); s = torch.empty(4, 2, device="cuda")
W = torch.full((128, 256), 0x38, dtype=torch.uint8, device="cuda"); S = torch.ones(1, 2, device="cuda")
y = torch.empty(4, 128, device="cuda")
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    qm.f8_quantize(qm.BF16, x, 4, 256, q, s)
    qm.f8_mm(W, S, 128, 256, q, s, 4, qm.F32, y)
g.replay()
torch.cuda.synchronize()
want = (q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 1)).sum(1)
assert torch.allclose(y, want[:, None].expand(4, 128), rtol=1e-4, atol=1e-4)
assert qm.device_status() == qm.OK
print("captured")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("cta", [0, 1])
@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (32, 20000, 256), (600, 1024, 512),
                                   (900, 700, 1600)],
                         ids=["shared_k", "few_rows", "pairs", "pairs_ragged"])
def test_wait_that_runs_out_is_reported(qm, m, n, k, cta):
    """One CTA loads nothing and every device wait gives up after 5 ms: the call
    returns, the status says so, and the next call is right."""
    import torch
    g = np.random.default_rng(71)
    xq, xs, wq, ws, xv, wv = f8_operands(g, m, n, k)
    args = (dev(wq[0]), dev(ws[0]), n, k, dev(xq), dev(xs), m, qm.F32)
    y = out_tensor(m, n, torch.float32)
    torch.cuda.synchronize()
    qm.set_fault_injection(5_000_000, cta)
    try:
        qm.f8_mm(*args, y)
        assert qm.device_status() == qm.ERR_TIMEOUT
        assert "wait" in qm.last_error()
    finally:
        qm.set_fault_injection(0, -1)
    qm.f8_mm(*args, y)
    assert qm.device_status() == qm.OK
    want, err = ref.product(xv, wv[0], ref.f8_terms(k))
    check(f64(y), want, ref.rounded(want, err, "f32"), "after the timeout")


@pytest.mark.parametrize("tokens", [1, 300])
def test_moe_wait_that_runs_out_is_reported(qm, tokens):
    dims = (tokens, 256, 256, 4, 2)
    g, x, residual, idx, w, stacks = moe_case(72, *dims, "bf16")
    args = (x.cuda(), dev(idx), dev(w), dev_stacks(stacks), residual.cuda())
    good = run_moe(qm, dims, "bf16", *args)
    assert qm.device_status() == qm.OK
    qm.set_fault_injection(5_000_000, 0)
    try:
        run_moe(qm, dims, "bf16", *args)
        assert qm.device_status() == qm.ERR_TIMEOUT
    finally:
        qm.set_fault_injection(0, -1)
    assert (run_moe(qm, dims, "bf16", *args) == good).all()
    assert qm.device_status() == qm.OK
