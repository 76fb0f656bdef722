"""GPU tests of every kernel form of the e4m3 and grouped products.  Each test
asks the library's own rule (tests/gmm_plan.py) which kernel its shape takes, so
that a changed threshold cannot leave a form without a test.  References and
tolerances: tests/f8_ref.py."""
import numpy as np
import pytest

from tests import f8_ref as ref
from tests import gmm_plan as plan
from tests.test_gpu_f8 import (check, dev, dev_stacks, f64, f8_operands, kinds, moe_case,
                               moe_reference, out_tensor, run_moe, wide_operands)

pytestmark = pytest.mark.gpu


def takes(want, kind, m, n, groups=None, swiglu=False):
    got = plan.kernel(kind, m, n, groups, swiglu, plan.device_sms())
    assert got == want, f"{kind} {m}x{n} in {groups} groups takes tiles of {got}, not {want}"


def operands(g, kind, m, n, k, e, out):
    """(arguments up to x's rows, x values, weight values, error terms)"""
    if kind == "f8":
        xq, xs, wq, ws, xv, wv = f8_operands(g, m, n, k, e)
        if out == "f16":  # keep y inside f16
            xs, xv = xs / 256, xv / 256
        return (dev(wq), dev(ws), dev(xq), dev(xs)), xv, wv, ref.f8_terms(k)
    x, w, xv, wv = wide_operands(g, m, n, k, e, kind)
    return (w.cuda(), None, x.cuda(), None), xv, wv, ref.wide_terms(k)


def type_of(qm, kind):
    return qm.E4M3 if kind == "f8" else kinds(qm)[kind][0]


# ------------------------------------------------- one group of every form
ONE_GROUP = [  # kernel, type, rows of x, rows of W, cols, more tiles than pairs
    (plan.NARROW, "f8", 260, 4096, 1040, False), (plan.NARROW, "f8", 700, 2050, 400, False),
    (plan.NARROW, "f8", 1000, 4096, 272, True), (plan.WIDE_F8, "f8", 640, 4096, 1040, False),
    (plan.WIDE_F8, "f8", 641, 4100, 528, False), (plan.WIDE_F8, "f8", 1500, 6100, 272, True),
    (plan.NARROW, "bf16", 260, 4096, 1536, False), (plan.NARROW, "f16", 300, 2050, 200, False),
    (plan.WIDE_16, "bf16", 640, 4096, 1536, False), (plan.WIDE_16, "f16", 700, 4100, 264, False),
    (plan.WIDE_16, "bf16", 1500, 6100, 136, True),
]


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gap", ["none", "odd", "padded"])
@pytest.mark.parametrize("want,kind,m,n,k,loops", ONE_GROUP,
                         ids=["{}x{}x{}_{}_{}".format(*c[2:5], c[1], c[0]) for c in ONE_GROUP])
def test_one_group(qm, want, kind, m, n, k, loops, gap, out):
    """Rows of y consecutive, an odd number of elements apart (no 16-byte rows), or
    padded to whole 16 bytes; what lies between rows stays."""
    takes(want, kind, m, n, 1)
    pairs = plan.device_sms() // 2
    assert (plan.pair_tiles(want, [m], n) > pairs) == loops
    code, dt = kinds(qm)[out]
    ldy = {"none": n, "odd": n + 7 - n % 2, "padded": (n + 15) // 8 * 8}[gap]
    g = np.random.default_rng(m + n + k)
    (w, ws, x, xs), xv, wv, terms = operands(g, kind, m, n, k, 1, out)
    y = out_tensor(m, ldy, dt)
    qm.mm_grouped(type_of(qm, kind), w, ws, 1, n, k, x, xs, m, dev(np.int32([0, m])), code, y,
                  ldy=ldy)
    assert qm.device_status() == qm.OK
    want_y, err = ref.product(xv, wv[0], terms)
    check(f64(y[:, :n]), want_y, ref.rounded(want_y, err, out), f"{kind} -> {out}")
    assert (y[:, n:] == 77.0).all()


# ---------------------------------------------------- groups of every form
GROUPED = [  # sizes, rows of W, kernels by type
    ([300, 0, 90, 1, 129], 2040, dict(f8=plan.NARROW, bf16=plan.NARROW, f16=plan.NARROW)),
    ([700, 0, 130, 513, 1, 260], 2100, dict(f8=plan.WIDE_F8, bf16=plan.WIDE_16, f16=plan.WIDE_16)),
    ([(i * 37) % 95 + (i % 7 == 0) * 100 for i in range(70)], 520,
     dict(f8=plan.NARROW, bf16=plan.WIDE_16, f16=plan.WIDE_16)),
]


@pytest.mark.parametrize("kind,out", [("f8", "f32"), ("f8", "bf16"), ("f8", "f16"),
                                      ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_groups(qm, case, kind, out):
    """Ragged groups over the pair kernels: rows before the first group and behind
    the last stay as they were."""
    sizes, n, want = GROUPED[case]
    lead, tail, e, k = 3, 5, len(sizes), 656
    m = lead + sum(sizes) + tail
    takes(want[kind], kind, m, n, e)
    g = np.random.default_rng(m)
    code, dt = kinds(qm)[out]
    (w, ws, x, xs), xv, wv, terms = operands(g, kind, m, n, k, e, out)
    off = np.cumsum([lead] + sizes).astype(np.int32)
    y = out_tensor(m, n, dt)
    qm.mm_grouped(type_of(qm, kind), w, ws, e, n, k, x, xs, m, dev(off), code, y)
    assert qm.device_status() == qm.OK
    got = f64(y)
    assert (got[:lead] == 77.0).all() and (got[off[-1]:] == 77.0).all()
    for i in range(e):
        r = slice(off[i], off[i + 1])
        if sizes[i]:
            want_y, err = ref.product(xv[r], wv[i], terms)
            check(got[r], want_y, ref.rounded(want_y, err, out), f"group {i}")


@pytest.mark.parametrize("kind,want", [("f8", plan.WIDE_F8), ("bf16", plan.WIDE_16)])
def test_groups_loop_over_many_tiles(qm, kind, want):
    """More tiles than pairs, several token tiles a group, K over many blocks."""
    sizes, n, k = [700, 0, 130, 513, 1], 4100, 1536
    e, m = len(sizes), sum([700, 0, 130, 513, 1])
    takes(want, kind, m, n, e)
    assert plan.pair_tiles(want, sizes, n) > plan.device_sms() // 2
    g = np.random.default_rng(91)
    (w, ws, x, xs), xv, wv, terms = operands(g, kind, m, n, k, e, "bf16")
    off = np.cumsum([0] + sizes).astype(np.int32)
    y = out_tensor(m, n, kinds(qm)["bf16"][1])
    qm.mm_grouped(type_of(qm, kind), w, ws, e, n, k, x, xs, m, dev(off), qm.BF16, y)
    assert qm.device_status() == qm.OK
    for i in range(e):
        r = slice(off[i], off[i + 1])
        want_y, err = ref.product(xv[r], wv[i], terms)
        check(f64(y[r]), want_y, ref.rounded(want_y, err, "bf16"), f"group {i}")


@pytest.mark.parametrize("kind,m,n,want", [
    ("f8", 300, 2060, plan.NARROW), ("f8", 640, 4100, plan.WIDE_F8),
    ("bf16", 300, 2060, plan.NARROW), ("bf16", 640, 4100, plan.WIDE_16)])
def test_strided_rows_and_nan(qm, kind, m, n, want):
    """Rows of x and y with gaps, the gaps of x full of NaN; a NaN in one row of x
    and one of W stays in its row and its column."""
    import torch
    takes(want, kind, m, n, 1)
    k, gap = 400, 48
    g = np.random.default_rng(m)
    (w, ws, x, xs), xv, wv, terms = operands(g, kind, m, n, k, 1, "f32")
    nan = 0x7F if kind == "f8" else float("nan")
    wide = torch.full((m, k + gap), nan, dtype=x.dtype, device="cuda")
    wide[:, :k] = x
    wide[m - 2, 77] = nan
    w[0, 150, 300] = nan
    xv[m - 2], wv[0, 150] = 0, 0
    y = out_tensor(m, n + 8, torch.float32)
    qm.mm_grouped(type_of(qm, kind), w, ws, 1, n, k, wide, xs, m, dev(np.int32([0, m])), qm.F32, y,
                  ldx=k + gap, ldy=n + 8)
    assert qm.device_status() == qm.OK
    want_y, err = ref.product(xv, wv[0], terms)
    tol = ref.rounded(want_y, err, "f32")
    want_y[m - 2, :] = np.nan
    want_y[:, 150] = np.nan
    check(f64(y[:, :n]), want_y, tol, "strided, NaN")
    assert (y[:, n:] == 77.0).all()


# --------------------------------------------- the layer over CTA pairs
LAYERS = [  # T, H, F, E, k, kernel of the down product
    (1400, 256, 640, 4, 2, plan.NARROW),   # an odd number of 128-row blocks
    (2000, 256, 512, 4, 2, plan.NARROW),   # an even one
    (1900, 2048, 384, 4, 2, plan.WIDE_F8),
    (1300, 128, 1152, 3, 3, plan.FEW),
]


def layer(T, H, F, E, k, kind):
    """moe_case with uneven routes: expert 0 few tokens, padding slots among them."""
    g, x, residual, idx, w, stacks = moe_case(T + F, T, H, F, E, k, kind)
    idx[7:T:3][idx[7:T:3] == 0] = E - 1
    idx[5, 0] = -1
    idx[T - 1, k - 1] = E
    return x, residual, idx, w, stacks


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "T{}H{}F{}E{}k{}".format(*c))
def test_moe_over_pairs(qm, case, kind):
    """Gate and up over CTA pairs, both halves of a pair with rows of their own and
    more tiles than pairs.  Compared: the first, the last and the tokens at the
    tiles' borders of every expert, and random ones."""
    dims, down = case[:5], case[5]
    T, H, F, E, k = dims
    takes(plan.SWIGLU_PAIRS, "f8", T * k, F, E, swiglu=True)
    takes(down, "f8", T * k, H, E)
    x, residual, idx, w, stacks = layer(*dims, kind)
    sizes = [int((idx == e).sum()) for e in range(E)]
    assert plan.pair_tiles(plan.SWIGLU_PAIRS, sizes, F) > plan.device_sms() // 2
    out = run_moe(qm, dims, kind, x.cuda(), dev(idx), dev(w), dev_stacks(stacks), residual.cuda())
    assert qm.device_status() == qm.OK
    rng = np.random.default_rng(1)
    pick = {0, 5, T - 1} | set(rng.integers(0, T, 12).tolist())
    for e in range(E):
        tokens = np.nonzero(idx.reshape(-1) == e)[0] // k
        for i in (0, 31, 32, 95, 96, len(tokens) // 2, len(tokens) - 1):
            if i < len(tokens):
                pick.add(int(tokens[i]))
    pick = sorted(pick)
    want, err = moe_reference(x.double().numpy()[pick], idx[pick], w[pick],
                              [s[2] for s in stacks], residual.double().numpy()[pick], kind)
    check(f64(out[pick]), want, ref.rounded(want, err, kind), "moe")


def test_moe_over_pairs_repeats_in_streams_and_graphs(qm):
    """The same bits from repeated calls, from two streams at once and from a
    captured graph, with launches of the other forms between them."""
    import torch
    dims = (1400, 256, 640, 4, 2)
    takes(plan.SWIGLU_PAIRS, "f8", 2800, 640, 4, swiglu=True)
    x, residual, idx, w, stacks = layer(*dims, "bf16")
    args = (x.cuda(), dev(idx), dev(w), dev_stacks(stacks), residual.cuda())
    first = run_moe(qm, dims, "bf16", *args).clone()
    g = np.random.default_rng(92)
    (W, WS, X, XS), _, _, _ = operands(g, "f8", 640, 4096, 272, 1, "f32")
    y = out_tensor(640, 4096, torch.float32)

    def product(m):
        qm.f8_mm(W, WS, 4096, 272, X, XS, m, qm.F32, y)
    product(640)
    whole = y.clone()
    shape = qm.moe_shape(*[dims[i] for i in (1, 2, 3, 4, 0)], qm.E4M3, qm.E4M3, qm.E4M3)
    n = qm.moe_experts_f8_workspace_size(shape)
    bufs = [(torch.cuda.Stream(), torch.empty(n, dtype=torch.uint8, device="cuda"),
             out_tensor(1400, 256, torch.bfloat16)) for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(12):
        for s, ws, out in bufs:
            run_moe(qm, dims, "bf16", *args, out=out, ws=ws, stream=s)
        product([640, 3, 260][i % 3])
    torch.cuda.synchronize()
    for _, _, out in bufs:
        assert torch.equal(out, first)
    product(640)
    assert torch.equal(y, whole)
    s, ws, out = bufs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            run_moe(qm, dims, "bf16", *args, out=out, ws=ws)
            run_moe(qm, dims, "bf16", *args, out=out, ws=ws)
    out.fill_(0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    assert qm.device_status() == qm.OK


# ------------------------------------------------- waits that run out
@pytest.mark.parametrize("cta", [0, 1, 7])
@pytest.mark.parametrize("kind,m,n,want", [
    ("f8", 260, 4096, plan.NARROW), ("f8", 640, 4096, plan.WIDE_F8),
    ("bf16", 260, 4096, plan.NARROW), ("bf16", 640, 4096, plan.WIDE_16),
    ("f16", 40, 2048, plan.FEW)])
def test_wait_that_runs_out_in_every_form(qm, kind, m, n, want, cta):
    """One CTA loads nothing and every device wait gives up after 5 ms: the call
    returns, the status says so, and the next call is right."""
    import torch
    takes(want, kind, m, n, 1)
    k = 1040
    g = np.random.default_rng(m)
    (w, ws, x, xs), xv, wv, terms = operands(g, kind, m, n, k, 1, "f32")
    args = (type_of(qm, kind), w, ws, 1, n, k, x, xs, m, dev(np.int32([0, m])), qm.F32)
    y = out_tensor(m, n, torch.float32)
    torch.cuda.synchronize()
    qm.set_fault_injection(5_000_000, cta)
    try:
        qm.mm_grouped(*args, y)
        assert qm.device_status() == qm.ERR_TIMEOUT
        assert "wait" in qm.last_error()
    finally:
        qm.set_fault_injection(0, -1)
    qm.mm_grouped(*args, y)
    assert qm.device_status() == qm.OK
    want_y, err = ref.product(xv, wv[0], terms)
    check(f64(y), want_y, ref.rounded(want_y, err, "f32"), "after the timeout")


@pytest.mark.parametrize("cta", [0, 1, 7])
@pytest.mark.parametrize("F", [640, 512])
def test_moe_wait_that_runs_out_over_pairs(qm, F, cta):
    dims = (1400, 256, F, 4, 2)
    takes(plan.SWIGLU_PAIRS, "f8", 2800, F, 4, swiglu=True)
    x, residual, idx, w, stacks = layer(*dims, "bf16")
    args = (x.cuda(), dev(idx), dev(w), dev_stacks(stacks), residual.cuda())
    good = run_moe(qm, dims, "bf16", *args)
    assert qm.device_status() == qm.OK
    qm.set_fault_injection(5_000_000, cta)
    try:
        run_moe(qm, dims, "bf16", *args)
        assert qm.device_status() == qm.ERR_TIMEOUT
    finally:
        qm.set_fault_injection(0, -1)
    assert (run_moe(qm, dims, "bf16", *args) == good).all()
    assert qm.device_status() == qm.OK
