"""GPU tests of w4_mm and w4_mm_grouped against the 64-bit forms of
tests/steps_ref.py, whose header derives the tolerances."""
import numpy as np
import pytest

from tests import steps_ref as ref
from tests.test_gpu_f8 import check, dev, f64, kinds
from tests.test_gpu_steps import strided

pytestmark = pytest.mark.gpu
TYPES = ["f32", "bf16", "f16"]


def weights(qm, g, e, n, k, S, stype, zeros):
    """Random codes, scales of wide range, zero points with their high bits set."""
    import torch
    q = g.integers(0, 256, (e, n, k // 2), dtype=np.uint8)
    s = torch.from_numpy(np.exp(g.uniform(-4, 0, (e, n, k // S))).astype(np.float32))
    s = s.to(kinds(qm)[stype][1]).cuda()
    z = g.integers(0, 256, (e, n, k // S), dtype=np.uint8) if zeros else None
    return dev(q), s, (None if z is None else dev(z)), ref.w4_values(q, f64(s), z, S)


def run_mm(qm, m, n, k, S, kind="bf16", okind=None, stype="f16", zeros=True, ldx=None, ldy=None,
           offset=0, x=None, sparse=False):
    import torch
    okind = okind or kind
    g = np.random.default_rng(m + 3 * n + 5 * k + S)
    q, s, z, wv = weights(qm, g, 1, n, k, S, stype, zeros)
    if x is None:
        x = g.standard_normal((m, k)) * (0.01 if "f16" in (kind, okind) else 1.0)
    xt, _ = strided(x, kind, qm, ldx, offset)
    y, store = strided(np.full((m, n), 55.0), okind, qm, ldy, offset)
    qm.w4_mm(q, kinds(qm)[stype][0], s, z, S, n, k, kinds(qm)[kind][0], xt, m, kinds(qm)[okind][0],
             y, ldx=ldx, ldy=ldy)
    assert qm.device_status() == qm.OK
    want, err = ref.w4_product(f64(xt[:, :k]), wv[0], S)
    check(f64(y[:, :n]), want, ref.rounded(want, err, okind), f"w4 {m}x{n}x{k}")
    if ldy:
        assert (y[:, n:] == 77.0).all()
    assert (store[:offset] == 77.0).all() and (store[offset + y.numel():] == 77.0).all()


SHAPES = [  # tokens, rows, cols, scale_cols
    (1, 1, 32, 32), (1, 4096, 4096, 128), (2, 100, 64, 64), (3, 130, 160, 32), (7, 33, 1280, 128),
    (8, 257, 192, 64), (9, 640, 1024, 128), (16, 15, 2048, 128), (17, 128, 96, 32),
    (33, 300, 512, 64), (64, 16, 4096, 128), (65, 200, 256, 32), (150, 129, 384, 128),
    (1, 5000, 128, 128), (5, 48, 14336, 128), (2, 20, 14400, 64), (1, 17, 40000, 32),
]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k,S", SHAPES)
def test_w4_mm(qm, kind, m, n, k, S):
    run_mm(qm, m, n, k, S, kind)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("okind", TYPES)
@pytest.mark.parametrize("stype", TYPES)
@pytest.mark.parametrize("zeros", [True, False])
def test_w4_mm_types(qm, kind, okind, stype, zeros):
    run_mm(qm, 11, 70, 256, 64, kind, okind, stype, zeros)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ldx,ldy,offset", [(264, 72, 0), (257, 65, 0), (256, 64, 1), (258, 67, 2),
                                            (256, 64, 4), (272, 80, 8)])
@pytest.mark.parametrize("m", [1, 12])
def test_w4_mm_strides(qm, kind, ldx, ldy, offset, m):
    run_mm(qm, m, 64, 256, 32, kind, ldx=ldx, ldy=ldy, offset=offset)


def test_w4_mm_f32_keeps_all_bits_of_x(qm):
    """f32 values with 24 significant bits, of sizes from 2^-100 to 2^100: the error stays
    within the bound of the sums (one bit lost would be 2^-23 of single terms)."""
    g = np.random.default_rng(5)
    k = 64
    for p in (-100, -20, 0, 20, 100):
        x = np.zeros((3, k), np.float32)
        x[0, 5] = np.float32(2.0 ** p) * np.float32(1 + 2.0 ** -23)
        x[1, 63] = np.float32(2.0 ** p) * np.float32(2 - 2.0 ** -23)
        x[2] = (g.standard_normal(k) * 2.0 ** p).astype(np.float32)
        run_mm(qm, 3, 40, k, 32, "f32", x=x)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m", [1, 5, 40])
def test_w4_mm_nan_and_infinities_stay_in_their_rows(qm, kind, m):
    """A NaN or infinite x makes its own row's outputs so (an infinity NaN where its
    weight is 0) and no other's; a NaN scale its own column's."""
    import torch
    n, k, S = 50, 128, 64
    g = np.random.default_rng(m)
    q, s, z, wv = weights(qm, g, 1, n, k, S, "f32", True)
    s[0, 7, 1] = float("nan")
    wv[0, 7, 64:] = np.nan
    x = (g.standard_normal((m, k)) * 0.01)
    x[0, 3] = np.inf
    if m > 1:
        x[m - 1, 100] = np.nan
    xt, _ = strided(x, kind, qm)
    y = torch.full((m, n), 55.0, device="cuda")
    qm.w4_mm(q, qm.F32, s, z, S, n, k, kinds(qm)[kind][0], xt, m, qm.F32, y)
    got = y.cpu().numpy()
    w3 = wv[0, :, 3]
    other = np.arange(n) != 7
    assert np.isnan(got[:, 7]).all()
    assert np.array_equal(np.isnan(got[0, other]), w3[other] == 0)
    live = other & (w3 != 0)
    assert np.array_equal(got[0, live], np.sign(w3[live]) * np.inf)
    if m > 1:
        assert np.isnan(got[m - 1]).all()
        rest = slice(1, m - 1)
        want, err = ref.w4_product(f64(xt)[rest], wv[0][other], S)
        check(got[rest][:, other], want, ref.rounded(want, err, "f32"), "the other rows")


GROUPS = {  # rows of each group
    "one each": [1] * 9, "ragged": [0, 3, 17, 0, 1, 40, 0], "first empty": [0, 0, 5],
    "large": [70, 1, 130, 0, 64], "none": [0, 0, 0], "one": [20],
}


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("n,k,S,zeros", [(100, 256, 128, True), (33, 96, 32, False),
                                         (768, 2048, 64, True)])
def test_w4_mm_grouped(qm, kind, name, n, k, S, zeros):
    """Groups by offsets, with rows before the first and behind the last: left as they
    were."""
    import torch
    sizes = GROUPS[name]
    e = len(sizes)
    g = np.random.default_rng(n + e)
    q, s, z, wv = weights(qm, g, e, n, k, S, "bf16", zeros)
    head, tail = 3, 4
    off = np.cumsum([head] + sizes).astype(np.int32)
    m = int(off[-1]) + tail
    xt, _ = strided(g.standard_normal((m, k)) * 0.01, kind, qm)
    y, _ = strided(np.full((m, n), 55.0), kind, qm)
    code = kinds(qm)[kind][0]
    qm.w4_mm_grouped(q, qm.BF16, s, z, S, e, n, k, code, xt, m, dev(off), code, y)
    assert qm.device_status() == qm.OK
    assert (y[:head] == 55.0).all() and (y[int(off[-1]):] == 55.0).all()
    xv, got = f64(xt), f64(y)
    for i in range(e):
        r = slice(off[i], off[i + 1])
        want, err = ref.w4_product(xv[r], wv[i], S)
        check(got[r], want, ref.rounded(want, err, kind), f"group {i}")


@pytest.mark.parametrize("e", [1, 33, 300, 1024])
def test_w4_mm_grouped_many_groups(qm, e):
    import torch
    n, k, S, m = 40, 64, 32, 200
    g = np.random.default_rng(e)
    q, s, z, wv = weights(qm, g, e, n, k, S, "f32", True)
    group = np.sort(g.integers(0, e, m))
    off = np.searchsorted(group, np.arange(e + 1)).astype(np.int32)
    xt, _ = strided(g.standard_normal((m, k)), "f32", qm)
    y = torch.zeros(m, n, device="cuda")
    qm.w4_mm_grouped(q, qm.F32, s, z, S, e, n, k, qm.F32, xt, m, dev(off), qm.F32, y)
    assert qm.device_status() == qm.OK
    xv = f64(xt)
    for i in range(m):
        want, err = ref.w4_product(xv[i:i + 1], wv[group[i]], S)
        check(f64(y[i:i + 1]), want, ref.rounded(want, err, "f32"), f"row {i}")


@pytest.mark.parametrize("off", [[0, 5, 3, 8], [-1, 2, 4, 8], [0, 2, 4, 9], [3, 2, 1, 0]])
def test_w4_mm_grouped_bad_offsets_are_reported(qm, off):
    import torch
    n, k = 40, 64
    g = np.random.default_rng(0)
    q, s, z, _ = weights(qm, g, 3, n, k, 32, "f32", True)
    y = torch.full((8, n), 55.0, device="cuda")
    x = torch.ones(8, k, device="cuda")
    qm.w4_mm_grouped(q, qm.F32, s, z, 32, 3, n, k, qm.F32, x, 8, dev(np.array(off, np.int32)),
                     qm.F32, y)
    assert qm.device_status() == qm.ERR_INVALID_ARGUMENT and "w4_mm_grouped" in qm.last_error()
    assert (y == 55.0).all()
    qm.w4_mm_grouped(q, qm.F32, s, z, 32, 3, n, k, qm.F32, x, 8,
                     dev(np.array([0, 2, 4, 8], np.int32)), qm.F32, y)
    assert qm.device_status() == qm.OK and (y != 55.0).all()


MANY = [  # tokens, rows, cols, scale_cols: sizes that the kernel for many rows takes
    (40, 4096, 4096, 128), (64, 14336, 1024, 64), (65, 14000, 992, 32), (130, 5000, 1120, 32),
    (200, 3000, 2240, 64), (333, 4097, 2176, 128), (600, 16385, 128, 128), (700, 8300, 96, 32),
    (1500, 1030, 1024, 64), (5000, 300, 640, 128), (20000, 40, 1152, 128),
]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k,S", MANY)
def test_w4_mm_many_rows(qm, kind, m, n, k, S):
    """Full and ragged tiles of tokens and of weight rows, halves of a tile without rows,
    K that ends inside a block, clusters that share K, scales in whole chunks and not."""
    import torch
    g = np.random.default_rng(m + n + k)
    zeros = k % 64 != 0
    q, s, z, wv = weights(qm, g, 1, n, k, S, "f16", zeros)
    code, dt = kinds(qm)[kind]
    x = torch.from_numpy(0.01 * g.standard_normal((m, k)).astype(np.float32)).to(dt).cuda()
    y = torch.full((m, n), 55.0, device="cuda")
    qm.w4_mm(q, qm.F16, s, z, S, n, k, code, x, m, qm.F32, y)
    assert qm.device_status() == qm.OK
    # (in 64 bits on the GPU: the products of the larger cases take a CPU minutes)
    xd, wd = x.double(), torch.from_numpy(wv[0]).cuda()
    want = xd @ wd.T
    terms = 1.01 * 2 * (16 + S / 16) + k / S + 1 + 32
    tol = terms * ref.U * (xd.abs() @ wd.abs().T) + ref.U * want.abs()
    off = (y.double() - want).abs() - tol
    assert float(off.max()) <= 0, f"{int((off > 0).sum())} of {off.numel()} outside"


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ldx,ldy,offset", [(1032, 1300, 0), (1025, 1281, 1), (1024, 1280, 4),
                                            (1040, 1290, 8)])
def test_w4_mm_many_rows_strides(qm, kind, ldx, ldy, offset):
    run_mm(qm, 500, 1280, 1024, 64, kind, okind="bf16", ldx=ldx, ldy=ldy, offset=offset)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("name,n,k,S", [("uneven", 520, 1024, 128), ("uneven", 768, 672, 32),
                                        ("many groups", 256, 512, 64)])
def test_w4_mm_grouped_many_rows(qm, kind, name, n, k, S):
    """Uneven groups with rows before the first and behind the last, which are left as
    they were, by the kernel for many rows."""
    import torch
    g = np.random.default_rng(n + k)
    if name == "uneven":
        sizes = [0, 150, 1, 64, 0, 65, 129, 7, 0, 300, 63, 2, 200, 0]
    else:
        sizes = list(g.integers(0, 70, 300))
    e, head, tail = len(sizes), 3, 5
    q, s, z, wv = weights(qm, g, e, n, k, S, "bf16", True)
    off = np.cumsum([head] + sizes).astype(np.int32)
    m = int(off[-1]) + tail
    code, dt = kinds(qm)[kind]
    x = torch.from_numpy(0.01 * g.standard_normal((m, k)).astype(np.float32)).to(dt).cuda()
    y = torch.full((m, n), 55.0, dtype=dt, device="cuda")
    qm.w4_mm_grouped(q, qm.BF16, s, z, S, e, n, k, code, x, m, dev(off), code, y)
    assert qm.device_status() == qm.OK
    assert (y[:head] == 55.0).all() and (y[int(off[-1]):] == 55.0).all()
    xv, got = f64(x), f64(y)
    for i in range(e):
        r = slice(off[i], off[i + 1])
        want, err = ref.w4_product(xv[r], wv[i], S)
        check(got[r], want, ref.rounded(want, err, kind), f"group {i}")


def test_many_rows_keep_nan_and_infinities_to_themselves(qm):
    import torch
    n, k, S, m = 2048, 1024, 128, 500
    g = np.random.default_rng(8)
    for kind in TYPES:
        q, s, z, wv = weights(qm, g, 1, n, k, S, "f32", True)
        s[0, 1000, 3] = float("nan")
        x = torch.randn(m, k, device="cuda") * 0.01
        x[77, 3], x[499, 100] = float("inf"), float("nan")
        x = x.to(kinds(qm)[kind][1])
        y = torch.zeros(m, n, device="cuda")
        qm.w4_mm(q, qm.F32, s, z, S, n, k, kinds(qm)[kind][0], x, m, qm.F32, y)
        assert qm.device_status() == qm.OK
        got = y.cpu().numpy()
        assert np.isnan(got[:, 1000]).all() and np.isnan(got[499]).all()
        rest = np.delete(np.delete(got, [77, 499], 0), 1000, 1)
        assert np.isfinite(rest).all()
        w3, other = wv[0][:, 3], np.arange(n) != 1000
        assert np.array_equal(np.isnan(got[77, other]), w3[other] == 0)
        live = other & (w3 != 0)
        assert np.array_equal(got[77, live], np.sign(w3[live]) * np.inf)


@pytest.mark.parametrize("cta", [0, 3])
@pytest.mark.parametrize("m,n,k", [(64, 4096, 4096), (600, 8000, 1024)], ids=["shared_k", "tiles"])
def test_wait_that_runs_out_is_reported(qm, m, n, k, cta):
    """One CTA of the kernel for many rows loads nothing and every device wait gives up
    after 5 ms: the call returns, the status says so, and the next call is right."""
    import torch
    g = np.random.default_rng(71)
    q, s, z, wv = weights(qm, g, 1, n, k, 128, "f16", True)
    x = (0.01 * torch.randn(m, k, device="cuda")).to(torch.bfloat16)
    y = torch.zeros(m, n, device="cuda")
    args = (q, qm.F16, s, z, 128, n, k, qm.BF16, x, m, qm.F32)
    torch.cuda.synchronize()
    qm.set_fault_injection(5_000_000, cta)
    try:
        qm.w4_mm(*args, y)
        assert qm.device_status() == qm.ERR_TIMEOUT
        assert "wait" in qm.last_error()
    finally:
        qm.set_fault_injection(0, -1)
    qm.w4_mm(*args, y)
    assert qm.device_status() == qm.OK
    pick = np.arange(0, n, 37)
    want, err = ref.w4_product(f64(x), wv[0][pick], 128)
    check(f64(y)[:, pick], want, ref.rounded(want, err, "f32"), "after the timeout")


def test_same_inputs_same_bits(qm):
    import torch
    g = np.random.default_rng(1)
    for m, n, k in ((1, 4096, 4096), (5, 1000, 2048), (200, 300, 512), (64, 4096, 4096),
                    (300, 9000, 1024)):
        q, s, z, _ = weights(qm, g, 1, n, k, 128, "f16", True)
        x = torch.randn(m, k, device="cuda").to(torch.bfloat16)
        ys = [torch.empty(m, n, device="cuda") for _ in range(4)]
        for y in ys:
            qm.w4_mm(q, qm.F16, s, z, 128, n, k, qm.BF16, x, m, qm.F32, y)
        assert all(torch.equal(ys[0], y) for y in ys[1:])


def test_a_row_does_not_depend_on_the_others(qm):
    """A token's outputs are the same bits alone, and within the bound in any batch."""
    import torch
    g = np.random.default_rng(2)
    n, k, S = 200, 512, 64
    q, s, z, wv = weights(qm, g, 1, n, k, S, "f16", True)
    x = torch.randn(70, k, device="cuda").to(torch.bfloat16)
    want, err = ref.w4_product(f64(x), wv[0], S)
    for m in (1, 2, 8, 9, 16, 31, 64, 70):
        y = torch.empty(m, n, device="cuda")
        qm.w4_mm(q, qm.F16, s, z, S, n, k, qm.BF16, x[:m], m, qm.F32, y)
        check(f64(y), want[:m], ref.rounded(want[:m], err[:m], "f32"), f"{m} tokens")


def test_weights_beyond_2_31_codes(qm):
    """A matrix of 2^32 codes: offsets of weights and scales that pass 32 bits."""
    import torch
    n, k, S = (1 << 20) + 3, 4096, 128
    q = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.rand(n, k // S, device="cuda").to(torch.float16)
    z = torch.randint(0, 16, (n, k // S), dtype=torch.uint8, device="cuda")
    x = torch.randn(2, k, device="cuda").to(torch.bfloat16)
    y = torch.zeros(2, n, device="cuda")
    qm.w4_mm(q, qm.F16, s, z, S, n, k, qm.BF16, x, 2, qm.F32, y)
    assert qm.device_status() == qm.OK
    pick = [0, 1, 524287, 524288, n - 17, n - 1]
    wv = ref.w4_values(q[pick].cpu().numpy(), f64(s[pick]), z[pick].cpu().numpy(), S)
    want, err = ref.w4_product(f64(x), wv, S)
    check(f64(y[:, pick]), want, ref.rounded(want, err, "f32"), "sampled rows")


def test_stack_beyond_2_31_bytes(qm):
    """The last group of a stack whose codes pass 2^31 bytes."""
    import torch
    e, n, k, S = 130, 4096, 8192, 128
    q = torch.randint(0, 256, (e, n, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.rand(e, n, k // S, device="cuda").to(torch.bfloat16)
    x = (0.01 * torch.randn(3, k, device="cuda")).to(torch.float16)
    off = torch.tensor([0] * (e - 1) + [1, 3], dtype=torch.int32, device="cuda")
    y = torch.zeros(3, n, device="cuda")
    assert q.numel() > 2 ** 31
    qm.w4_mm_grouped(q, qm.BF16, s, None, S, e, n, k, qm.F16, x, 3, off, qm.F32, y)
    assert qm.device_status() == qm.OK
    for i, r in ((e - 2, slice(0, 1)), (e - 1, slice(1, 3))):
        pick = [0, 100, n - 1]
        wv = ref.w4_values(q[i][pick].cpu().numpy(), f64(s[i][pick]), None, S)
        want, err = ref.w4_product(f64(x[r]), wv, S)
        check(f64(y[r][:, pick]), want, ref.rounded(want, err, "f32"), f"group {i}")


@pytest.mark.parametrize("t", [1, 30])
def test_layer_of_4_bit_experts(qm, t):
    """Routes, sort, 4-bit gate, up and down products and the weighted sum in a run,
    f32 activations throughout: each step within its own bound, together below
    2^-14 of the outputs' size (five steps of at most 2^-17 for these lengths)."""
    import torch
    g = np.random.default_rng(t)
    e, k, h, f, S = 16, 4, 256, 128, 64
    x = torch.randn(t, h, device="cuda")
    logits = torch.randn(t, e, device="cuda")
    stacks = [weights(qm, g, e, n, c, S, "f16", True) for n, c in ((f, h), (f, h), (h, f))]
    P = t * k
    idx = torch.empty(t, k, dtype=torch.int32, device="cuda")
    pos, w = torch.empty_like(idx), torch.empty(t, k, device="cuda")
    rows, y, out = (torch.empty(n, h, device="cuda") for n in (P, P, t))
    a = [torch.empty(P, f, device="cuda") for _ in range(2)]
    off = torch.empty(e + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(qm.moe_permute_workspace_size(t, e, k), dtype=torch.uint8, device="cuda")
    qm.moe_route(qm.F32, logits, t, e, k, idx, w)
    qm.moe_permute(qm.F32, x, t, h, idx, e, k, rows, off, pos, ws)
    for i in range(2):
        q, s, z, _ = stacks[i]
        qm.w4_mm_grouped(q, qm.F16, s, z, S, e, f, h, qm.F32, rows, P, off, qm.F32, a[i])
    q, s, z, _ = stacks[2]
    act = torch.relu(a[0]) * a[1]
    qm.w4_mm_grouped(q, qm.F16, s, z, S, e, h, f, qm.F32, act, P, off, qm.F32, y)
    qm.moe_combine(qm.F32, y, P, h, pos, w, t, k, qm.F32, x, out)
    assert qm.device_status() == qm.OK
    i, wt, _ = ref.route(f64(logits), k, True)
    xv, want, size = f64(x), f64(x), 0.0
    for tok in range(t):
        for slot in range(k):
            gate, up, down = (st[3][i[tok, slot]] for st in stacks)
            term = wt[tok, slot] * (down @ (np.maximum(gate @ xv[tok], 0) * (up @ xv[tok])))
            want[tok] += term
    off_by = np.linalg.norm(f64(out) - want) / np.linalg.norm(want)
    assert off_by <= 2.0 ** -14, off_by


# ------------------------------------------------- streams, graphs, addresses
def test_first_calls_may_be_captured():
    """A process whose first call of each function is inside a capture."""
    import os
    import subprocess
    import sys
    code = """
import torch, moe_ffn_gb300 as qm
t, e, k, h = 3, 8, 2, 128
def new(*s, dt=torch.float32): return torch.zeros(*s, dtype=dt, device="cuda")
x, logits = torch.randn(t, h, device="cuda"), torch.randn(t, e, device="cuda")
idx, w, pos = new(t, k, dt=torch.int32), new(t, k), new(t, k, dt=torch.int32)
rows, off, out = new(t * k, h), new(e + 1, dt=torch.int32), new(t, h)
gw, gy, gl = new(t, k), new(t * k, h), new(t, e)
ws = torch.empty(qm.moe_permute_workspace_size(t, e, k), dtype=torch.uint8, device="cuda")
# code 9 and scale 1 everywhere: every output is the sum of its row of x
W, s = torch.full((64, h // 2), 0x99, dtype=torch.uint8, device="cuda"), torch.ones(64, 1, device="cuda")
big, bs = torch.full((4096, 512), 0x99, dtype=torch.uint8, device="cuda"), torch.ones(4096, 8, device="cuda")
xb, yb = torch.ones(64, 1024, device="cuda").bfloat16(), new(64, 4096)
y = new(t, 64)
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    qm.moe_route(qm.F32, logits, t, e, k, idx, w)
    qm.moe_permute(qm.F32, x, t, h, idx, e, k, rows, off, pos, ws)
    qm.moe_combine(qm.F32, rows, t * k, h, pos, w, t, k, qm.F32, None, out)
    qm.moe_combine_backward(qm.F32, rows, t * k, h, pos, w, t, k, qm.F32, x, gy, gw)
    qm.moe_route_backward(qm.F32, logits, t, e, k, idx, w, gw, gl)
    qm.w4_mm(W, qm.F32, s, None, 128, 64, h, qm.F32, x, t, qm.F32, y)
    qm.w4_mm(big, qm.F32, bs, None, 128, 4096, 1024, qm.BF16, xb, 64, qm.F32, yb)
g.replay()
torch.cuda.synchronize()
assert qm.device_status() == qm.OK
assert torch.allclose(out, x, atol=1e-5)          # (weights add up to 1)
assert torch.allclose(y, x.sum(1, keepdim=True).expand(t, 64), atol=1e-4)
assert (yb == 1024).all()
assert torch.allclose(gl.sum(1), new(t), atol=1e-4)
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("m", [3, 400])
def test_streams_graphs_and_addresses(qm, m):
    """The same bits on another stream (current, or named), by addresses, and replayed from a
    graph beside a plain call on a second stream."""
    import torch
    g = np.random.default_rng(m)
    n, k, S = 1500, 1024, 64
    q, s, z, _ = weights(qm, g, 1, n, k, S, "f16", True)
    x = torch.randn(m, k, device="cuda").to(torch.bfloat16)

    def call(y, stream=None, addresses=False):
        a = [t.data_ptr() for t in (q, s, z, x, y)] if addresses else [q, s, z, x, y]
        qm.w4_mm(a[0], qm.F16, a[1], a[2], S, n, k, qm.BF16, a[3], m, qm.F32, a[4], stream=stream)
    want = torch.zeros(m, n, device="cuda")
    call(want)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    ys = [torch.zeros(m, n, device="cuda") for _ in range(5)]
    torch.cuda.synchronize()
    with torch.cuda.stream(one):
        call(ys[0])
    call(ys[1], stream=one)
    call(ys[2], stream=two.cuda_stream, addresses=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=one):
        call(ys[3])
    torch.cuda.synchronize()
    with torch.cuda.stream(one):
        graph.replay()
    with torch.cuda.stream(two):
        call(ys[4])
    torch.cuda.synchronize()
    assert all(torch.equal(want, y) for y in ys)
    assert qm.device_status() == qm.OK


@pytest.mark.parametrize("m", [1, 300])
def test_reads_what_the_stream_has_just_written(qm, m):
    """Weights, scales and rows written by the launches right before the call."""
    import torch
    n, k, S = 2000, 2048, 128
    g = np.random.default_rng(4)
    q, s, z, wv = weights(qm, g, 1, n, k, S, "f32", True)
    x = (0.01 * torch.randn(m, k, device="cuda")).to(torch.float16)
    live = [torch.zeros_like(t) for t in (q, s, z, x)]
    y = torch.zeros(m, n, device="cuda")
    want, err = ref.w4_product(f64(x), wv[0], S)
    for _ in range(20):
        for a in live:
            a.zero_()
        qm.w4_mm(live[0], qm.F32, live[1], live[2], S, n, k, qm.F16, live[3], m, qm.F32, y)
        for a, b in zip(live, (q, s, z, x)):
            a.copy_(b)
        qm.w4_mm(live[0], qm.F32, live[1], live[2], S, n, k, qm.F16, live[3], m, qm.F32, y)
    check(f64(y), want, ref.rounded(want, err, "f32"), "after copies")
