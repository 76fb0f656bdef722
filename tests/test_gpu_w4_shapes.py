"""GPU tests of the 4-bit products' kernel for many rows at the ends of its range: the
shortest K (a part of one k-block, token columns past K not there at all), and matrices
of few rows with very many rows of x."""
import numpy as np
import pytest

from tests import steps_ref as ref
from tests.test_gpu_f8 import kinds
from tests.test_gpu_w4 import TYPES, weights
from tests.test_w4_rule import many  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

SHAPES = [  # tokens, rows, cols, scale_cols
    (150, 16384, 32, 32), (130, 16384, 64, 64), (130, 16384, 64, 32), (3000, 1025, 32, 32),
    (120000, 3, 1024, 128), (200000, 1, 2048, 64), (4000, 257, 160, 32),
]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k,S", SHAPES)
def test_ends_of_the_many_rows_kernel(qm, many, kind, m, n, k, S):  # noqa: F811
    import torch
    assert many(m, 1, n, k, kind)
    g = np.random.default_rng(m + n + k)
    q, s, z, wv = weights(qm, g, 1, n, k, S, "f16", True)
    code, dt = kinds(qm)[kind]
    x = (0.01 * torch.randn(m, k, device="cuda")).to(dt)
    y = torch.full((m, n), 55.0, device="cuda")
    qm.w4_mm(q, qm.F16, s, z, S, n, k, code, x, m, qm.F32, y)
    assert qm.device_status() == qm.OK
    wd = torch.from_numpy(wv[0]).cuda()
    terms = 1.01 * 2 * (16 + S / 16) + k / S + 1 + 32
    for a in range(0, m, 20000):
        xd = x[a:a + 20000].double()
        want = xd @ wd.T
        tol = terms * ref.U * (xd.abs() @ wd.abs().T) + ref.U * want.abs()
        assert bool(((y[a:a + 20000].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("kind", TYPES)
def test_groups_of_short_rows(qm, many, kind):  # noqa: F811
    """K of 32 columns, uneven groups, rows before the first and behind the last."""
    import torch
    sizes = [0, 300, 1, 0, 64, 65, 700, 0]
    e, n, k, S, head, tail = len(sizes), 2100, 32, 32, 3, 5
    g = np.random.default_rng(3)
    q, s, z, wv = weights(qm, g, e, n, k, S, "bf16", False)
    off = np.cumsum([head] + sizes).astype(np.int32)
    m = int(off[-1]) + tail
    assert many(m, e, n, k, kind)
    code, dt = kinds(qm)[kind]
    x = (0.01 * torch.randn(m, k, device="cuda")).to(dt)
    y = torch.full((m, n), 55.0, device="cuda")
    qm.w4_mm_grouped(q, qm.BF16, s, z, S, e, n, k, code, x, m, torch.from_numpy(off).cuda(),
                     qm.F32, y)
    assert qm.device_status() == qm.OK
    assert (y[:head] == 55.0).all() and (y[int(off[-1]):] == 55.0).all()
    for i in range(e):
        xd, wd = x[off[i]:off[i + 1]].double(), torch.from_numpy(wv[i]).cuda()
        want = xd @ wd.T
        terms = 1.01 * 2 * (16 + S / 16) + k / S + 1 + 32
        tol = terms * ref.U * (xd.abs() @ wd.abs().T) + ref.U * want.abs()
        assert bool(((y[off[i]:off[i + 1]].double() - want).abs() <= tol).all()), i
