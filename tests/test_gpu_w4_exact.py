"""GPU tests of the 4-bit products where no sum rounds: f32 rows keep every bit."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k,S", [(3, 40, 64, 32), (9, 200, 1280, 128), (16, 4096, 4096, 64),
                                     (40, 4096, 4096, 128), (64, 14336, 1024, 64),
                                     (130, 5000, 1120, 32)])
def test_f32_rows_keep_every_bit(qm, m, n, k, S):
    """Rows with one value that is not 0, of 24 significant bits and sizes from 2^-80 to
    2^100, weights of 1, 2, 4 and 8 times +-1: the value's three parts of eight bits times a
    power of two are exact, and so is their sum in any order (16 bits, then 24, all an
    f32's), so y equals the multiple of x bit for bit.  The first three shapes run the kernel
    for few rows, the others the one for many."""
    import torch
    g = np.random.default_rng(m + n + k)
    x = np.zeros((m, k), np.float32)
    at = g.integers(0, k, m)
    at[0], at[-1] = 0, k - 1
    frac = g.integers(1 << 23, 1 << 24, m)
    frac[0], frac[1], frac[2] = (1 << 24) - 1, (1 << 23) + 1, (1 << 23) + (1 << 15) + 1
    value = np.ldexp(frac.astype(np.float64) * g.choice([-1, 1], m), g.integers(-80, 101, m) - 23)
    x[np.arange(m), at] = value.astype(np.float32)
    assert (x[np.arange(m), at] == value).all()
    zero = np.full((n, k // S), 8, np.uint8)
    code = (8 + g.choice([1, 2, 4, -1, -2, -4, -8], (n, k))).astype(np.uint8)
    low = g.random((n, k // S)) < 0.5        # half of the scales with zero point 0: 1, 2, 4, 8
    zero[low] = 0
    code = np.where(np.repeat(low, S, 1), g.choice([1, 2, 4, 8], (n, k)), code).astype(np.uint8)
    q = code[:, 0::2] | (code[:, 1::2] << 4)
    y = torch.full((m, n), 55.0, device="cuda")
    qm.w4_mm(torch.from_numpy(q).cuda(), qm.F32, torch.ones(n, k // S, device="cuda"),
             torch.from_numpy(zero).cuda(), S, n, k, qm.F32, torch.from_numpy(x).cuda(), m,
             qm.F32, y)
    assert qm.device_status() == qm.OK
    factor = code[:, at].T.astype(np.float64) - zero[:, at // S].T
    assert np.array_equal(y.cpu().numpy(), (factor * value[:, None]).astype(np.float32))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(3, 40, 256), (16, 4096, 4096), (40, 4096, 4096),
                                   (130, 5000, 1152)])
def test_scales_do_what_the_formula_says(qm, m, n, k, kind):
    """Small whole numbers, so that no sum rounds: powers of two down to 2^-100 scale exactly,
    and infinite ones make their columns NaN, and no other (the formula's weights are then
    infinities of both signs, and NaN where a code is at its zero point)."""
    import torch
    from tests.test_gpu_f8 import kinds
    g = np.random.default_rng(m + k)
    S = 64
    q = g.integers(0, 256, (n, k // 2), dtype=np.uint8)
    code = np.stack((q & 15, q >> 4), -1).reshape(n, k).astype(np.float64) - 8
    x = g.integers(-2, 3, (m, k)).astype(np.float64)
    x[1, :S] = 0
    scale = np.full((n, k // S), 2.0 ** -100)
    scale[7, 0], scale[20, 1], scale[30, :2] = np.inf, -np.inf, np.inf
    s = torch.from_numpy(scale.astype(np.float32)).cuda()
    got_dt, dt = kinds(qm)[kind]
    y = torch.full((m, n), 55.0, device="cuda")
    qm.w4_mm(torch.from_numpy(q).cuda(), qm.F32, s, None, S, n, k, got_dt,
             torch.from_numpy(x.astype(np.float32)).to(dt).cuda(), m, qm.F32, y)
    assert qm.device_status() == qm.OK
    with np.errstate(invalid="ignore"):
        w = np.repeat(scale, S, 1) * code
        want = x @ np.delete(w, [7, 20, 30], 0).T
        for row in (7, 20, 30):
            assert np.isnan(x @ w[row]).all()
            want = np.insert(want, row, np.nan, 1)
    got = y.cpu().numpy().astype(np.float64)
    assert np.array_equal(got, want, equal_nan=True)
