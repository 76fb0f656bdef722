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
