"""GPU tests of the 4-bit products' kernel for few rows where clusters of CTAs share K:
every size of cluster, clusters with several tiles, one, or none at all."""
import numpy as np
import pytest

from tests import steps_ref as ref
from tests.test_gpu_f8 import check, dev, f64, kinds
from tests.test_gpu_w4 import TYPES, weights

pytestmark = pytest.mark.gpu


def product(qm, g, m, n, k, S, kind, times=3):
    import torch
    q, s, z, wv = weights(qm, g, 1, n, k, S, "f16", True)
    code, dt = kinds(qm)[kind]
    x = torch.from_numpy(0.01 * g.standard_normal((m, k)).astype(np.float32)).to(dt).cuda()
    ys = [torch.full((m, n), 55.0, device="cuda") for _ in range(times)]
    for y in ys:
        qm.w4_mm(q, qm.F16, s, z, S, n, k, code, x, m, qm.F32, y)
    assert qm.device_status() == qm.OK
    assert all(torch.equal(ys[0], y) for y in ys[1:])
    want, err = ref.w4_product(f64(x), wv[0], S)
    check(f64(ys[0]), want, ref.rounded(want, err, "f32"), f"{m}x{n}x{k}")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k,S", [(8, 4096, 14336, 128), (16, 4096, 4096, 128),
                                     (4, 130, 8192, 64), (2, 16, 4096, 32), (1, 17, 2560, 128),
                                     (13, 1000, 5120, 32)])
def test_k_shared_by_clusters(qm, kind, m, n, k, S):
    product(qm, np.random.default_rng(m + n + k), m, n, k, S, kind)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("sizes", [[0, 0, 0, 0], [0, 5, 0, 0], [1, 0, 0, 2], [3, 3, 3, 3]])
def test_clusters_without_a_tile(qm, kind, sizes):
    """The launch has clusters for as many tiles as the rows could make; groups without rows
    leave some of them, or all, with nothing to do."""
    import torch
    e, n, k, S, m = len(sizes), 200, 6144, 128, 12
    g = np.random.default_rng(sum(sizes))
    q, s, z, wv = weights(qm, g, e, n, k, S, "bf16", True)
    code, dt = kinds(qm)[kind]
    x = torch.from_numpy(0.01 * g.standard_normal((m, k)).astype(np.float32)).to(dt).cuda()
    y = torch.full((m, n), 55.0, device="cuda")
    off = np.cumsum([0] + sizes).astype(np.int32)
    for _ in range(5):
        qm.w4_mm_grouped(q, qm.BF16, s, z, S, e, n, k, code, x, m, dev(off), qm.F32, y)
    assert qm.device_status() == qm.OK
    xv, got = f64(x), f64(y)
    for i in range(e):
        r = slice(off[i], off[i + 1])
        want, err = ref.w4_product(xv[r], wv[i], S)
        check(got[r], want, ref.rounded(want, err, "f32"), f"group {i}")
    assert (got[off[-1]:] == 55.0).all()
