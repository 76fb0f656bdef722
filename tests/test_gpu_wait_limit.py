"""GPU test of the limit of bounded device waits where it is counted in tries of a barrier."""
import time

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(64, 4096, 4096), (600, 8000, 1024)], ids=["shared_k", "tiles"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_a_wait_gives_up_after_its_limit(qm, m, n, k, kind):
    """One CTA of the 4-bit products' kernel for many rows loads nothing.  Its warps wait side
    by side, so the call ends once one limit has passed; how long a try takes may depend on
    the clock, which is why the interface promises it to a factor of two."""
    import torch
    from tests.test_gpu_f8 import kinds
    code, dt = kinds(qm)[kind]
    q = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.ones(n, k // 128, device="cuda")
    x = torch.randn(m, k, device="cuda").to(dt)
    y = torch.zeros(m, n, device="cuda")
    args = (q, qm.F32, s, None, 128, n, k, code, x, m, qm.F32, y)
    qm.w4_mm(*args)
    torch.cuda.synchronize()
    qm.set_fault_injection(50_000_000, 3)
    try:
        t = time.perf_counter()
        qm.w4_mm(*args)
        status = qm.device_status()
        t = time.perf_counter() - t
    finally:
        qm.set_fault_injection(0, -1)
    assert status == qm.ERR_TIMEOUT
    assert 0.025 <= t <= 0.1, t
    qm.w4_mm(*args)
    assert qm.device_status() == qm.OK
