"""Refusals of the Python binding of the e4m3 and grouped products that come
before the library is called."""
import pytest

import moe_ffn_gb300 as qm
from tests.test_f8_abi import INV, OnDevice, lib, shape  # noqa: F401  (lib is a fixture)


@pytest.mark.parametrize("dtype,size,ok", [
    ("uint8", 4096, True), ("float32", 1024, True), ("uint8", 4095, False),
    ("float32", 1023, False), ("uint8", 0, False)])
def test_workspace_holds_the_bytes_it_is_said_to_hold(lib, dtype, size, ok):  # noqa: F811
    """ws_bytes is what the library goes by: a tensor that holds fewer is
    refused.  (A call with no tokens, which touches nothing.)"""
    torch = pytest.importorskip("torch")
    s = shape(n_tokens=0)
    ws = OnDevice(torch.empty(size, dtype=getattr(torch, dtype)))

    def call():
        qm.moe_experts_f8(*[None] * 6, s, qm.BF16, None, None, None, None, None, ws,
                          ws_bytes=4096, stream=0)
    if ok:
        call()
        return
    with pytest.raises(qm.QmoeError) as ei:
        call()
    assert ei.value.status == INV and "moe_experts_f8: ws holds" in str(ei.value)
