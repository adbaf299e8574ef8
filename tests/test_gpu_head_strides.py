"""The output layer's losses with a single row in hidden, in the weight or in
a gradient: its row stride is never taken, so any is right."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from tests import head_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

FAR = 1 << 45     # in bytes more than a tensor map holds


@pytest.fixture(scope="module")
def g():
    import dense_gemm_tensor_tcgen05_gb300 as g
    from dense_gemm_tensor_tcgen05_gb300 import build
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    build.build()
    return g


@pytest.mark.parametrize("odd", [0, 1], ids=["even", "odd"])
@pytest.mark.parametrize("grad", [0, 1], ids=["16", "f32"])
@pytest.mark.parametrize("N,V,D", [(1, 300, 64), (1, 300, 33), (40, 1, 64), (300, 1, 65), (1, 1, 9)])
def test_stride_of_a_single_row(g, N, V, D, grad, odd):
    H, W, t, gl = ref.inputs(N, V, D, torch.bfloat16, N + V + D)
    a = g.HeadArgs(dtype=1, grad_dtype=grad, tokens=N, vocab=V, dim=D, hidden=H.data_ptr(),
                   ldh=FAR + odd if N == 1 else D, weight=W.data_ptr(), ldw=FAR + odd if V == 1 else D,
                   logit_scale=1.0, target=t.data_ptr(), target_stride=1, ignore_index=-100)
    dtype = torch.float32 if grad else torch.bfloat16
    loss, lse = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    dh, dw = torch.empty(N, D, dtype=dtype, device="cuda"), torch.empty(V, D, dtype=dtype, device="cuda")
    n = g.gemm_head_workspace(a, 0, 0)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    g.gemm_ce_forward(a, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), n)
    n = g.gemm_head_workspace(a, 0, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    g.gemm_ce_backward(a, lse.data_ptr(), gl.data_ptr(), 1, dh.data_ptr(), FAR + odd if N == 1 else D,
                       dw.data_ptr(), FAR + odd if V == 1 else D, ws.data_ptr(), n)
    g.gemm_device_error(0)
    r = ref.Reference(H, W, gl, target=t, grad_dtype=torch.float32 if grad else None)
    for name, x in (("loss", loss), ("lse", lse), ("dhidden", dh), ("dweight", dw)):
        r.check(name, x)
