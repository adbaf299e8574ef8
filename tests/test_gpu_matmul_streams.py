"""matmul on a stream that is not the one its operands were made on: the
caller drops them when the call has returned, while the stream has yet to
read them."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import dense_gemm_tensor_tcgen05_gb300 as g
    from dense_gemm_tensor_tcgen05_gb300 import build
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    build.build()
    return g


@pytest.mark.parametrize("dtype,opts", [(torch.bfloat16, {}), (torch.float32, {}), (torch.float16, {"alpha": 2.0})],
                         ids=["bf16", "f32", "options"])
def test_operands_may_be_dropped(g, dtype, opts):
    gen = torch.Generator(device="cuda").manual_seed(82)
    A = torch.randn(300, 500, generator=gen, device="cuda").to(dtype)
    B = torch.randn(500, 700, generator=gen, device="cuda").to(dtype)
    want = g.matmul(A, B, **opts)
    side = torch.cuda.Stream()
    x, y = A.clone(), B.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):          # work of some 50 ms before the call's
        busy = torch.ones(4096, 4096, device="cuda")
        for _ in range(12):
            busy = (busy @ busy).clamp_(0, 1)
    got = g.matmul(x, y, stream=side, **opts)
    del x, y
    taken = [torch.empty(s, dtype=dtype, device="cuda").zero_() for s in (A.shape, B.shape) * 4]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del taken
