"""The output layer's losses on a stream that is not the one the inputs were
made on: the caller drops the inputs when the call has returned, while the
stream has yet to read them."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from tests import head_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

N, V, D = 300, 2000, 128


@pytest.fixture(scope="module")
def g():
    import dense_gemm_tensor_tcgen05_gb300 as g
    from dense_gemm_tensor_tcgen05_gb300 import build
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    build.build()
    return g


def keep_busy(stream):
    """Work of some 50 ms on the stream (plain products)."""
    with torch.cuda.stream(stream):
        x = torch.ones(4096, 4096, device="cuda")
        for _ in range(12):
            x = (x @ x).clamp_(0, 1)


def overwrite(like):
    """Takes freed memory of these sizes again and writes into it."""
    taken = []
    for t in like:
        for _ in range(4):
            x = torch.empty(t[0], dtype=t[1], device="cuda")
            taken.append(x.zero_())
    return taken


@pytest.mark.parametrize("kind", ["ce", "kd"])
def test_inputs_may_be_dropped(g, kind):
    H, W, t, gl = ref.inputs(N, V, D, torch.bfloat16, 81)
    at, a = ref.teacher(N, V, 8, torch.float32, 81)
    side = torch.cuda.Stream()

    def inputs():
        return [x.clone() for x in ((H, W, t) if kind == "ce" else (H, W, at, a))]

    fwd = g.linear_cross_entropy if kind == "ce" else g.linear_distillation
    back = g.linear_cross_entropy_backward if kind == "ce" else g.linear_distillation_backward
    x = inputs()
    shapes = [(y.shape, y.dtype) for y in x] + [(gl.shape, gl.dtype)]
    want = fwd(*x)
    want += back(gl, *x, want[1])
    torch.cuda.synchronize()
    del x

    x = inputs()
    side.wait_stream(torch.cuda.current_stream())
    keep_busy(side)
    loss, lse = fwd(*x, stream=side)
    del x
    taken = overwrite(shapes)
    torch.cuda.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
    del taken

    x, gc = inputs(), gl.clone()
    side.wait_stream(torch.cuda.current_stream())
    keep_busy(side)
    dh, dw = back(gc, *x, lse, stream=side)
    del x, gc
    taken = overwrite(shapes)
    torch.cuda.synchronize()
    assert torch.equal(dh, want[2]) and torch.equal(dw, want[3])
