"""What the losses' calls write: gradients with any row stride and start, and
nothing beside them -- not between their rows, not behind the workspace, loss
or lse.  The workspace holds NaN before the call."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from tests import head_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
GUARD = 4096          # bytes


@pytest.fixture(scope="module")
def g():
    import dense_gemm_tensor_tcgen05_gb300 as g
    from dense_gemm_tensor_tcgen05_gb300 import build
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    build.build()
    return g


class Fenced:
    """nbytes to be written (0xFF, which is NaN in every type, before), with
    the same pattern on both sides."""

    def __init__(self, nbytes):
        self.buf = torch.full((GUARD + nbytes + GUARD,), 0xFF, dtype=torch.uint8, device="cuda")

    def ptr(self):
        return self.buf.data_ptr() + GUARD

    def outside_is_untouched(self):
        return bool((self.buf[:GUARD] == 0xFF).all() and (self.buf[-GUARD:] == 0xFF).all())


class Matrix:
    """rows x cols in a fenced buffer, `ld` apart, from element `start` on."""

    def __init__(self, rows, cols, dtype, ld, start):
        self.rows, self.cols, self.ld, self.start, self.dtype = rows, cols, ld, start, dtype
        self.flat = torch.full((512 + rows * ld + 512,), 77.0, dtype=dtype, device="cuda")

    def ptr(self):
        return self.flat.data_ptr() + (256 + self.start) * self.flat.element_size()

    def value(self):
        at = 256 + self.start
        return self.flat[at: at + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols].clone()

    def beside_is_untouched(self):
        at = 256 + self.start
        x = self.flat.clone()
        x[at: at + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = 77.0
        return bool((x == 77.0).all())


SIZES = [(5, 300, 64), (130, 333, 72), (257, 1030, 136), (300, 700, 33), (4100, 500, 64)]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("grad", [0, 1], ids=["16", "f32"])
@pytest.mark.parametrize("pad,start", [(0, 0), (8, 0), (8, 8), (4, 4), (1, 0), (3, 1), (2, 5)])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_strides_of_the_gradients(g, size, pad, start, grad, dtype):
    N, V, D = size
    H, W, t, gl = ref.inputs(N, V, D, dtype, N + V + pad)
    t[::5] = -100
    if pad == 8:
        gl[::3] *= 2.0 ** -12                 # FP16: rows with scales of their own
    out = F32 if grad else dtype
    h = g.HeadArgs(dtype=int(dtype == BF16), grad_dtype=grad, tokens=N, vocab=V, dim=D, hidden=H.data_ptr(), ldh=D,
                   weight=W.data_ptr(), ldw=D, logit_scale=1.0, target=t.data_ptr(), target_stride=1,
                   ignore_index=-100, piece_bytes=2 * N * 512 if pad == 3 else 0)
    n = g.gemm_head_workspace(h, 0, 0)
    ws, loss, lse = Fenced(n), Fenced(4 * N), Fenced(4 * N)
    g.gemm_ce_forward(h, loss.ptr(), lse.ptr(), ws.ptr(), n)
    for x in (ws, loss, lse):
        assert x.outside_is_untouched()
    dh, dw = Matrix(N, D, out, D + pad, start), Matrix(V, D, out, D + pad, start)
    n = g.gemm_head_workspace(h, 0, 1)
    ws = Fenced(n)
    g.gemm_ce_backward(h, lse.ptr(), gl.data_ptr(), 1, dh.ptr(), D + pad, dw.ptr(), D + pad, ws.ptr(), n)
    g.gemm_device_error(0)
    assert ws.outside_is_untouched() and dh.beside_is_untouched() and dw.beside_is_untouched()
    r = ref.Reference(H, W, gl, target=t, grad_dtype=F32 if grad else None)
    r.check("dhidden", dh.value())
    r.check("dweight", dw.value())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("N,V,D,k", [(1, 3, 1, 1), (6, 300, 33, 256), (300, 520, 136, 33), (513, 77, 65, 5)])
def test_distillation_stays_inside(g, N, V, D, k, dtype):
    H, W, _, gl = ref.inputs(N, V, D, dtype, N + V)
    at, a = ref.teacher(N, V, k, F32, k)
    h = g.HeadArgs(dtype=int(dtype == BF16), tokens=N, vocab=V, dim=D, hidden=H.data_ptr(), ldh=D, weight=W.data_ptr(),
                   ldw=D, logit_scale=1.0, temperature=2.0, teacher_index=at.data_ptr(), ld_index=k,
                   teacher_logits=a.data_ptr(), ld_logits=k, top_k=k)
    n = g.gemm_head_workspace(h, 1, 0)
    ws, loss, lse = Fenced(n), Fenced(4 * N), Fenced(4 * N)
    g.gemm_distill_forward(h, loss.ptr(), lse.ptr(), ws.ptr(), n)
    for x in (ws, loss, lse):
        assert x.outside_is_untouched()
    dh, dw = Matrix(N, D, dtype, D + 3, 1), Matrix(V, D, dtype, D + 3, 1)
    n = g.gemm_head_workspace(h, 1, 1)
    ws = Fenced(n)
    g.gemm_distill_backward(h, lse.ptr(), gl.data_ptr(), 1, dh.ptr(), D + 3, dw.ptr(), D + 3, ws.ptr(), n)
    g.gemm_device_error(0)
    assert ws.outside_is_untouched() and dh.beside_is_untouched() and dw.beside_is_untouched()
    r = ref.Reference(H, W, gl, teacher_index=at, teacher_logits=a, temperature=2.0)
    r.check("dhidden", dh.value())
    r.check("dweight", dw.value())


def test_no_tokens_and_a_stride(g):
    dw = Matrix(300, 33, F32, 40, 3)
    h = g.HeadArgs(dtype=1, grad_dtype=1, tokens=0, vocab=300, dim=33, ldh=33, weight=1 << 40, ldw=33, logit_scale=1.0)
    g.gemm_ce_backward(h, 0, 0, 0, 0, 33, dw.ptr(), 40, 0, 0)
    torch.cuda.synchronize()
    assert dw.beside_is_untouched() and not dw.value().any()
