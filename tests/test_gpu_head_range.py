"""The output layer's losses at the ends of their numbers' range: weights of
tokens, z terms and teacher logits that are huge, tiny, infinite or NaN.
Bounds as in head_ref.py unless said otherwise."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from tests import head_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def g():
    import dense_gemm_tensor_tcgen05_gb300 as g
    from dense_gemm_tensor_tcgen05_gb300 import build
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    build.build()
    return g


def done(g):
    g.gemm_device_error(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan], ids=["inf", "-inf", "nan"])
@pytest.mark.parametrize("N,D,piece", [(70, 64, 0), (300, 64, 0), (140, 101, 2 * 140 * 256)],
                         ids=["few", "many", "pieces"])
@pytest.mark.parametrize("kind", ["ce", "kd"])
def test_a_weight_that_is_not_finite_stays_with_its_token(g, kind, N, D, piece, value, dtype):
    # the other rows of dhidden are those of a call in which the token counts
    # for nothing; the weight's gradient sums all rows
    V, at = 900, 5
    H, W, t, gl = ref.inputs(N, V, D, dtype, 71)
    words, a = ref.teacher(N, V, 6, F32, 71)
    words[at] = torch.arange(6, device="cuda")
    a[at] = 0.0
    gl[at] = value
    if kind == "ce":
        loss, lse = g.linear_cross_entropy(H, W, t)
        dh, dw = g.linear_cross_entropy_backward(gl, H, W, t, lse, piece_bytes=piece)
        dh2, none = g.linear_cross_entropy_backward(gl, H, W, t, lse, piece_bytes=piece, need_weight=False)
    else:
        loss, lse = g.linear_distillation(H, W, words, a)
        dh, dw = g.linear_distillation_backward(gl, H, W, words, a, lse, piece_bytes=piece)
        dh2, none = g.linear_distillation_backward(gl, H, W, words, a, lse, piece_bytes=piece, need_weight=False)
    done(g)
    zero = gl.clone()
    zero[at] = 0.0
    o = dict(target=t) if kind == "ce" else dict(teacher_index=words, teacher_logits=a)
    r = ref.Reference(H, W, zero, **o)
    others = torch.arange(N, device="cuda") != at
    for got in (dh, dh2):
        assert not torch.isfinite(got[at]).any()
        rows = torch.where(others[:, None], got, torch.zeros_like(got))
        r.check("dhidden", rows)
    assert not torch.isfinite(dw).any()


def test_all_weights_infinite(g):
    H, W, t, _ = ref.inputs(40, 300, 64, BF16, 72)
    loss, lse = g.linear_cross_entropy(H, W, t)
    dh, dw = g.linear_cross_entropy_backward(torch.full((1,), math.inf, device="cuda"), H, W, t, lse)
    done(g)
    assert not torch.isfinite(dh).any() and not torch.isfinite(dw).any()
