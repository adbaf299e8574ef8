"""Sizes of the output layer's losses that take paths of their own: many tokens
and few words, where dweight's sums are cut along the tokens and joined; more
than 1024 channels, where the logits' gradient sums more than one chunk; more
than 2^17 words."""
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


def step(g, kind, N, V, D, dtype, *, ignored=0, grad_dtype=None, need=(True, True), piece=0, **o):
    """A training step and its reference; the gradients not asked for are None."""
    H, W, t, gl = ref.inputs(N, V, D, dtype, N + V + D)
    b = dict(grad_dtype=grad_dtype, need_hidden=need[0], need_weight=need[1], piece_bytes=piece)
    if kind == "ce":
        if ignored:
            t[::ignored] = -100
            H[::ignored] = math.nan
        loss, lse = g.linear_cross_entropy(H, W, t, **o)
        dh, dw = g.linear_cross_entropy_backward(gl, H, W, t, lse, **o, **b)
        r = ref.Reference(H, W, gl, target=t, grad_dtype=grad_dtype, **o)
    else:
        at, a = ref.teacher(N, V, 12, dtype, N + V)
        H[4::5] = math.inf
        loss, lse = g.linear_distillation(H, W, at, a, **o)
        dh, dw = g.linear_distillation_backward(gl, H, W, at, a, lse, **o, **b)
        r = ref.Reference(H, W, gl, teacher_index=at, teacher_logits=a, grad_dtype=grad_dtype, **o)
    g.gemm_device_error(torch.cuda.current_stream().cuda_stream)
    assert (dh is not None, dw is not None) == need
    for name, x in (("loss", loss), ("lse", lse), ("dhidden", dh), ("dweight", dw)):
        if x is not None:
            r.check(name, x)


MANY = [(8192, 500, 64), (2048, 500, 512), (8192, 4096, 256), (5001, 499, 65)]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", MANY, ids=lambda s: "x".join(map(str, s)))
def test_many_tokens_and_few_words(g, shape, dtype):
    step(g, "ce", *shape, dtype)


@pytest.mark.parametrize("kind", ["ce", "kd"])
@pytest.mark.parametrize("grad_dtype", [None, F32], ids=["same", "f32"])
@pytest.mark.parametrize("need", [(True, True), (False, True), (True, False)], ids=["both", "weight", "hidden"])
def test_many_tokens_with_masks(g, need, grad_dtype, kind):
    # two thirds of the slices' tokens are there; some slices of K end early
    step(g, kind, 4099, 700, 72, BF16, ignored=3, grad_dtype=grad_dtype, need=need)


def test_many_tokens_of_which_few_count(g):
    # most slices of dweight's sums are empty
    H, W, t, gl = ref.inputs(8000, 500, 64, BF16, 5)
    keep = torch.zeros(8000, dtype=torch.bool, device="cuda")
    keep[[0, 4000, 7999]] = True
    t[~keep] = -100
    loss, lse = g.linear_cross_entropy(H, W, t)
    dh, dw = g.linear_cross_entropy_backward(gl, H, W, t, lse)
    r = ref.Reference(H, W, gl, target=t)
    for name, x in (("loss", loss), ("lse", lse), ("dhidden", dh), ("dweight", dw)):
        r.check(name, x)


def test_many_tokens_in_pieces(g):
    # dweight's parts are used again by every piece of the vocabulary
    step(g, "ce", 4100, 1500, 64, F16, ignored=9, piece=2 * 4100 * 512)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("kind", ["ce", "kd"])
@pytest.mark.parametrize("shape", [(20, 600, 1025), (70, 600, 2100), (300, 520, 4608), (130, 300, 5001)],
                         ids=lambda s: "x".join(map(str, s)))
def test_many_channels(g, shape, kind, dtype):
    step(g, kind, *shape, dtype, ignored=6 if kind == "ce" else 0)


@pytest.mark.parametrize("kind", ["ce", "kd"])
@pytest.mark.parametrize("shape,dtype", [((1, 262144, 64), BF16), ((40, 180001, 40), F16), ((300, 151936, 24), BF16)],
                         ids=["1", "40", "300"])
def test_many_words(g, shape, dtype, kind):
    step(g, kind, *shape, dtype)
