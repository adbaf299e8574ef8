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


class Gradients:
    """dhidden and dweight of the cross entropy in 64 bits (CPU) for any z
    term, with bounds.

    z and lse are off by dz and dlse as in head_ref.py.  The logits' gradient
    of token n is G = k (p (1 + t) - y), k = grad_loss scale, t = 2 z_loss lse,
    at most S_n = |k| (1 + |t|) in size; the errors of p and t move it by

        |k| (p |1 + t| (dz + dlse + 2^-20) + 2 z_loss p dlse)

    and FP32 by 2^-22 of its terms.  It is rounded to 16 bits: u of itself,
    and in FP16 at least half a step of 2^-24 in the unit 2^-14 max S."""

    def __init__(self, H, W, t, gl, z_loss, grad_dtype, scale=1.0):
        ty = H.dtype
        H, W, t = H.cpu().double(), W.cpu().double(), t.cpu()
        N, D = H.shape
        V = W.shape[0]
        k = gl.cpu().double().expand(N) * scale
        z = (H @ W.T) * scale
        lse = torch.logsumexp(z, 1)
        y = torch.zeros(N, V, dtype=torch.float64).scatter_(1, t[:, None], 1.0)
        p = torch.exp(z - lse[:, None])
        term = 2.0 * z_loss * lse
        G = (p * (1.0 + term)[:, None] - y) * k[:, None]
        self.dhidden, self.dweight = G @ W, G.T @ H
        dz = ref.acc(D) * (H.abs() @ W.abs().T) * scale + 2.0 ** -22 * z.abs()
        dlse = (dz.amax(1) + 2.0 ** -15 + 2.0 ** -21 * z.abs().amax(1))[:, None]
        size, K = (1.0 + term).abs()[:, None], k.abs()[:, None]
        S = K * (1.0 + term.abs())[:, None]
        u, go = ref.U[ty], ref.U[grad_dtype]
        step = 0.0 if ty == BF16 else 2.0 ** -39 * S.max()
        dG = K * p * (size * (dz + dlse + 2.0 ** -20) + 2.0 * z_loss * dlse) + 2.0 ** -22 * K * (p * size + y) \
            + u * G.abs() + step + 2.0 ** -125 * (S + 1)
        tiny = 2.0 ** -25 if grad_dtype == F16 else 2.0 ** -125
        self.tol = {
            "dhidden": (dG + ref.acc(V) * G.abs()) @ W.abs() * (1 + go) + (go + 2.0 ** -22) * self.dhidden.abs() + tiny,
            "dweight": (dG + ref.acc(N) * G.abs()).T @ H.abs() * (1 + go) + (go + 2.0 ** -22) * self.dweight.abs() + tiny,
        }

    check = ref.Reference.check


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("N", [70, 300])
@pytest.mark.parametrize("z_loss,spread,shift", [(1.0, 20.0, 0.0), (0.1, 120.0, 0.0), (1.0, 1.5, -256.0),
                                                 (10.0, 1.5, 256.0), (1e-4, 1.5, 0.0)],
                         ids=["1", "0.1-wide", "negative", "10-large", "usual"])
def test_z_terms_of_any_size(g, z_loss, spread, shift, N, dtype):
    # 1 + 2 z_loss lse from -500 to 5000: the logits' gradient passes FP16's
    # range many times, the gradients themselves are ordinary numbers
    H, W, t, gl = ref.inputs(N, 700, 64, dtype, 73, spread=spread)
    if shift:                              # a channel that moves all logits
        H[:, 0] = 8.0
        W[:, 0] = shift / 8.0
    gl *= 1e-3
    loss, lse = g.linear_cross_entropy(H, W, t, z_loss=z_loss)
    dh, dw = g.linear_cross_entropy_backward(gl, H, W, t, lse, z_loss=z_loss, grad_dtype=F32)
    done(g)
    r = Gradients(H, W, t, gl, z_loss, F32)
    r.check("dhidden", dh)
    r.check("dweight", dw)


def row_by_row(got, gl, unit):
    """Rows of dhidden for weights gl that are powers of two, divided by them
    (exact): each is bounded as the row of a call in which every token has
    weight 1, whatever the others' weights are."""
    x = got.detach().cpu().double() / gl.cpu().double()[:, None]
    unit.check("dhidden", x)


@pytest.mark.parametrize("N,V,D,piece", [(40, 5000, 64, 0), (300, 3001, 72, 0), (130, 2500, 101, 2 * 130 * 512),
                                         (24, 40000, 40, 0)], ids=["few", "many", "pieces", "wide"])
@pytest.mark.parametrize("kind", ["ce", "kd", "z"])
def test_rows_of_little_weight(g, kind, N, V, D, piece):
    # FP16, weights from 1 down to 2^-40, either sign, both gradients at once
    # and each alone
    H, W, t, _ = ref.inputs(N, V, D, F16, 74)
    gl = (2.0 ** -torch.randint(0, 41, (N,), generator=torch.Generator().manual_seed(1)).double()).float()
    gl[0], gl[1], gl[2] = 1.0, 2.0 ** -24, -2.0 ** -20
    gl = gl.cuda()
    one = torch.ones(N, device="cuda")
    if kind == "kd":
        at, a = ref.teacher(N, V, 9, F32, 74)
        o = dict(temperature=2.0)
        loss, lse = g.linear_distillation(H, W, at, a, **o)
        back = lambda **k: g.linear_distillation_backward(gl, H, W, at, a, lse, grad_dtype=F32, piece_bytes=piece, **o, **k)
        unit = ref.Reference(H, W, one, teacher_index=at, teacher_logits=a, grad_dtype=F32, **o)
        r = ref.Reference(H, W, gl, teacher_index=at, teacher_logits=a, grad_dtype=F32, **o)
    else:
        o = dict(z_loss=1e-3) if kind == "z" else {}
        t[6::7] = -100
        loss, lse = g.linear_cross_entropy(H, W, t, **o)
        back = lambda **k: g.linear_cross_entropy_backward(gl, H, W, t, lse, grad_dtype=F32, piece_bytes=piece, **o, **k)
        unit = ref.Reference(H, W, one, target=t, grad_dtype=F32, **o)
        r = ref.Reference(H, W, gl, target=t, grad_dtype=F32, **o)
    dh, dw = back()
    dh1, none = back(need_weight=False)
    none, dw1 = back(need_hidden=False)
    done(g)
    row_by_row(dh, gl, unit)
    r.check("dweight", dw)
    assert torch.equal(dh, dh1)
    r.check("dweight", dw1)


def test_a_weight_that_is_not_finite_beside_small_ones(g):
    H, W, t, _ = ref.inputs(50, 900, 64, F16, 75)
    gl = torch.full((50,), 2.0 ** -30, device="cuda")
    gl[0], gl[7], gl[8] = 1.0, math.inf, 0.0
    loss, lse = g.linear_cross_entropy(H, W, t)
    dh, dw = g.linear_cross_entropy_backward(gl, H, W, t, lse, grad_dtype=F32)
    done(g)
    assert not torch.isfinite(dh[7]).any() and not torch.isfinite(dw).any() and not dh[8].any()
    keep = torch.tensor([i for i in range(50) if i not in (7, 8)])
    unit = ref.Reference(H[keep], W, torch.ones(48, device="cuda"), target=t[keep], grad_dtype=F32)
    row_by_row(dh[keep], gl[keep], unit)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [0.25, 0.5, 1.0, 4.0])
def test_teacher_logits_at_the_ends_of_their_type(g, T, dtype):
    # the lowest finite number counts for nothing beside others and for all
    # where there are no others, at any temperature; so does the largest
    H, W, _, gl = ref.inputs(40, 300, 64, BF16, 76)
    at, a = ref.teacher(40, 300, 8, dtype, 76)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    a[:, 4:] = low
    a[7] = low
    a[8, :2] = high
    a[10] = high
    at[7], at[10] = torch.arange(8, device="cuda"), torch.arange(8, device="cuda")
    loss, lse = g.linear_distillation(H, W, at, a, temperature=T)
    dh, dw = g.linear_distillation_backward(gl, H, W, at, a, lse, temperature=T)
    done(g)
    r = ref.Reference(H, W, gl, teacher_index=at, teacher_logits=a, temperature=T)
    for name, x in (("loss", loss), ("lse", lse), ("dhidden", dh), ("dweight", dw)):
        r.check(name, x)


def test_a_graph_takes_weights_of_either_kind(g):
    # captured with equal weights, replayed with ones that differ much: the
    # device decides at every replay
    N, V, D = 90, 1500, 64
    H, W, t, _ = ref.inputs(N, V, D, F16, 77)
    gl = torch.ones(N, device="cuda")
    loss, lse = g.linear_cross_entropy(H, W, t)
    g.linear_cross_entropy_backward(gl, H, W, t, lse, grad_dtype=F32)      # loads the kernels
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dh, dw = g.linear_cross_entropy_backward(gl, H, W, t, lse, grad_dtype=F32)
    unit = ref.Reference(H, W, torch.ones(N, device="cuda"), target=t, grad_dtype=F32)
    for low in (0, 30, 0):
        gl.copy_((2.0 ** -(torch.arange(N) % (low + 1)).double()).float())
        graph.replay()
        done(g)
        row_by_row(dh, gl, unit)
        ref.Reference(H, W, gl, target=t, grad_dtype=F32).check("dweight", dw)
