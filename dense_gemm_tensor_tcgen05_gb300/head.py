"""The output layer's losses: cross entropy and distillation of
logits = logit_scale * hidden @ weight.T without the tokens x vocab logits.

The gemm_* functions carry the C ABI's names and arguments (a ``HeadArgs``
structure, device pointers as ints, a stream handle); the ``linear_*``
functions take torch tensors, and torch supplies outputs and workspace.  A
training step is

    loss, lse = linear_cross_entropy(hidden, weight, target)
    dhidden, dweight = linear_cross_entropy_backward(grad_loss, hidden, weight, target, lse)

with grad_loss the gradient of what is optimised with respect to each token's
loss (for the mean over the tokens: 1 / their number).  autograd does not see
these calls: their results have no graph, also where hidden or weight requires
a gradient, so the backward call has to be made.  The formulas, the
treatment of tokens without a target and the precision are those of
include/gb300gemm.h.

Every call returns at once; the work is on the current stream, or on the one
given as ``stream``.  As with the C calls, what the stream waits for is the
caller's: inputs made on another stream need ``stream.wait_stream(...)``
first, and so does a stream that reads the results.  The inputs' memory is
not given to anyone else before that stream is done with it.
"""
from __future__ import annotations

import ctypes

from . import HeadArgs, _check, lib

torch = None   # imported by the first linear_* call; the C entry points need none


def _load_torch():
    global torch, _FLOAT16, _TEACHER_DTYPE
    import torch as module
    _FLOAT16 = {module.float16: 0, module.bfloat16: 1}
    _TEACHER_DTYPE = {module.float32: 0, module.float16: 1, module.bfloat16: 2}
    torch = module


# ---- the C ABI, one Python function per entry point (marshalling only) ----

def gemm_head_workspace(head: HeadArgs, distill: int, backward: int) -> int:
    n = ctypes.c_int64()
    _check(lib().gemm_head_workspace(head, distill, backward, n))
    return n.value


def gemm_ce_forward(head: HeadArgs, loss: int, lse: int, workspace: int, workspace_bytes: int,
                    stream: int = 0) -> None:
    _check(lib().gemm_ce_forward(head, loss, lse, workspace, workspace_bytes, stream or None))


def gemm_ce_stall_selftest(head: HeadArgs, loss: int, lse: int, workspace: int,
                           workspace_bytes: int, limit_ms: int, stall_cluster: int, stall_fill: int,
                           stream: int = 0) -> None:
    _check(lib().gemm_ce_stall_selftest(head, loss, lse, workspace, workspace_bytes, limit_ms,
                                        stall_cluster, stall_fill, stream or None))


def gemm_ce_backward(head: HeadArgs, lse: int, grad_loss: int, grad_stride: int, dhidden: int,
                     lddh: int, dweight: int, lddw: int, workspace: int, workspace_bytes: int,
                     stream: int = 0) -> None:
    _check(lib().gemm_ce_backward(head, lse, grad_loss, grad_stride, dhidden or None, lddh,
                                  dweight or None, lddw, workspace, workspace_bytes,
                                  stream or None))


def gemm_distill_forward(head: HeadArgs, loss: int, lse: int, workspace: int,
                         workspace_bytes: int, stream: int = 0) -> None:
    _check(lib().gemm_distill_forward(head, loss, lse, workspace, workspace_bytes, stream or None))


def gemm_distill_backward(head: HeadArgs, lse: int, grad_loss: int, grad_stride: int,
                          dhidden: int, lddh: int, dweight: int, lddw: int, workspace: int,
                          workspace_bytes: int, stream: int = 0) -> None:
    _check(lib().gemm_distill_backward(head, lse, grad_loss, grad_stride, dhidden or None, lddh,
                                       dweight or None, lddw, workspace, workspace_bytes,
                                       stream or None))


# ---- torch tensors ----------------------------------------------------------
#
# The smallest calls take less time on the GPU than their Python: the checks
# below read each attribute once.

def _rows(t, name: str, shared: bool = False) -> int:
    """Row stride of a 2-D tensor with unit column stride; rows that overlap
    (an expanded tensor) only where `shared` allows one row for all."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    ld, unit = t.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    if rows <= 1:
        return cols or 1
    if ld < cols and not (shared and ld == 0):
        raise ValueError(f"the rows of {name} overlap")
    return ld


def _numbers(t, name: str, tokens: int) -> int:
    """Stride of a tensor of one FP32 number a token (0: one for all)."""
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    shape = t.shape
    if len(shape) <= 1 and t.numel() == 1:
        return 0
    if shape != (tokens,):
        raise ValueError(f"{name} must have one number for each token")
    return t.stride(0)


def _on_one_gpu(index, others):
    """All tensors on the GPU of that index, which is the current one."""
    if index < 0:
        raise ValueError("all tensors must be on one GPU")
    for t in others:
        if t.get_device() != index:
            raise ValueError("all tensors must be on one GPU")
    if index != torch.cuda.current_device():
        raise ValueError("the tensors are not on the current device")


def _ce_head(hidden, weight, target, others, ignore_index, logit_scale, label_smoothing, z_loss,
             piece_bytes=0):
    if torch is None:
        _load_torch()
    dtype = _FLOAT16.get(hidden.dtype)
    if hidden.dtype != weight.dtype:
        raise TypeError("hidden and weight must have the same dtype")
    if dtype is None:
        raise TypeError(f"hidden must be float16 or bfloat16, not {hidden.dtype}")
    if target.dtype != torch.int64:
        raise TypeError("target must be int64")
    ldh, ldw = _rows(hidden, "hidden"), _rows(weight, "weight")
    tokens, dim = hidden.shape
    vocab, channels = weight.shape
    if channels != dim:
        raise ValueError(f"hidden has {dim} channels and weight {channels}")
    if target.shape != (tokens,):
        raise ValueError("target must have one word for each token")
    _on_one_gpu(hidden.get_device(), (weight, target, *others))
    return HeadArgs(dtype, 0, tokens, vocab, dim, hidden.data_ptr(), ldh, weight.data_ptr(), ldw,
                    logit_scale, label_smoothing, z_loss, 0.0, target.data_ptr(), target.stride(0),
                    ignore_index, None, 0, None, 0, 0, 0, piece_bytes)


def _distill_head(hidden, weight, index, logits, others, temperature, logit_scale, piece_bytes=0):
    if torch is None:
        _load_torch()
    dtype, teacher_dtype = _FLOAT16.get(hidden.dtype), _TEACHER_DTYPE.get(logits.dtype)
    if hidden.dtype != weight.dtype:
        raise TypeError("hidden and weight must have the same dtype")
    if dtype is None:
        raise TypeError(f"hidden must be float16 or bfloat16, not {hidden.dtype}")
    if index.dtype != torch.int64:
        raise TypeError("teacher_index must be int64")
    if teacher_dtype is None:
        raise TypeError("teacher_logits must be float32, float16 or bfloat16")
    ldh, ldw = _rows(hidden, "hidden"), _rows(weight, "weight")
    tokens, dim = hidden.shape
    vocab, channels = weight.shape
    if channels != dim:
        raise ValueError(f"hidden has {dim} channels and weight {channels}")
    shape = index.shape
    if len(shape) != 2 or shape != logits.shape or shape[0] != tokens:
        raise ValueError("teacher_index and teacher_logits must be tokens x top_k")
    ld_index, ld_logits = _rows(index, "teacher_index", True), _rows(logits, "teacher_logits", True)
    _on_one_gpu(hidden.get_device(), (weight, index, logits, *others))
    return HeadArgs(dtype, 0, tokens, vocab, dim, hidden.data_ptr(), ldh, weight.data_ptr(), ldw,
                    logit_scale, 0.0, 0.0, temperature, None, 0, 0, index.data_ptr(), ld_index,
                    logits.data_ptr(), ld_logits, teacher_dtype, shape[1], piece_bytes)


def _run(call, head, distill, backward, device, inputs, outputs, stream):
    """Outputs and workspace from torch on the stream that the call runs on:
    `outputs` makes the tensors and gives what `call` takes between head and
    workspace.  A caller may drop the inputs once the call has returned, so
    torch is told when the stream is not the one that they were made on."""
    if stream is None:
        made, args = outputs()
        n = gemm_head_workspace(head, distill, backward)
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        handle = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        with torch.cuda.stream(stream):
            made, args = outputs()
            n = gemm_head_workspace(head, distill, backward)
            ws = torch.empty(n, dtype=torch.uint8, device=device)
        handle = stream.cuda_stream
        for t in inputs:
            t.record_stream(stream)
    call(head, *args, ws.data_ptr(), n, handle)
    return made


def _forward(head, distill, inputs, stream):
    device = inputs[0].device

    def outputs():
        loss = torch.empty(head.tokens, dtype=torch.float32, device=device)
        lse = torch.empty(head.tokens, dtype=torch.float32, device=device)
        return (loss, lse), (loss.data_ptr(), lse.data_ptr())

    return _run(gemm_distill_forward if distill else gemm_ce_forward, head, distill, 0, device,
                inputs, outputs, stream)


def _backward(head, distill, inputs, need_hidden, need_weight, grad_dtype, stream):
    grad_loss, lse, hidden, weight = inputs[:4]
    dtype = hidden.dtype
    if grad_dtype is not None and grad_dtype != dtype:
        if grad_dtype != torch.float32:
            raise TypeError(f"gradients are {dtype} or float32, not {grad_dtype}")
        head.grad_dtype, dtype = 1, grad_dtype
    tokens, dim = hidden.shape
    stride = _numbers(grad_loss, "grad_loss", tokens)
    if lse.dtype != torch.float32 or lse.shape != (tokens,) or (tokens > 1 and lse.stride(0) != 1):
        raise ValueError("lse must be the forward call's")
    device = hidden.device

    def outputs():
        dh = torch.empty((tokens, dim), dtype=dtype, device=device) if need_hidden else None
        dw = torch.empty((weight.shape[0], dim), dtype=dtype, device=device) if need_weight else None
        return (dh, dw), (lse.data_ptr(), grad_loss.data_ptr(), stride,
                          dh.data_ptr() if need_hidden else 0, dim or 1,
                          dw.data_ptr() if need_weight else 0, dim or 1)

    return _run(gemm_distill_backward if distill else gemm_ce_backward, head, distill, 1, device,
                inputs, outputs, stream)


def linear_cross_entropy(hidden, weight, target, *, ignore_index=-100, logit_scale=1.0,
                         label_smoothing=0.0, z_loss=0.0, stream=None):
    """(loss, lse), float32, one number for each token: the cross entropy of
    logits = logit_scale * hidden @ weight.T with target, and the logits'
    log-sum-exp (which the backward call takes).

    hidden: tokens x dim; weight: vocab x dim; both float16 or both bfloat16,
    row-major with any row stride.  target: int64, one word for each token;
    a token with target == ignore_index has loss 0 and lse 0.  See
    include/gb300gemm.h for label_smoothing and z_loss.  Returns at once, on
    the current (or given) stream, without a graph for autograd.
    """
    head = _ce_head(hidden, weight, target, (), ignore_index, logit_scale, label_smoothing, z_loss)
    return _forward(head, 0, (hidden, weight, target), stream)


def linear_cross_entropy_backward(grad_loss, hidden, weight, target, lse, *, ignore_index=-100,
                                  logit_scale=1.0, label_smoothing=0.0, z_loss=0.0,
                                  need_hidden=True, need_weight=True, grad_dtype=None,
                                  piece_bytes=0, stream=None):
    """(dhidden, dweight): the gradients of sum(grad_loss * loss).

    grad_loss: float32, one number for each token (any stride) or a single
    one for all.  lse: the forward call's; the other arguments are those of
    the forward call.  Gradients have hidden's dtype, or float32 with
    grad_dtype=torch.float32 (not rounded again, but with the errors of the
    logits' gradient, which is held in hidden's dtype); one that is not needed is None and not
    computed.  piece_bytes bounds the piece of the logits' gradient that is
    held at a time (0: 1 GiB; float16 has room for two copies of it).
    """
    head = _ce_head(hidden, weight, target, (grad_loss, lse), ignore_index, logit_scale,
                    label_smoothing, z_loss, piece_bytes)
    return _backward(head, 0, (grad_loss, lse, hidden, weight, target), need_hidden, need_weight,
                     grad_dtype, stream)


def linear_distillation(hidden, weight, teacher_index, teacher_logits, *, temperature=1.0,
                        logit_scale=1.0, stream=None):
    """(loss, lse), float32, one number for each token: temperature^2 times
    the divergence of softmax(logits / temperature), logits = logit_scale *
    hidden @ weight.T, from the softmax of the teacher's top logits /
    temperature, and the log-sum-exp of logits / temperature.

    teacher_index: int64, tokens x top_k, the teacher's words; an entry
    outside [0, vocab) (-1, say) is not there.  teacher_logits: float32,
    float16 or bfloat16 of the same shape; -inf masks an entry too.  A token
    without an entry has loss 0 and lse 0.
    """
    head = _distill_head(hidden, weight, teacher_index, teacher_logits, (), temperature, logit_scale)
    return _forward(head, 1, (hidden, weight, teacher_index, teacher_logits), stream)


def linear_distillation_backward(grad_loss, hidden, weight, teacher_index, teacher_logits, lse, *,
                                 temperature=1.0, logit_scale=1.0, need_hidden=True,
                                 need_weight=True, grad_dtype=None, piece_bytes=0, stream=None):
    """(dhidden, dweight): the gradients of sum(grad_loss * loss) of
    linear_distillation, with the arguments of
    linear_cross_entropy_backward."""
    head = _distill_head(hidden, weight, teacher_index, teacher_logits, (grad_loss, lse),
                         temperature, logit_scale, piece_bytes)
    return _backward(head, 1, (grad_loss, lse, hidden, weight, teacher_index, teacher_logits),
                     need_hidden, need_weight, grad_dtype, stream)
