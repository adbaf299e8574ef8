"""Train the output layer of a small student on a teacher's words.

    python -m dense_gemm_tensor_tcgen05_gb300.train_head [--tokens 2048] [--vocab 32768] \
        [--dim 1024] [--top-k 32] [--temperature 2] [--steps 20]

Each step draws hidden states, asks a fixed teacher layer for its logits (the
library's GEMM), keeps the teacher's top list and samples a target word for
each token from it; some tokens get no target, as a prompt's would.  The
student's layer then takes one step down the mean of cross entropy and
distillation:

    loss, lse = linear_cross_entropy(hidden, weight, target)
    _, dweight = linear_cross_entropy_backward(1 / n, ...)
    loss, lse = linear_distillation(hidden, weight, words, logits, temperature=T)
    _, dweight = linear_distillation_backward(1 / n, ...)

The gradients come back in FP32 (grad_dtype) and move an FP32 copy of the
weight by a fixed share of its length.  Prints both losses, and the mean time of a step's loss calls.
"""
from __future__ import annotations

import argparse


def train(tokens=2048, vocab=32768, dim=1024, top_k=32, temperature=2.0, steps=20, rate=0.1, seed=1,
          say=print):
    """The mean losses of the first and of the last step: ((ce, kd), (ce, kd))."""
    if steps < 1:
        raise ValueError("steps must be at least 1")
    import torch

    import dense_gemm_tensor_tcgen05_gb300 as g

    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda", generator=gen)
    teacher = (torch.randn(vocab, dim, **dev) * (3.0 / dim ** 0.5)).bfloat16()
    master = torch.randn(vocab, dim, **dev) * (0.5 / dim ** 0.5)
    states = torch.randn(tokens, dim, **dev)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    seen, spent = [], 0.0
    for step in range(steps):
        hidden = (states + 0.1 * torch.randn(tokens, dim, **dev)).bfloat16()
        logits = g.matmul(hidden, teacher.t())
        top, words = logits.topk(top_k, dim=1)
        chance = torch.rand(tokens, top_k, **dev).clamp_(1e-9, 1 - 1e-7)
        pick = (top - torch.log(-torch.log(chance))).argmax(1, keepdim=True)
        target = words.gather(1, pick)[:, 0]
        prompt = torch.rand(tokens, **dev) < 0.25
        target[prompt] = -100
        words[prompt] = -1
        each = (1.0 / (~prompt).sum().clamp(min=1)).float()   # a batch of prompts only takes no step
        weight = master.bfloat16()
        begin.record()
        ce, lse = g.linear_cross_entropy(hidden, weight, target)
        _, d1 = g.linear_cross_entropy_backward(each, hidden, weight, target, lse, need_hidden=False,
                                                grad_dtype=torch.float32)
        kd, lse = g.linear_distillation(hidden, weight, words, top, temperature=temperature)
        _, d2 = g.linear_distillation_backward(each, hidden, weight, words, top, lse, temperature=temperature,
                                               need_hidden=False, grad_dtype=torch.float32)
        end.record()
        down = d1 + d2
        master -= down * (rate * master.norm() / down.norm().clamp(min=1e-30))
        seen.append((float(ce.sum() * each), float(kd.sum() * each)))
        g.gemm_device_error(torch.cuda.current_stream().cuda_stream)
        if step:
            spent += begin.elapsed_time(end)
        say(f"step {step}: cross entropy {seen[-1][0]:.4f}, distillation {seen[-1][1]:.4f}")
    if steps > 1:
        say(f"{tokens} tokens x {vocab} words x {dim} channels: {spent / (steps - 1):.3f} ms a step in the loss calls")
    return seen[0], seen[-1]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=32768)
    ap.add_argument("--dim", type=int, default=1024)
    ap.add_argument("--top-k", type=int, default=32)
    ap.add_argument("--temperature", type=float, default=2.0)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=0.1, help="length of a step, in lengths of the weight")
    a = ap.parse_args()

    from dense_gemm_tensor_tcgen05_gb300 import build

    build.build()
    train(a.tokens, a.vocab, a.dim, a.top_k, a.temperature, a.steps, a.rate)


if __name__ == "__main__":
    main()
