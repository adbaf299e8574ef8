"""The training command's corners: no steps, and steps whose tokens are all a
prompt's, which have no target to learn from."""
from __future__ import annotations

import math

import pytest

pytest.importorskip("torch")


def test_no_steps():
    from dense_gemm_tensor_tcgen05_gb300 import train_head
    with pytest.raises(ValueError, match="steps"):
        train_head.train(steps=0)


@pytest.mark.gpu
def test_steps_without_a_target():
    # one token a step, a quarter of them a prompt's: the weight stays a number
    from dense_gemm_tensor_tcgen05_gb300 import build, train_head
    build.build()
    seen = []
    train_head.train(tokens=1, vocab=512, dim=64, top_k=4, steps=24, say=seen.append)
    losses = [float(x.split()[-1]) for x in seen[:-1]]
    assert len(losses) == 24 and all(math.isfinite(x) for x in losses)
    assert 0.0 in losses and losses[-1] < 1e6
