"""The output layer's workspace at the largest sizes that its calls accept (on
the host: no pointer is followed)."""
from __future__ import annotations

import ctypes
import itertools

import pytest

import dense_gemm_tensor_tcgen05_gb300 as g
from dense_gemm_tensor_tcgen05_gb300 import build

P = 1 << 32
MOST = (1 << 31) - 1024


@pytest.fixture(scope="module")
def L():
    build.build()
    return g.lib()


@pytest.mark.parametrize("distill", [0, 1])
@pytest.mark.parametrize("dtype", [0, 1])
def test_workspace_never_wraps(L, dtype, distill):
    # what is accepted needs at least its matrices' place and a count of bytes
    # that 64 bits hold; what is not is refused
    accepted = refused = 0
    for n, v, d in itertools.product((1, 1000, 1 << 19, 1 << 25, MOST), repeat=3):
        h = g.HeadArgs(dtype=dtype, tokens=n, vocab=v, dim=d, hidden=P, ldh=d, weight=2 * P, ldw=d, logit_scale=1.0,
                       temperature=1.0, target=3 * P, target_stride=1, teacher_index=3 * P, ld_index=4,
                       teacher_logits=4 * P, ld_logits=4, top_k=4, piece_bytes=(1 << 63) - 1)
        for backward in (0, 1):
            size = ctypes.c_int64(-1)
            st = L.gemm_head_workspace(h, distill, backward, size)
            if max(n * v, n * d, v * d) > 1 << 50:
                assert st == 1 and b"2^50" in L.gemm_last_cuda_error()
                refused += 1
                continue
            assert st == 0
            least = (2 if dtype == 1 else 4) * n * v + 2 * n * d if backward else n * v // 16
            assert least <= size.value < 1 << 61, (n, v, d, backward, size.value)
            accepted += 1
    assert accepted and refused
