"""Host threads whose first CUDA call is a call of this library: no context is
current on such a thread, and some plans encode tensor maps before anything
that would make one current."""
from __future__ import annotations

import threading

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


def on_a_new_thread(call):
    errors = []

    def run():
        try:
            call()
        except Exception as e:   # noqa: BLE001
            errors.append(repr(e))

    for _ in range(2):           # the library's own caches are filled by the first
        th = threading.Thread(target=run)
        th.start()
        th.join()
    torch.cuda.synchronize()
    assert not errors, errors


@pytest.mark.parametrize("M,N,K", [(256, 256, 256), (2048, 2048, 256), (4096, 4096, 512), (100, 100, 64),
                                   (64, 8192, 4096)])
@pytest.mark.parametrize("name", ["gemm_f16f32", "gemm_ex", "gemm_ex_noalloc"])
def test_gemm(g, name, M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    A = torch.randint(-8, 9, (M, K), generator=gen, device="cuda").half()
    B = torch.randint(-8, 9, (K, N), generator=gen, device="cuda").half()
    C = torch.full((M, N), -1.0, device="cuda")
    torch.cuda.synchronize()
    args = (A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, K, N, N)
    kw = {} if name == "gemm_f16f32" else dict(dtype=0)
    on_a_new_thread(lambda: getattr(g, name)(*args, **kw))
    assert torch.equal(C, A.float() @ B.float())     # sums of integers below 2^24: exact in any order
