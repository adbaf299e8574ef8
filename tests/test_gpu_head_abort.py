"""The losses' tensor-core kernel when a pipeline wait runs out.

gemm_ce_stall_selftest runs an ordinary cross-entropy call with every wait
limited to some milliseconds and one cluster's copies withheld from a stage on.
The kernel gives up and returns, gemm_device_error says so once, and the next
call is right, bit for bit.  Nothing faults or hangs."""
from __future__ import annotations

import time

import pytest

torch = pytest.importorskip("torch")

from tests import head_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

LIMIT_MS = 20


@pytest.fixture(scope="module")
def g():
    import dense_gemm_tensor_tcgen05_gb300 as g
    from dense_gemm_tensor_tcgen05_gb300 import build
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    build.build()
    return g


class Call:
    def __init__(self, g, N, V, D):
        self.g = g
        self.tensors = H, W, t, _ = ref.inputs(N, V, D, torch.bfloat16, N)
        self.head = g.HeadArgs(dtype=1, tokens=N, vocab=V, dim=D, hidden=H.data_ptr(), ldh=D, weight=W.data_ptr(),
                               ldw=D, logit_scale=1.0, target=t.data_ptr(), target_stride=1, ignore_index=-100)
        self.n = g.gemm_head_workspace(self.head, 0, 0)
        self.ws = torch.empty(self.n, dtype=torch.uint8, device="cuda")
        self.out = torch.empty(2, N, device="cuda")
        self.stream = torch.cuda.current_stream().cuda_stream
        self.args = (self.head, self.out[0].data_ptr(), self.out[1].data_ptr(), self.ws.data_ptr(), self.n)

    def plain(self):
        self.out.fill_(-1.0)
        self.g.gemm_ce_forward(*self.args, self.stream)
        self.g.gemm_device_error(self.stream)
        return self.out.clone()

    def stalled(self, cluster, fill):
        self.g.gemm_ce_stall_selftest(*self.args, LIMIT_MS, cluster, fill, self.stream)


# few tokens (a ring of its own), rows read in place, gathered rows, and
# several tiles to a cluster
SIZES = [(20, 2000, 1024), (200, 2000, 1024), (600, 2000, 1024), (600, 40000, 512)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fill", [0, 2, 5])
def test_withheld_copies_time_out_and_the_next_call_is_right(g, size, fill):
    c = Call(g, *size)
    want = c.plain()
    began = time.perf_counter()
    c.stalled(0, fill)
    with pytest.raises(g.GemmError) as e:
        g.gemm_device_error(c.stream)
    assert e.value.name == "GEMM_ERR_DEVICE_TIMEOUT"
    assert time.perf_counter() - began < 1.5
    g.gemm_device_error(c.stream)             # said once
    for _ in range(2):
        assert torch.equal(c.plain(), want)


def test_the_last_cluster_in_its_second_tile(g):
    c = Call(g, 600, 40000, 512)              # 3 x 157 tiles of 4 stages
    want = c.plain()
    c.stalled(75, 6)
    with pytest.raises(g.GemmError) as e:
        g.gemm_device_error(c.stream)
    assert e.value.name == "GEMM_ERR_DEVICE_TIMEOUT"
    assert torch.equal(c.plain(), want)


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_stage_past_the_last_changes_nothing(g, size):
    c = Call(g, *size)
    want = c.plain()
    c.out.fill_(-1.0)
    c.stalled(0, 1 << 30)
    g.gemm_device_error(c.stream)
    assert torch.equal(c.out, want)


def test_refusals(g):
    c = Call(g, 20, 2000, 64)                 # eight tiles
    for cluster, fill in ((-1, 0), (8, 0), (0, -1)):
        with pytest.raises(g.GemmError) as e:
            c.stalled(cluster, fill)
        assert e.value.name == "GEMM_ERR_INVALID_VALUE"
    for limit in (0, 2001):
        with pytest.raises(g.GemmError) as e:
            g.gemm_ce_stall_selftest(*c.args, limit, 0, 0, c.stream)
        assert e.value.name == "GEMM_ERR_INVALID_VALUE"
