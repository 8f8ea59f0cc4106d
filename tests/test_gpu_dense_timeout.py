"""The dense products' bounded waits, without a GPU fault: the finished
accumulators are not announced (pi_debug_wait_fault), every load and product is
issued and lands as always, and each wait is limited to 2 ms.  The kernels give
up, record PI_ERR_TIMEOUT and complete; the same workspace serves the next call,
whose results are exact."""
import pytest
import torch

import dense_plans as dp
from activation_sparse_decode_gemv_b200 import binding as pb
from test_gpu_dense_plans import _backward, _forward, _product

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _layer(T, d, f):
    w = [torch.randn(f, d, device="cuda").to(BF16) for _ in range(3)]
    layer = pb.GatedFfnLayer(*w)
    return layer, pb.make_gated_ffn_workspace(layer, T, True), [torch.zeros(T, n, dtype=BF16, device="cuda")
                                                                for n in (d, d, f, f, d, d)]


def _timed_out(ws, call):
    try:
        pb.pi_debug_wait_fault(0, 2000)
        call()
        torch.cuda.synchronize()  # the kernels completed
    finally:
        pb.pi_debug_wait_fault(-1, 0)
    assert pb.pi_get_device_status(ws) == pb.PI_ERR_TIMEOUT
    assert pb.pi_get_device_status(ws) == pb.PI_OK  # reading clears it


# (product's tiling: two accumulator buffers, one, split), a tile for each CTA pair and several
PLANS = [{}, {dp.GLU: (2, 128, 0), dp.STORE: (2, 192, 0), dp.DGLU: (1, 256, 0), dp.WEIGHT: (2, 256, 0)},
         {dp.GLU: (2, 256, 0), dp.STORE: (1, 160, 0), dp.DGLU: (1, 128, 0), dp.WEIGHT: (1, 256, 0)},
         {dp.GLU: (1, 16, 1), dp.STORE: (1, 48, 4), dp.DGLU: (1, 128, 8)}]


@pytest.mark.parametrize("plans", PLANS, ids=["rule", "pairs", "pairs2", "split"])
@pytest.mark.parametrize("T,d,f", [(2, 1096, 520), (300, 1096, 520), (700, 1096, 9000)])
def test_waits_run_out_and_the_workspace_recovers(cuda_device, T, d, f, plans):
    layer, ws, (u, y, gate, up, dy, du) = _layer(T, d, f)
    dw = [torch.zeros(f, d, dtype=F32, device="cuda") for _ in range(3)]
    try:
        for product, p in plans.items():
            pb.pi_debug_dense_plan(product, *p)
        _timed_out(ws, lambda: pb.pi_gated_ffn_forward(layer, u, y, ws, gate=gate, up=up))
        _timed_out(ws, lambda: pb.pi_gated_ffn_backward(layer, u, gate, up, dy, ws, du, *dw))
        # the same workspace, another call: u = 0 gives 0, and a stale value would show
        y.fill_(7)
        pb.pi_gated_ffn_forward(layer, u, y, ws, gate=gate, up=up)
        assert pb.pi_get_device_status(ws) == 0 and torch.all(y == 0) and torch.all(gate == 0) and torch.all(up == 0)
        _forward(T, d, f, BF16)
        _backward(T, d, f, BF16)
    finally:
        pb.pi_debug_dense_plan(-1)


@pytest.mark.parametrize("plan", [(1, 256, 0), (1, 128, 0), (1, 64, 2)])
@pytest.mark.parametrize("T,n", [(2, 520), (700, 19000)])
def test_waits_of_the_8_bit_product(cuda_device, T, n, plan):
    k = 1040
    xq, wq = (torch.ones(r, k, dtype=torch.int8, device="cuda") for r in (T, n))
    xs, sw, y = torch.ones(T, device="cuda"), torch.ones(n, device="cuda"), torch.zeros(T, n, device="cuda")
    ws = pb.make_matmul_i8_workspace(T, n, k)
    try:
        pb.pi_debug_dense_plan(dp.I8, *plan)
        _timed_out(ws, lambda: pb.pi_matmul_i8(xq, xs, wq, sw, y, ws))
        pb.pi_matmul_i8(xq, xs, wq, sw, y, ws)
        assert pb.pi_get_device_status(ws) == 0 and torch.all(y == k)
        _product(T, n, k, F32, None)
    finally:
        pb.pi_debug_dense_plan(-1)


def test_a_short_limit_alone_changes_nothing(cuda_device):
    """Waits that do not run out: results as always."""
    try:
        pb.pi_debug_wait_fault(-1, 500_000)
        _forward(300, 264, 520, BF16)
        _backward(300, 264, 520, BF16)
    finally:
        pb.pi_debug_wait_fault(-1, 0)
