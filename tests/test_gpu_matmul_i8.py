"""The 8-bit quantiser and product.  The integer sums are exact, so the
product is compared with a few fp32 roundings of its scales; codes and scales
are compared bit for bit with their fp32 definition."""
import pytest
import torch

import dense_ref as ref
from activation_sparse_decode_gemv_b200 import binding as pb

pytestmark = pytest.mark.gpu

D = torch.float64
E = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
SHAPES = [(1, 1, 16), (1, 1000, 528), (2, 129, 4096), (16, 128, 128), (17, 333, 272), (33, 1031, 1040), (64, 256, 2048),
          (65, 77, 144), (128, 512, 384), (129, 513, 1024), (200, 4099, 640), (257, 2050, 1296), (700, 1111, 400),
          (1500, 4099, 1040), (1000, 9001, 1040), (1600, 4099, 384), (2000, 5000, 400), (300, 5000, 528),
          (430, 9000, 272), (300, 12000, 272), (380, 10000, 400)]


def _codes(rows, k, gen):
    return torch.randint(-128, 128, (rows, k), generator=gen, device="cuda", dtype=torch.int32).to(torch.int8)


@pytest.mark.parametrize("out", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,n,k", SHAPES)
def test_product(cuda_device, T, n, k, out):
    gen = torch.Generator(device="cuda").manual_seed(T + n + k)
    xq, wq = _codes(T, k, gen), _codes(n, k, gen)
    xs = torch.rand(T, generator=gen, device="cuda") * 0.01
    ws_ = torch.rand(n, generator=gen, device="cuda") * 0.01
    bias = torch.randn(n, generator=gen, device="cuda") if k % 32 else None
    ws = pb.make_matmul_i8_workspace(T, n, k)
    pad = 64
    buf = torch.full((T * n + 2 * pad,), 7.0, dtype=out, device="cuda")
    y = buf[pad:pad + T * n].view(T, n)
    pb.pi_matmul_i8(xq, xs, wq, ws_, y, ws, bias=bias)
    assert pb.pi_get_device_status(ws) == 0
    assert torch.all(buf[:pad] == 7) and torch.all(buf[pad + T * n:] == 7), "written outside"
    main = (xq.to(D) @ wq.to(D).T) * xs.to(D)[:, None] * ws_.to(D)
    want = main if bias is None else main + bias.to(D)
    # int32 -> fp32, the product with one scale, the fused product with the other
    tol = 3 * E * main.abs() + 2 * E * want.abs() + (ref.step(out) * want.abs() if out is not F32 else 0)
    tol = tol + (2.0 ** -25 if out is F16 else 0)
    assert torch.all((y.to(D) - want).abs() <= tol)


def test_extreme_codes_and_longest_rows(cuda_device):
    """All codes -128 at the largest k: the sums come within 2^15 of 2^31."""
    k = 131056
    xq = torch.full((3, k), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((40, k), -128, dtype=torch.int8, device="cuda")
    wq[1], wq[2] = 127, 0
    one3, one = torch.ones(3, device="cuda"), torch.ones(40, device="cuda")
    y = torch.empty(3, 40, device="cuda")
    pb.pi_matmul_i8(xq, one3, wq, one, y, pb.make_matmul_i8_workspace(3, 40, k))
    want = (xq.to(D) @ wq.to(D).T).float()
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 16), (3, 528), (40, 1040), (1000, 64), (5, 8192), (2, 28672), (3, 40000)])
def test_quantiser(cuda_device, rows, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + k)
    x = (torch.randn(rows, k, generator=gen, device="cuda") * torch.exp(
        2 * torch.randn(rows, 1, generator=gen, device="cuda"))).to(dtype)
    if rows > 2:
        x[1] = 0
        x[2, :8] = x[2].abs().max() / 2  # ties: 63.5 to even
    q = torch.full((rows, k), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    pb.pi_quantize_i8(x, q, s)
    wq, wsc = ref.quantize(x.float())
    assert torch.equal(s, wsc) and torch.equal(q, wq)


def test_quantiser_on_extreme_values(cuda_device):
    x = torch.zeros(6, 32, device="cuda")
    x[0, 3] = float("nan")
    x[1, 5] = float("-inf")
    x[2] = 3.0e38
    x[3, 0] = 1e-45  # its scale underflows to zero
    x[4, 0], x[4, 1] = 1.5e-38, -3e-39  # subnormal scale
    x[5, 31] = -1.0
    q, s = torch.full((6, 32), 99, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    pb.pi_quantize_i8(x, q, s)
    assert torch.isnan(s[:2]).all() and torch.all(q[:2] == 0)
    assert torch.all(q[2] == 127) and torch.all(q[3] == 0) and s[3] == 0
    assert q[4, 0] == 127 and q[4, 1] == -25 and torch.all(q[4, 2:] == 0)  # 0.2 * 127 = 25.4
    assert q[5, 31] == -127 and torch.all(q[5, :31] == 0)
    # rows with a NaN scale poison their products, and no others
    w = torch.randint(-127, 128, (24, 32), device="cuda", dtype=torch.int32).to(torch.int8)
    y = torch.empty(6, 24, device="cuda")
    pb.pi_matmul_i8(q, s, w, torch.ones(24, device="cuda"), y, pb.make_matmul_i8_workspace(6, 24, 32))
    assert torch.isnan(y[:2]).all() and torch.isfinite(y[3:]).all()
    # row 2's products, near 3e38 * 1000, lie past fp32's largest value: infinities of their sign
    exact = (q[2].to(D) @ w.to(D).T) * s[2].to(D)
    assert torch.equal(y[2][exact.abs() > 3.5e38], torch.sign(exact[exact.abs() > 3.5e38]).float() * float("inf"))


@pytest.mark.parametrize("T", [1, 50, 300])
def test_quantised_product_is_near_the_plain_one(cuda_device, T):
    """Codes are off by half a step at most: |error| <= sum over k of the two half steps' products."""
    n, k = 520, 1040
    x, w = torch.randn(T, k, device="cuda", dtype=D), torch.randn(n, k, device="cuda", dtype=D) * 0.02
    xq, wq = torch.empty(T, k, dtype=torch.int8, device="cuda"), torch.empty(n, k, dtype=torch.int8, device="cuda")
    xs, ws_ = torch.empty(T, device="cuda"), torch.empty(n, device="cuda")
    pb.pi_quantize_i8(x.float(), xq, xs)
    pb.pi_quantize_i8(w.float(), wq, ws_)
    y = torch.empty(T, n, device="cuda")
    pb.pi_matmul_i8(xq, xs, wq, ws_, y, pb.make_matmul_i8_workspace(T, n, k))
    hx, hw = 0.501 * xs.to(D)[:, None], 0.501 * ws_.to(D)[:, None]
    bound = x.abs() @ hw.expand(n, k).T + hx.expand(T, k) @ (w.abs() + hw).T
    assert torch.all((y.to(D) - x @ w.T).abs() <= bound)


def test_no_tokens_and_replay(cuda_device):
    gen = torch.Generator(device="cuda").manual_seed(1)
    wq, sw = _codes(96, 64, gen), torch.ones(96, device="cuda")
    ws = pb.make_matmul_i8_workspace(40, 96, 64)
    e = torch.empty(0, 64, dtype=torch.int8, device="cuda")
    pb.pi_quantize_i8(torch.empty(0, 64, device="cuda"), e, torch.empty(0, device="cuda"))
    pb.pi_matmul_i8(e, torch.empty(0, device="cuda"), wq, sw, torch.empty(0, 96, device="cuda"), ws)
    x = torch.randn(40, 64, device="cuda")
    q, s, y = torch.empty(40, 64, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda"), torch.empty(40, 96, device="cuda")

    def step_():
        pb.pi_quantize_i8(x, q, s)
        pb.pi_matmul_i8(q, s, wq, sw, y, ws)
    step_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_()
    x.copy_(torch.randn(40, 64, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    got = y.clone()
    step_()
    assert torch.equal(got, y) and pb.pi_get_device_status(ws) == 0
