"""Every tiling of every dense product, whatever the rule would take: exact on
whole numbers (see test_gpu_gated_ffn), with more tiles than the machine holds
at once, ragged edges on both axes, and from one K block to several turns of
the ring."""
import pytest
import torch

import dense_plans as dp
import dense_ref as ref
from activation_sparse_decode_gemv_b200 import binding as pb
from test_gpu_gated_ffn import _guarded, _int_case

pytestmark = pytest.mark.gpu

D = torch.float64
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF = pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])


@pytest.fixture
def plan():
    yield lambda product, mb, nt, split: pb.pi_debug_dense_plan(product, mb, nt, split)
    pb.pi_debug_dense_plan(-1)


def _forward(T, d, f, dtype):
    u, wg, wu, wd, _ = _int_case(T, d, f, dtype)
    layer = pb.GatedFfnLayer(wg, wu, wd, act="relu")
    ws = pb.make_gated_ffn_workspace(layer, T)
    outs = [_guarded(T, n, dtype) for n in (d, f, f)]
    (y, _), (g, _), (p, _) = outs
    pb.pi_gated_ffn_forward(layer, u, y, ws, gate=g, up=p)
    assert pb.pi_get_device_status(ws) == 0
    [check() for _, check in outs]
    _, gr, pr, ar = ref.ffn_forward("relu", u.to(D), wg.to(D), wu.to(D), wd.to(D))
    assert gr.abs().max() <= 256 and ar.abs().max() <= 2048
    assert torch.equal(g.to(D), gr) and torch.equal(p.to(D), pr)
    yr = ar.to(dtype).to(D) @ wd.to(D)
    assert yr.abs().max() < 2 ** 24 and torch.equal(y, yr.to(dtype))


def _backward(T, d, f, dtype, gtype=None, start=None, only=None):
    """only: names of the outputs wanted; start: the value that gradients are added to."""
    u, wg, wu, wd, dy = _int_case(T, d, f, dtype)
    layer = pb.GatedFfnLayer(wg, wu, wd, act="relu")
    ws = pb.make_gated_ffn_workspace(layer, T, True)
    _, g, p, _ = ref.ffn_forward("relu", u.to(D), wg.to(D), wu.to(D), wd.to(D))
    g, p = g.to(dtype), p.to(dtype)
    names = only or ("du", "dw_gate", "dw_up", "dw_down_t")
    outs = {k: _guarded(T, d, dtype) if k == "du" else _guarded(f, d, gtype or dtype) for k in names}
    if start is not None:
        [o.fill_(start) for k, (o, _) in outs.items() if k != "du"]
    pb.pi_gated_ffn_backward(layer, u, g, p, dy, ws, **{k: o for k, (o, _) in outs.items()},
                             flags=0 if start is None else pb.PI_GRAD_ACCUMULATE)
    assert pb.pi_get_device_status(ws) == 0
    *_, dg, dpp, a = ref.ffn_backward("relu", u.to(D), g.to(D), p.to(D), dy.to(D), wg.to(D), wu.to(D), wd.to(D))
    dg, dpp, a = (t.to(dtype).to(D) for t in (dg, dpp, a))
    want = {"du": lambda: dg @ wg.to(D) + dpp @ wu.to(D), "dw_gate": lambda: dg.T @ u.to(D),
            "dw_up": lambda: dpp.T @ u.to(D), "dw_down_t": lambda: a.T @ dy.to(D)}
    for k, (o, check) in outs.items():
        check()
        w = want[k]() + (0 if start is None or k == "du" else start)
        assert w.abs().max() < 2 ** 24 and torch.equal(o, w.to(o.dtype)), k


def _product(T, n, k, out, bias):
    gen = torch.Generator(device="cuda").manual_seed(T + n + k)
    code = lambda r: torch.randint(-128, 128, (r, k), generator=gen, device="cuda", dtype=torch.int32).to(torch.int8)  # noqa: E731
    xq, wq = code(T), code(n)
    # powers of two: the scaled sums, and with whole biases the results, are exact in fp32 below 2^24
    xs = 2.0 ** torch.randint(-3, 3, (T,), generator=gen, device="cuda")
    sw = 2.0 ** torch.randint(-3, 3, (n,), generator=gen, device="cuda")
    ws = pb.make_matmul_i8_workspace(T, n, k)
    y, check = _guarded(T, n, out)
    pb.pi_matmul_i8(xq, xs, wq, sw, y, ws, bias=bias)
    assert pb.pi_get_device_status(ws) == 0
    check()
    main = (xq.to(D) @ wq.to(D).T) * xs.to(D)[:, None] * sw.to(D)
    want = main if bias is None else (main + bias.to(D)).to(F32).to(D)  # one fused rounding
    if out is F16:
        assert torch.equal(torch.isinf(y), want.abs() >= 65520)
        want = want.clamp(-65504, 65504)
        y = y.clamp(-65504, 65504)
    assert torch.equal(y, want.to(F32).to(out))


K16 = pytest.mark.parametrize("K", [8, 72, 136, 1000])  # 1, 2, 3 and 16 blocks of 64


@HALF
@K16
@pytest.mark.parametrize("mb,nt", dp.PAIR[dp.GLU])
def test_gate_and_up_on_pairs(cuda_device, plan, mb, nt, K, dtype):
    plan(dp.GLU, mb, nt, 0)
    _forward(700, K, 19000, dtype)


@HALF
@K16
@pytest.mark.parametrize("mb,nt", dp.PAIR[dp.STORE])
def test_outputs_on_pairs(cuda_device, plan, mb, nt, K, dtype):
    plan(dp.STORE, mb, nt, 0)
    _forward(700, 15368, K, dtype)
    _backward(700, 15368, K, dtype, only=("du",))


@HALF
@K16
@pytest.mark.parametrize("mb,nt", dp.PAIR[dp.DGLU])
def test_gradients_of_the_activation_on_pairs(cuda_device, plan, mb, nt, K, dtype):
    plan(dp.DGLU, mb, nt, 0)
    _backward(700, K, 19000, dtype)


@HALF
@pytest.mark.parametrize("T", [3, 100, 130, 1000])
@pytest.mark.parametrize("gtype,start", [("own", None), ("f32", None), ("own", 3.0), ("f32", -5.0)])
@pytest.mark.parametrize("mb,nt", dp.PAIR[dp.WEIGHT])
def test_gradients_of_the_weights(cuda_device, plan, mb, nt, gtype, start, T, dtype):
    plan(dp.WEIGHT, mb, nt, 0)
    _backward(T, 2568, 4104, dtype, F32 if gtype == "f32" else dtype, start)


@pytest.mark.parametrize("out", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,biased", [(19000, 16, False), (19001, 272, True), (19002, 528, True), (9003, 2064, False)])
@pytest.mark.parametrize("mb,nt", dp.PAIR[dp.I8])
def test_codes_on_pairs(cuda_device, plan, mb, nt, n, k, biased, out):
    plan(dp.I8, mb, nt, 0)
    _product(700, n, k, out, torch.arange(n, device="cuda", dtype=F32) - 99 if biased else None)


@pytest.mark.parametrize("nt,split", dp.SPLIT)
def test_split_products(cuda_device, plan, nt, split):
    """Three token tiles, the last of three tokens, over 40 to 80 feature tiles of 18 K blocks."""
    T = 2 * nt + 3
    for dtype in (F16, BF16):
        plan(dp.GLU, 1, nt, split)
        _forward(T, 1096, 5000, dtype)
        pb.pi_debug_dense_plan(-1)
        plan(dp.STORE, 1, nt, split)
        _forward(T, 5000, 1096, dtype)
        _backward(T, 5000, 1096, dtype, only=("du",))
        pb.pi_debug_dense_plan(-1)
        plan(dp.DGLU, 1, nt, split)
        _backward(T, 1096, 5000, dtype)
        pb.pi_debug_dense_plan(-1)
    plan(dp.I8, 1, nt, split)
    for out, n in ((F32, 5001), (F16, 5002), (BF16, 5004)):
        _product(T, n, 2064, out, torch.arange(n, device="cuda", dtype=F32))


def test_a_split_that_k_does_not_hold_is_refused(cuda_device, plan):
    plan(dp.I8, 1, 16, 8)
    e = lambda *s, dt: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    with pytest.raises(pb.PiError):
        pb.pi_matmul_i8(e(1, 1920, dt=torch.int8), e(1, dt=F32), e(16, 1920, dt=torch.int8), e(16, dt=F32),
                        e(1, 16, dt=F32), pb.make_matmul_i8_workspace(1, 16, 1920))


@HALF
@pytest.mark.parametrize("T,d,f", [(1, 3400, 25024), (1, 2968, 28672), (2, 5128, 16648), (1, 25024, 1032)])
def test_few_tokens_in_several_rounds(cuda_device, T, d, f, dtype):
    """By the rule: tile counts just over one round of the machine, widths that are no multiple of 64."""
    _forward(T, d, f, dtype)
    _backward(T, d, f, dtype)
