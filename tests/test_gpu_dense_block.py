"""The dense block operators used together: a feed-forward block of a decoder,
pre-norm -> gated FFN -> post-norm, gate and residual -> next pre-norm, forward
and backward, against the same computation in fp64; the same block served with
8-bit weights; and a prompt that is handed over to the sparse decode path."""
import pytest
import torch

import dense_ref as ref
from activation_sparse_decode_gemv_b200 import binding as pb

pytestmark = pytest.mark.gpu

D, F32 = torch.float64, torch.float32
E = 2.0 ** -24


def _block(T, d, f, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    w = [n(f, d, std=1.5 / d ** 0.5).to(dtype), n(f, d, std=1.5 / d ** 0.5).to(dtype), n(f, d, std=f ** -0.5).to(dtype)]
    return {"x": n(T, d, std=1.0), "w": w, "w0": 1 + n(d, std=0.1), "w_post": 1 + n(d, std=0.1),
            "w1": 1 + n(d, std=0.1), "gate": n(-(-T // 50), d, std=0.3), "du": n(T, d, std=0.3).to(dtype),
            "dx": n(T, d, std=0.2)}


def _run(b, T, d, f, dtype, act):
    e = lambda *s, dt=dtype: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    n0 = pb.BlockNorm(d, u_dtype=dtype, y_dtype=dtype, w_pre=b["w0"])
    n1 = pb.BlockNorm(d, u_dtype=dtype, y_dtype=dtype, post_norm=True, w_post=b["w_post"], w_pre=b["w1"],
                      gate=b["gate"], tokens_per_gate=50, branch_scale=0.5)
    layer = pb.GatedFfnLayer(*b["w"], act=act)
    ws = pb.make_gated_ffn_workspace(layer, T, True)
    nws = pb.make_block_norm_workspace(n1, T)
    u, y, gp, up, k0 = e(T, d), e(T, d), e(T, f), e(T, f), e(T, dt=F32)
    x1, u1, kp, kr = e(T, d, dt=F32), e(T, d), e(T, dt=F32), e(T, dt=F32)
    pb.pi_block_norm_forward(n0, b["x"], None, None, u, rstd_pre=k0)
    pb.pi_gated_ffn_forward(layer, u, y, ws, gate=gp, up=up)
    pb.pi_block_norm_forward(n1, b["x"], y, x1, u1, rstd_post=kp, rstd_pre=kr)
    # backward
    dx, dy, du0 = e(T, d, dt=F32), e(T, d), e(T, d)
    dw = [e(f, d, dt=F32) for _ in range(3)]
    dn = {"dw_post": e(d, dt=F32), "dw_pre": e(d, dt=F32), "dgate": torch.empty_like(b["gate"])}
    dw0 = e(d, dt=F32)
    pb.pi_block_norm_backward(n1, x1, y, kp, kr, b["du"], b["dx"], dx, dy, nws, **dn)
    pb.pi_gated_ffn_backward(layer, u, gp, up, dy, ws, du0, *dw)
    pb.pi_block_norm_backward(n0, b["x"], None, None, k0, du0, dx, dx, None, nws, dw_pre=dw0)
    assert pb.pi_get_device_status(ws) == 0
    return {"x1": x1, "u1": u1, "dx": dx, "dw_gate": dw[0], "dw_up": dw[1], "dw_down": dw[2], "dw0": dw0, **dn}


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T,d,f,act", [(1, 264, 520, "silu"), (133, 520, 1544, "silu"), (700, 1032, 2056, "gelu")])
def test_training_step_of_a_block(cuda_device, T, d, f, act, dtype):
    b = _block(T, d, f, dtype, T)
    got = _run(b, T, d, f, dtype, act)
    # the same in fp64, by automatic differentiation
    p = {k: b[k].to(D).requires_grad_() for k in ("x", "w0", "w_post", "w1", "gate")}
    w = [t.to(D).requires_grad_() for t in b["w"]]
    eps = float(torch.tensor(1e-6, dtype=F32))
    _, u, _, _ = ref.norm_forward(p["x"], None, eps=eps, w_pre=p["w0"])
    y, *_ = ref.ffn_forward(act, u, *w)
    x1, u1, _, _ = ref.norm_forward(p["x"], y, eps=eps, beta=0.5, post_norm=True, w_post=p["w_post"], w_pre=p["w1"],
                                    gate=p["gate"], per=50)
    grads = torch.autograd.grad((u1 * b["du"].to(D)).sum() + (x1 * b["dx"].to(D)).sum(),
                                [p["x"], *w, p["w0"], p["w_post"], p["w1"], p["gate"]])
    want = dict(zip(("dx", "dw_gate", "dw_up", "dw_down", "dw0", "dw_post", "dw_pre", "dgate"), grads))
    want.update(x1=x1, u1=u1)
    # Each rounding to the 16-bit type is a relative error of at most h, independent from element to element. On
    # the way forward u, g, p, a, y and u1 are rounded (6), on the way back dy, dg, dp, a and du (5), and the inputs
    # of a product carry the errors before them: the 2-norm error is below h sqrt(11) times the amplification of
    # one stage by the next, which the norms and the gate keep below 2 (phi' <= 1.13, post-norm of unit gain).
    h = ref.step(dtype)
    for k, v in got.items():
        rel = ((v.to(D) - want[k]).norm() / want[k].norm()).item()
        assert rel <= 2 * 11 ** 0.5 * h, (k, rel / h)
    # bit for bit the same again
    again = _run(b, T, d, f, dtype, act)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("T", [1, 90])
def test_block_served_in_8_bits(cuda_device, T):
    """norm -> codes -> gate and up products -> codes -> down product -> residual, near the fp16 block."""
    d, f = 512, 1552
    b = _block(T, d, f, torch.float16, 7)
    e = lambda *s, dt: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    q = [(e(f, d, dt=torch.int8), e(f, dt=F32)) for _ in range(2)] + [(e(d, f, dt=torch.int8), e(d, dt=F32))]
    for (c, s), wt in zip(q, (b["w"][0], b["w"][1], b["w"][2].t().contiguous())):
        pb.pi_quantize_i8(wt, c, s)
    n0 = pb.BlockNorm(d, u_dtype=torch.float16, w_pre=b["w0"])
    u, uc, us = e(T, d, dt=torch.float16), e(T, d, dt=torch.int8), e(T, dt=F32)
    g, p, y, ac, asc = e(T, f, dt=F32), e(T, f, dt=F32), e(T, d, dt=F32), e(T, f, dt=torch.int8), e(T, dt=F32)
    w1, w2 = pb.make_matmul_i8_workspace(T, f, d), pb.make_matmul_i8_workspace(T, d, f)
    pb.pi_block_norm_forward(n0, b["x"], None, None, u)
    pb.pi_quantize_i8(u, uc, us)
    pb.pi_matmul_i8(uc, us, *q[0], g, w1)
    pb.pi_matmul_i8(uc, us, *q[1], p, w1)
    a = (torch.nn.functional.silu(g) * p).contiguous()
    pb.pi_quantize_i8(a, ac, asc)
    pb.pi_matmul_i8(ac, asc, *q[2], y, w2)
    x1 = e(T, d, dt=F32)
    pb.pi_block_norm_forward(pb.BlockNorm(d, y_dtype=F32), b["x"], y, x1, None)
    want, *_ = ref.ffn_forward("silu", u.to(D), *(t.to(D) for t in b["w"]))
    # A code is off by at most half a step s = amax / 127, uniformly: s / sqrt 12 in the 2-norm per element. With
    # amax below 5 (u, w) and 12 (a, heavier tails) deviations, each quantised operand is off by amax / (127 sqrt 12)
    # = 1.1 to 2.7% of its norm: u and w (g and p, each 1.6%, through phi' and the product 2 x 1.6%), then a 2.7%, w2 1.1%
    rel = ((y.to(D) - want).norm() / want.norm()).item()
    assert rel <= (2 * 0.016 ** 2 * 4 + 0.027 ** 2 + 0.011 ** 2) ** 0.5, rel
    assert torch.equal(x1, b["x"] + y)


def test_dense_forward_agrees_with_the_sparse_path_over_all_neurons(cuda_device):
    """The prompt pass and the decode pass of one SwiGLU layer are the same function: with every neuron in the
    sets, pi_sparse_ffn and pi_gated_ffn_forward differ by their roundings only."""
    d, f, r, B = 512, 1024, 64, 4
    dt = torch.float16
    b = _block(B, d, f, dt, 3)
    wg, wu, wd = b["w"]
    p1, p2 = torch.zeros(r, d, dtype=dt, device="cuda"), torch.zeros(f, r, dtype=dt, device="cuda")
    sparse = pb.FfnLayer(wu, wd, p1, p2, torch.ones(f, device="cuda"), act="swiglu", wtype="f16", d=d, f=f, r=r, w_gate=wg)
    ws = pb.make_workspace([sparse], B)
    u = torch.randn(B, d, device="cuda").to(dt)
    idx = torch.arange(f, dtype=torch.int32, device="cuda").repeat(B, 1).contiguous()
    cnt = torch.full((B,), f, dtype=torch.int32, device="cuda")
    ys = torch.empty(B, d, device="cuda")
    pb.pi_sparse_ffn(sparse, u, idx, cnt, ys, ws)
    dense = pb.GatedFfnLayer(wg, wu, wd)
    yd = torch.empty(B, d, dtype=dt, device="cuda")
    pb.pi_gated_ffn_forward(dense, u, yd, pb.make_gated_ffn_workspace(dense, B))
    _, _, _, a = ref.ffn_forward("silu", u.to(D), wg.to(D), wu.to(D), wd.to(D))
    S = torch.sqrt((a * a) @ (wd.to(D) ** 2))
    h = ref.step(dt)  # a is rounded once in each path, y in the dense one
    assert torch.all((yd.to(D) - ys.to(D)).abs() <= 2 * 7 * h * S + h * ys.to(D).abs() + 1e-5 * S)
