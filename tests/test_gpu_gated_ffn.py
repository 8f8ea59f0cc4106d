"""The gated feed-forward block and its gradients against plain fp64 forms.

Integer cases are exact: with small whole numbers every product and sum is
exact in fp32, so each stored value is the correctly rounded one and is
compared bit for bit, whatever the summation order.  Random cases use
tolerances that count the roundings (see ``_tol``).
"""
import pytest
import torch

import dense_ref as ref
from activation_sparse_decode_gemv_b200 import binding as pb

pytestmark = pytest.mark.gpu

D = torch.float64
TYPES = [torch.float16, torch.bfloat16]
# tokens x d x f: every tile width of both kernels, one past it, ragged rows and columns
SHAPES = [(1, 8, 8), (1, 520, 264), (2, 64, 128), (3, 72, 40), (16, 256, 512), (17, 264, 136), (32, 1000, 64),
          (33, 136, 1032), (64, 512, 384), (65, 776, 2056), (128, 128, 128), (129, 1032, 520), (200, 2056, 4104),
          (256, 512, 512), (300, 2568, 8), (513, 264, 2760), (1025, 72, 5128),
          (1500, 4104, 1032), (2000, 4104, 2056), (300, 520, 5128), (700, 2056, 4104),
          (430, 1544, 5128), (440, 5128, 2056), (380, 4104, 4104), (310, 2568, 5640), (620, 2056, 4616)]


def _ints(gen, *shape, lo, hi, dtype, keep=1.0):
    v = torch.randint(lo, hi + 1, shape, generator=gen, device="cuda")
    if keep < 1.0:
        v = v * (torch.rand(*shape, generator=gen, device="cuda") < keep)
    return v.to(dtype)


def _layer(wg, wu, wd, act, T, backward=False):
    layer = pb.GatedFfnLayer(wg, wu, wd, act=act)
    return layer, pb.make_gated_ffn_workspace(layer, T, backward)


def _guarded(rows, cols, dtype, fill=7.0):
    """A [rows, cols] output inside a buffer of known values, and a check that nothing around it changed."""
    pad = -(-cols // 8) * 8
    buf = torch.full((rows * cols + 2 * pad,), fill, dtype=dtype, device="cuda")
    out = buf[pad:pad + rows * cols].view(rows, cols)

    def check():
        assert torch.all(buf[:pad] == fill) and torch.all(buf[pad + rows * cols:] == fill), "written outside"
    return out, check


def _forward(layer, u, ws, keep=True):
    T, dt = u.shape[0], u.dtype
    y, cy = _guarded(T, layer.d, dt)
    g, cg = _guarded(T, layer.f, dt)
    p, cp = _guarded(T, layer.f, dt)
    pb.pi_gated_ffn_forward(layer, u, y, ws, **({"gate": g, "up": p} if keep else {}))
    assert pb.pi_get_device_status(ws) == 0
    cy(), cg(), cp()
    return y, g, p


def _int_case(T, d, f, dtype, seed=0):
    """Whole numbers small enough that g, p, a, dg, dp are exact in bf16 (|.| <= 256) and sums in fp32."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + T * 31 + d * 7 + f)
    sparse = min(1.0, 24.0 / d)  # about 24 nonzero products a sum: |g|, |p| stay near 5
    u = _ints(gen, T, d, lo=-1, hi=1, dtype=dtype)
    wg = _ints(gen, f, d, lo=-1, hi=1, dtype=dtype, keep=sparse)
    wu = _ints(gen, f, d, lo=-1, hi=1, dtype=dtype, keep=sparse)
    wd = _ints(gen, f, d, lo=-2, hi=2, dtype=dtype)
    dy = _ints(gen, T, d, lo=-1, hi=1, dtype=dtype, keep=sparse)
    return u, wg, wu, wd, dy


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("T,d,f", SHAPES)
def test_forward_is_exact_on_whole_numbers(cuda_device, T, d, f, dtype):
    u, wg, wu, wd, _ = _int_case(T, d, f, dtype)
    layer, ws = _layer(wg, wu, wd, "relu", T)
    y, g, p = _forward(layer, u, ws)
    yr, gr, pr, ar = ref.ffn_forward("relu", u.to(D), wg.to(D), wu.to(D), wd.to(D))
    assert gr.abs().max() <= 256 and ar.abs().max() <= 2048
    assert torch.equal(g.to(D), gr) and torch.equal(p.to(D), pr)
    # a is rounded to the layer's type on its way to the second product
    yr = ar.to(dtype).to(D) @ wd.to(D)
    assert torch.equal(y, yr.to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("T,d,f", SHAPES)
def test_backward_is_exact_on_whole_numbers(cuda_device, T, d, f, dtype):
    u, wg, wu, wd, dy = _int_case(T, d, f, dtype)
    layer, ws = _layer(wg, wu, wd, "relu", T, True)
    _, g, p, _ = ref.ffn_forward("relu", u.to(D), wg.to(D), wu.to(D), wd.to(D))
    g, p = g.to(dtype), p.to(dtype)
    du, c0 = _guarded(T, d, dtype)
    outs = [_guarded(f, d, dtype) for _ in range(3)]
    pb.pi_gated_ffn_backward(layer, u, g, p, dy, ws, du, *(o for o, _ in outs))
    assert pb.pi_get_device_status(ws) == 0
    c0()
    for _, c in outs:
        c()
    *_, dg, dp, a = ref.ffn_backward("relu", u.to(D), g.to(D), p.to(D), dy.to(D), wg.to(D), wu.to(D), wd.to(D))
    dg, dp, a = (t.to(dtype).to(D) for t in (dg, dp, a))
    expect = (dg @ wg.to(D) + dp @ wu.to(D), dg.T @ u.to(D), dp.T @ u.to(D), a.T @ dy.to(D))
    for name, got, want in zip(("du", "dw_gate", "dw_up", "dw_down_t"), (du, *(o for o, _ in outs)), expect):
        assert want.abs().max() < 2 ** 24, name
        assert torch.equal(got, want.to(dtype)), name


def _rand_case(T, d, f, dtype, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = lambda *s, std: (torch.randn(*s, generator=gen, device="cuda") * std).to(dtype)  # noqa: E731
    w = 1.5 / d ** 0.5
    return (n(T, d, std=1.0), n(f, d, std=w), n(f, d, std=w), n(f, d, std=w), n(T, d, std=0.5))


def _tol(A, B, dtype, rel_a):
    """Tolerance of (A @ B) rounded to dtype, A carrying independent relative errors up to rel_a.

    With S = sqrt(A^2 @ B^2), the size of the sum of its terms taken with
    independent signs:
    - rel_a: each term is off by at most rel_a |a b|, independently, so the
      sum is off by less than 7 rel_a S (7 standard deviations, were every
      error at its bound);
    - the fp32 accumulation rounds K partial sums of size about S to 2^-23
      relative at worst (the tensor core may truncate): K 2^-23 S;
    - the result is rounded once: half a step."""
    K = A.shape[1]
    S = torch.sqrt((A * A) @ (B * B))
    return (7 * rel_a + K * 2.0 ** -23) * S + ref.step(dtype) * (A @ B).abs()


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("T,d,f", [(1, 264, 1032), (40, 512, 1000), (130, 1032, 2048), (700, 520, 1544)])
def test_forward_and_backward_on_random_values(cuda_device, T, d, f, act, dtype):
    u, wg, wu, wd, dy = _rand_case(T, d, f, dtype, T + d)
    h = ref.step(dtype)
    layer, ws = _layer(wg, wu, wd, act, T, True)
    y, g, p = _forward(layer, u, ws)
    u6, wg6, wu6, wd6, dy6 = (t.to(D) for t in (u, wg, wu, wd, dy))
    yr, gr, pr, ar = ref.ffn_forward(act, u6, wg6, wu6, wd6)
    assert torch.all((g.to(D) - gr).abs() <= _tol(u6, wg6.T, dtype, 0.0))
    assert torch.all((p.to(D) - pr).abs() <= _tol(u6, wu6.T, dtype, 0.0))
    # a is off by its rounding (h) and by g's and p's fp32 errors, which are far below h
    assert torch.all((y.to(D) - yr).abs() <= _tol(ar, wd6, dtype, 1.05 * h))
    # without the kept outputs the result is the same
    y2, _, _ = _forward(layer, u, ws, keep=False)
    assert torch.equal(y, y2)

    du = torch.empty_like(u)
    dw = [torch.empty_like(wg) for _ in range(3)]
    pb.pi_gated_ffn_backward(layer, u, g, p, dy, ws, du, *dw)
    assert pb.pi_get_device_status(ws) == 0
    want = ref.ffn_backward(act, u6, g.to(D), p.to(D), dy6, wg6, wu6, wd6)
    dg, dp, a = want[4:]
    # dg, dp, a: one rounding each; near phi' = 0 dg's error is relative to da p, below 2^-20 of it
    eps_a = 1.05 * h
    assert torch.all((du.to(D) - want[0]).abs()
                     <= _tol(torch.cat([dg, dp], 1), torch.cat([wg6, wu6]), dtype, eps_a) + 2.0 ** -20)
    for got, w, left, right in ((dw[0], want[1], dg, u6), (dw[1], want[2], dp, u6), (dw[2], want[3], a, dy6)):
        assert torch.all((got.to(D) - w).abs() <= _tol(left.T.contiguous(), right, dtype, eps_a) + 2.0 ** -20)


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
def test_gradients_agree_with_differences(cuda_device, dtype):
    """<gradient, v> against (L(+e v) - L(-e v)) / 2e of the fp64 forward pass, L = <y, dy>."""
    T, d, f, act = 37, 136, 200, "silu"
    u, wg, wu, wd, dy = _rand_case(T, d, f, dtype, 5)
    layer, ws = _layer(wg, wu, wd, act, T, True)
    _, g, p = _forward(layer, u, ws)
    du, dw = torch.empty_like(u), [torch.empty_like(wg) for _ in range(3)]
    pb.pi_gated_ffn_backward(layer, u, g, p, dy, ws, du, *dw)
    base = [t.to(D) for t in (u, wg, wu, wd)]
    loss = lambda ts: (ref.ffn_forward(act, *ts)[0] * dy.to(D)).sum()  # noqa: E731
    e, gen = 1e-5, torch.Generator(device="cuda").manual_seed(3)
    for k, grad in enumerate((du, *dw)):
        v = torch.randn(base[k].shape, generator=gen, device="cuda", dtype=D)
        plus, minus = ([b + s * e * v if i == k else b for i, b in enumerate(base)] for s in (1, -1))
        diff = (loss(plus) - loss(minus)) / (2 * e)
        got = (grad.to(D) * v).sum()
        # g, p (relative h each, through dg), dg or dp or a, and the gradient itself are rounded: at most
        # 4 independent relative errors h per element of a sum with random signs, 7 deviations
        size = torch.sqrt((grad.to(D) ** 2 * v ** 2).sum())
        assert (got - diff).abs() <= 7 * 4 * ref.step(dtype) * size + 1e-6 * diff.abs(), k


@pytest.mark.parametrize("gtype", ["own", "f32"])
def test_gradients_accumulate_and_may_be_left_out(cuda_device, gtype):
    T, d, f, dtype = 129, 136, 264, torch.bfloat16
    u, wg, wu, wd, dy = _int_case(T, d, f, dtype)
    layer, ws = _layer(wg, wu, wd, "relu", T, True)
    _, g, p, _ = ref.ffn_forward("relu", u.to(D), wg.to(D), wu.to(D), wd.to(D))
    g, p = g.to(dtype), p.to(dtype)
    gt = dtype if gtype == "own" else torch.float32
    dw = [torch.empty(f, d, dtype=gt, device="cuda") for _ in range(3)]
    du = torch.empty_like(u)
    pb.pi_gated_ffn_backward(layer, u, g, p, dy, ws, du, *dw)
    first = [t.clone() for t in dw]
    for k, name in enumerate(("dw_gate", "dw_up", "dw_down_t")):  # each alone, added to a known value
        out = torch.full((f, d), 3.0, dtype=gt, device="cuda")
        pb.pi_gated_ffn_backward(layer, u, g, p, dy, ws, **{name: out}, flags=pb.PI_GRAD_ACCUMULATE)
        *_, dg, dp, a = ref.ffn_backward("relu", u.to(D), g.to(D), p.to(D), dy.to(D), wg.to(D), wu.to(D), wd.to(D))
        left = (dg, dp, a)[k].to(dtype).to(D)
        right = (u, u, dy)[k].to(D)
        assert torch.equal(out, (left.T @ right + 3.0).to(gt)), name
    du2 = torch.empty_like(u)
    pb.pi_gated_ffn_backward(layer, u, g, p, dy, ws, du=du2)
    assert torch.equal(du, du2)
    assert all(torch.equal(a, b) for a, b in zip(first, dw))
    pb.pi_gated_ffn_backward(layer, u, g, p, dy, ws)  # nothing wanted
    assert pb.pi_get_device_status(ws) == 0


def test_no_tokens(cuda_device):
    wg = torch.ones(64, 32, dtype=torch.float16, device="cuda")
    layer, ws = _layer(wg, wg, wg, "silu", 0, True)
    u, g = wg.new_empty(0, 32), wg.new_empty(0, 64)
    pb.pi_gated_ffn_forward(layer, u, wg.new_empty(0, 32), ws)
    dw = [torch.full_like(wg, 5.0) for _ in range(3)]
    pb.pi_gated_ffn_backward(layer, u, g, g, u, ws, u, *dw, flags=pb.PI_GRAD_ACCUMULATE)
    assert all(torch.all(t == 5.0) for t in dw)
    pb.pi_gated_ffn_backward(layer, u, g, g, u, ws, u, *dw)
    assert all(torch.all(t == 0.0) for t in dw)


@pytest.mark.parametrize("T", [3, 100, 600])
def test_non_finite_tokens_stay_in_their_rows(cuda_device, T):
    d, f, dtype = 264, 520, torch.float16
    u, wg, wu, wd, dy = _rand_case(T, d, f, dtype, 11)
    layer, ws = _layer(wg, wu, wd, "silu", T, True)
    clean, _, _ = _forward(layer, u, ws)
    bad = u.clone()
    bad[1, 5], bad[T - 1, 7] = float("nan"), float("inf")
    y, _, _ = _forward(layer, bad, ws)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[1] = keep[T - 1] = False
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[T - 1]).any()


@pytest.mark.parametrize("T", [1, 300])
def test_captured_and_replayed_and_on_another_stream(cuda_device, T):
    d, f, dtype = 520, 1032, torch.bfloat16
    u, wg, wu, wd, dy = _rand_case(T, d, f, dtype, 21)
    layer, ws = _layer(wg, wu, wd, "silu", T, True)
    y, g, p = (torch.empty(T, n, dtype=dtype, device="cuda") for n in (d, f, f))
    du, dw = torch.empty_like(u), [torch.empty_like(wg) for _ in range(3)]

    def step_():
        pb.pi_gated_ffn_forward(layer, u, y, ws, gate=g, up=p)
        pb.pi_gated_ffn_backward(layer, u, g, p, dy, ws, du, *dw)
    step_()
    want = [t.clone() for t in (y, g, p, du, *dw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in (y, g, p, du, *dw):
            t.zero_()
        step_()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y, g, p, du, *dw)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_()
    u2 = _rand_case(T, d, f, dtype, 22)[0]
    u.copy_(u2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, g, p, du, *dw)]
    step_()
    assert all(torch.equal(a, b) for a, b in zip(got, (y, g, p, du, *dw)))
    assert pb.pi_get_device_status(ws) == 0


def test_weights_changed_in_place_are_seen(cuda_device):
    T, d, f, dtype = 20, 136, 264, torch.float16
    u, wg, wu, wd, _ = _rand_case(T, d, f, dtype, 31)
    layer, ws = _layer(wg, wu, wd, "silu", T)
    _forward(layer, u, ws)
    for w in (wg, wu, wd):
        w.mul_(0.5)
    y, _, _ = _forward(layer, u, ws)
    fresh, ws2 = _layer(wg.clone(), wu.clone(), wd.clone(), "silu", T)
    assert torch.equal(y, _forward(fresh, u, ws2)[0])


def test_offsets_past_32_bits(cuda_device):
    """More than 2^31 activations: the last rows are the rows of a call on those tokens alone."""
    T, d, f, dtype = 70_000, 8, 32_776, torch.float16
    assert T * f > 2 ** 31
    u, wg, wu, wd, dy = _int_case(T, d, f, dtype)
    wd = (wd * (torch.arange(f, device="cuda") % 64 == 0)[:, None]).to(dtype)  # y stays in range
    layer, ws = _layer(wg, wu, wd, "relu", T, True)
    y, g, p = (torch.empty(T, n, dtype=dtype, device="cuda") for n in (d, f, f))
    pb.pi_gated_ffn_forward(layer, u, y, ws, gate=g, up=p)
    du = torch.empty_like(u)
    pb.pi_gated_ffn_backward(layer, u, g, p, dy, ws, du=du)
    assert pb.pi_get_device_status(ws) == 0
    for rows in (slice(0, 300), slice(T - 300, T)):
        u6, dy6 = u[rows].to(D), dy[rows].to(D)
        yr, gr, pr, ar = ref.ffn_forward("relu", u6, wg.to(D), wu.to(D), wd.to(D))
        assert torch.equal(g[rows].to(D), gr) and torch.equal(p[rows].to(D), pr)
        assert torch.equal(y[rows], yr.to(dtype))
        *_, dg, dp, _ = ref.ffn_backward("relu", u6, gr, pr, dy6, wg.to(D), wu.to(D), wd.to(D))
        assert torch.equal(du[rows], (dg @ wg.to(D) + dp @ wu.to(D)).to(dtype))


CAPTURE_FIRST = """
import torch
from activation_sparse_decode_gemv_b200 import binding as pb
T, d, f = %d, 264, 1032
g = torch.Generator(device="cuda").manual_seed(0)
w = [(torch.randn(f, d, generator=g, device="cuda") * 0.05).half() for _ in range(3)]
layer = pb.GatedFfnLayer(*w)
ws = pb.make_gated_ffn_workspace(layer, T, True)
u = torch.randn(T, d, generator=g, device="cuda").half()
y, gp, up = torch.empty_like(u), u.new_empty(T, f), u.new_empty(T, f)
du, dw = torch.empty_like(u), [torch.empty_like(w[0]) for _ in range(3)]
n = pb.BlockNorm(d, y_dtype=torch.float16, u_dtype=torch.float16, post_norm=True)
x, r, kp, kr = torch.randn(T, d, generator=g, device="cuda"), u.new_empty(T, d).float(), u.new_empty(T).float(), u.new_empty(T).float()
nws, dx, dwp = pb.make_block_norm_workspace(n, T), torch.empty(T, d, device="cuda"), torch.empty(d, device="cuda")
q, s, wq, wsc = u.new_empty(T, 256).to(torch.int8), kp.clone(), torch.ones(96, 256, dtype=torch.int8, device="cuda"), torch.ones(96, device="cuda")
z, xi = torch.empty(T, 96, device="cuda"), torch.randn(T, 256, generator=g, device="cuda")
iws = pb.make_matmul_i8_workspace(T, 96, 256)
torch.cuda.synchronize()
def step():
    pb.pi_gated_ffn_forward(layer, u, y, ws, gate=gp, up=up)
    pb.pi_block_norm_forward(n, x, y, r, None, rstd_post=kp)
    pb.pi_block_norm_backward(n, None, y, kp, None, None, x, dx, None, nws, dw_post=dwp)
    pb.pi_gated_ffn_backward(layer, u, gp, up, y, ws, du, *dw)
    pb.pi_quantize_i8(xi, q, s)
    pb.pi_matmul_i8(q, s, wq, wsc, z, iws)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (y, r, dx, dwp, du, *dw, z)]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (y, r, dx, dwp, du, *dw, z)))
assert pb.pi_get_device_status(ws) == 0 and pb.pi_get_device_status(iws) == 0
print("captured first")
"""


@pytest.mark.parametrize("T", [3, 400])
def test_first_calls_of_a_process_may_be_captured(cuda_device, T):
    """Nothing that a first call sets up needs a call outside of a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", CAPTURE_FIRST % T], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "captured first" in out.stdout, out.stderr[-2000:]


def test_one_of_the_kept_outputs_alone(cuda_device):
    for T in (5, 300):
        u, wg, wu, wd, _ = _rand_case(T, 264, 520, torch.float16, 41)
        layer, ws = _layer(wg, wu, wd, "silu", T)
        y, g, p = _forward(layer, u, ws)
        for k, want in (("gate", g), ("up", p)):
            y2, out = torch.empty_like(y), torch.empty_like(want)
            pb.pi_gated_ffn_forward(layer, u, y2, ws, **{k: out})
            assert torch.equal(out, want) and torch.equal(y, y2)


def test_two_streams_at_once(cuda_device):
    """Calls on two streams with a workspace each, large and small, forward and backward."""
    jobs = []
    for k, (T, d, f) in enumerate([(300, 1032, 2056), (2, 2056, 4104)]):
        u, wg, wu, wd, dy = _rand_case(T, d, f, torch.bfloat16, 50 + k)
        layer, ws = _layer(wg, wu, wd, "silu", T, True)
        o = [torch.empty(T, n, dtype=torch.bfloat16, device="cuda") for n in (d, f, f, d)]
        dw = [torch.empty_like(wg) for _ in range(3)]

        def job(layer=layer, ws=ws, u=u, dy=dy, o=o, dw=dw):
            pb.pi_gated_ffn_forward(layer, u, o[0], ws, gate=o[1], up=o[2])
            pb.pi_gated_ffn_backward(layer, u, o[1], o[2], dy, ws, o[3], *dw)
        job()
        jobs.append((job, o + dw, [t.clone() for t in o + dw]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _, outs, _ in jobs:
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for (job, _, _), st in zip(jobs, streams):
            with torch.cuda.stream(st):
                job()
    torch.cuda.synchronize()
    for _, outs, want in jobs:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
