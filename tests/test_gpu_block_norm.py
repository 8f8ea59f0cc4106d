"""The norms around a block and their gradients against plain fp64 forms.

E = 2^-24 is half an fp32 step.  A block sum of d values adds at most 42
roundings (32 in a thread, 5 + 5 in the shuffles), so a mean of squares is off
by 42 E relative and its inverse root by 21 E + 4 E (rsqrtf, 2 ulp); 40 E
covers it with the products around it.
"""
import pytest
import torch

import dense_ref as ref
from activation_sparse_decode_gemv_b200 import binding as pb

pytestmark = pytest.mark.gpu

D = torch.float64
E = 2.0 ** -24
EPS = 1e-6
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _case(T, d, yt, ut, post, per, seed=0, weights=True):
    gen = torch.Generator(device="cuda").manual_seed(seed + 13 * T + d)
    n = lambda *s, std=1.0, dtype=F32: (torch.randn(*s, generator=gen, device="cuda") * std).to(dtype)  # noqa: E731
    c = {"x": n(T, d, std=3.0), "y": n(T, d, std=0.5, dtype=yt), "du": n(T, d, std=0.3, dtype=ut),
         "dx_out": n(T, d, std=0.2), "w_pre": 1 + n(d, std=0.1) if weights else None,
         "w_post": 1 + n(d, std=0.1) if weights and post else None,
         "gate": n(-(-T // per), d, std=0.5) if per else None, "alpha": 0.9, "beta": 0.7, "post": post, "per": per}
    c["norm"] = pb.BlockNorm(d, y_dtype=yt, u_dtype=ut, eps=EPS, residual_scale=c["alpha"], branch_scale=c["beta"],
                             post_norm=post, w_post=c["w_post"], w_pre=c["w_pre"], gate=c["gate"],
                             tokens_per_gate=per)
    return c


def _d(t):
    return None if t is None else t.to(D)


def _scales(c):
    """The scales as the library holds them (fp32)."""
    return {k: float(torch.tensor(c[k], dtype=F32)) for k in ("alpha", "beta")}, float(torch.tensor(EPS, dtype=F32))


def _reference(c, x=None, y=None, gate=None, w_post=None, w_pre=None):
    s, eps = _scales(c)
    pick = lambda a, k: a if a is not None else _d(c[k])  # noqa: E731
    return ref.norm_forward(pick(x, "x"), pick(y, "y"), eps=eps, **s, post_norm=c["post"],
                            w_post=pick(w_post, "w_post"), w_pre=pick(w_pre, "w_pre"), gate=pick(gate, "gate"),
                            per=c["per"])


SHAPES = [(1, 8), (1, 8192), (2, 64), (5, 128), (37, 1000), (300, 136), (130, 2048), (64, 2056), (9, 5120), (7, 7168),
          (3, 16384), (1000, 24),
          (5, 8200), (200, 12288), (700, 512), (2100, 72), (150, 6152)]
KINDS = [(F32, F16, False, 0), (F16, F16, True, 0), (BF16, BF16, True, 1), (F32, F32, True, 7), (BF16, F16, False, 3)]


@pytest.mark.parametrize("yt,ut,post,per", KINDS, ids=["f32-f16", "f16-post", "bf16-gate1", "f32-gate7", "mixed"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward(cuda_device, T, d, yt, ut, post, per):
    c = _case(T, d, yt, ut, post, per)
    r, u = torch.empty(T, d, device="cuda"), torch.empty(T, d, dtype=ut, device="cuda")
    kp = torch.empty(T, device="cuda") if post else None
    kr = torch.empty(T, device="cuda")
    pb.pi_block_norm_forward(c["norm"], c["x"], c["y"], r, u, kp, kr)
    rr, ur, kpr, krr = _reference(c)
    s, _ = _scales(c)
    branch = rr - s["alpha"] * c["x"].to(D)
    tol_r = E * (2 * s["alpha"] * c["x"].to(D).abs() + 40 * branch.abs() + rr.abs())
    assert torch.all((r.to(D) - rr).abs() <= tol_r)
    slope = krr[:, None] * (_d(c["w_pre"]).abs() if c["w_pre"] is not None else 1)
    tol_u = ref.step(ut) * ur.abs() + slope * tol_r + 45 * E * ur.abs()
    if ut is F16:
        tol_u = tol_u + 2.0 ** -25  # half a step of fp16's subnormals
    assert torch.all((u.to(D) - ur).abs() <= tol_u)
    assert torch.all((kr.to(D) - krr).abs() <= 45 * E * krr)
    if post:
        assert torch.all((kp.to(D) - kpr).abs() <= 40 * E * kpr)
    # in place, and each output alone: the same values
    x2 = c["x"].clone()
    pb.pi_block_norm_forward(c["norm"], x2, c["y"], x2, None)
    assert torch.equal(x2, r)
    u2 = torch.empty_like(u)
    pb.pi_block_norm_forward(c["norm"], c["x"], c["y"], None, u2)
    assert torch.equal(u2, u)


def test_forward_without_a_branch_and_without_weights(cuda_device):
    c = _case(11, 264, F16, F16, False, 0, weights=False)
    r, u = torch.empty(11, 264, device="cuda"), torch.empty(11, 264, dtype=F16, device="cuda")
    pb.pi_block_norm_forward(c["norm"], c["x"], None, r, u)
    assert torch.equal(r, torch.tensor(0.9, device="cuda") * c["x"])
    s, eps = _scales(c)
    _, ur, _, _ = ref.norm_forward(c["x"].to(D), None, eps=eps, alpha=s["alpha"])
    assert torch.all((u.to(D) - ur).abs() <= (ref.step(F16) + 50 * E) * ur.abs() + 2.0 ** -25)


def test_decode_step_matches_the_stack_norm(cuda_device):
    """Unit scales and no weights give u = x / sqrt(mean x^2 + eps), the stack's pre-FFN norm, to one fp16 step."""
    x = torch.randn(4, 512, device="cuda")
    y = torch.randn(4, 512, device="cuda")
    n = pb.BlockNorm(512, y_dtype=F32, u_dtype=F16)
    u, r = torch.empty(4, 512, dtype=F16, device="cuda"), torch.empty_like(x)
    pb.pi_block_norm_forward(n, x, y, r, u)
    assert torch.equal(r, x + y)
    want = r / torch.sqrt((r.to(D) ** 2).mean(1, keepdim=True).float() + 1e-6)
    assert torch.all((u.float() - want).abs() <= 1.01 * ref.step(F16) * want.abs() + 2.0 ** -25)


def _grads(c):
    """fp64 gradients by autograd of the plain forward, at the stored stream: the backward call is given r and y."""
    x, y = (_d(c[k]).requires_grad_() for k in ("x", "y"))
    par = {k: _d(c[k]).requires_grad_() for k in ("gate", "w_post", "w_pre") if c[k] is not None}
    r, u, kp, kr = _reference(c, x, y, **par)
    return x, y, par, r, u, kp, kr


def _run_backward(c, T, d, rstd_post, rstd_pre, r, **kw):
    out = {"dx": torch.empty(T, d, device="cuda"), "dy": torch.empty_like(c["y"]),
           "dw_post": torch.empty(d, device="cuda") if c["post"] else None,
           "dw_pre": torch.empty(d, device="cuda"),
           "dgate": None if c["gate"] is None else torch.empty_like(c["gate"])}
    ws = pb.make_block_norm_workspace(c["norm"], T)
    pb.pi_block_norm_backward(c["norm"], r, c["y"], rstd_post, rstd_pre, c["du"], c["dx_out"], out["dx"], out["dy"],
                              ws, out["dw_post"], out["dw_pre"], out["dgate"], **kw)
    return out


@pytest.mark.parametrize("yt,ut,post,per", KINDS, ids=["f32-f16", "f16-post", "bf16-gate1", "f32-gate7", "mixed"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_backward(cuda_device, T, d, yt, ut, post, per):
    c = _case(T, d, yt, ut, post, per, seed=1)
    s, eps = _scales(c)
    # the forward pass's outputs, as the library stores them
    r, u = torch.empty(T, d, device="cuda"), torch.empty(T, d, dtype=ut, device="cuda")
    kp = torch.empty(T, device="cuda") if post else None
    kr = torch.empty(T, device="cuda")
    pb.pi_block_norm_forward(c["norm"], c["x"], c["y"], r, u, kp, kr)
    out = _run_backward(c, T, d, kp, kr, r)
    # plain formulas in fp64 at the stored r, y, kp, kr
    R, y, du, g0 = r.to(D), c["y"].to(D), c["du"].to(D), c["dx_out"].to(D)
    k = kr.to(D)[:, None]
    w = _d(c["w_pre"])
    wp = _d(c["w_post"]) if c["w_post"] is not None else torch.ones(d, dtype=D, device="cuda")
    rows = torch.arange(T, device="cuda") // per if per else None
    gate = _d(c["gate"])[rows] if per else torch.ones(1, d, dtype=D, device="cuda")
    n, v = R * k, du * w
    cc = (v * n).sum(1, keepdim=True)
    dr = g0 + k * (v - n * cc / d)
    m = y * (kp.to(D)[:, None] if post else 1)
    db = s["beta"] * dr * gate
    q = s["beta"] * gate * wp * m
    e = (db * wp * m).sum(1, keepdim=True)
    dy = kp.to(D)[:, None] * (db * wp - m * e / d) if post else db
    # tolerances: roundings of each term, 50 E for a block sum over the sum of its terms' sizes
    d_cd = k / d * 50 * E * (v * n).abs().sum(1, keepdim=True)
    tol_dr = E * (3 * g0.abs() + 6 * (k * v).abs() + 6 * (k * cc / d * n).abs() + 2 * dr.abs()) + n.abs() * d_cd
    assert torch.all((out["dx"].to(D) - s["alpha"] * dr).abs() <= s["alpha"] * (tol_dr + E * dr.abs())), "dx"
    lead = s["beta"] * (gate * wp).abs()
    if post:
        cd = (k * cc / d).abs()
        d_e = (50 * E * (q.abs() * (g0.abs() + (k * v).abs())).sum(1, keepdim=True)
               + cd * 50 * E * (q * n).abs().sum(1, keepdim=True)
               + d_cd * (q * n).sum(1, keepdim=True).abs() + 4 * E * e.abs()) / d
        tol_dy = kp.to(D)[:, None] * (lead * tol_dr + 6 * E * (db * wp).abs() + m.abs() * d_e
                                      + 6 * E * (m * e / d).abs())
    else:
        tol_dy = lead * tol_dr + 4 * E * db.abs()
    tol_dy = tol_dy + ref.step(yt) * dy.abs() + (2.0 ** -25 if yt is F16 else 0.0)
    assert torch.all((out["dy"].to(D) - dy).abs() <= tol_dy), "dy"
    # column sums: T terms, each partial sum rounded
    adds = (T + 20) * E
    t = du * n
    assert torch.all((out["dw_pre"].to(D) - t.sum(0)).abs() <= (adds + 3 * E) * t.abs().sum(0)), "dw_pre"
    if post:
        t = db * m
        tol = (adds * t.abs() + (s["beta"] * gate * m).abs() * tol_dr + 5 * E * t.abs()).sum(0)
        assert torch.all((out["dw_post"].to(D) - t.sum(0)).abs() <= tol), "dw_post"
    if per:
        t = s["beta"] * dr * wp * m
        tol = adds * t.abs() + (s["beta"] * wp * m).abs() * tol_dr + 5 * E * t.abs()
        z = torch.zeros_like(_d(c["gate"]))
        want, bound = z.index_add(0, rows, t), z.index_add(0, rows, tol)
        assert torch.all((out["dgate"].to(D) - want).abs() <= bound), "dgate"
    # the same again: bit for bit; added to known values; in place
    again = _run_backward(c, T, d, kp, kr, r)
    assert all(torch.equal(out[x], again[x]) for x in out if out[x] is not None)
    ws = pb.make_block_norm_workspace(c["norm"], T)
    acc = {x: torch.full_like(out[x], 2.0) for x in ("dw_post", "dw_pre", "dgate") if out[x] is not None}
    dx, dyy = c["dx_out"].clone(), c["y"].clone()
    pb.pi_block_norm_backward(c["norm"], r, dyy, kp, kr, c["du"], dx, dx, dyy, ws, flags=pb.PI_GRAD_ACCUMULATE, **acc)
    assert torch.equal(dx, out["dx"]) and torch.equal(dyy, out["dy"])
    for x, t in acc.items():
        assert torch.all((t - 2 - out[x]).abs() <= 4 * E * (2 + out[x].abs()) + adds * 4), x


def test_gradients_agree_with_differences(cuda_device):
    """<gradient, v> against (L(+h v) - L(-h v)) / 2h of the fp64 forward pass, L = <u, du> + <r, dx_out>."""
    T, d, per = 29, 200, 8
    c = _case(T, d, F32, F32, True, per, seed=4)
    r, u = torch.empty(T, d, device="cuda"), torch.empty(T, d, device="cuda")
    kp, kr = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    pb.pi_block_norm_forward(c["norm"], c["x"], c["y"], r, u, kp, kr)
    out = _run_backward(c, T, d, kp, kr, r)
    names = {"x": "dx", "y": "dy", "gate": "dgate", "w_post": "dw_post", "w_pre": "dw_pre"}

    def loss(**kw):
        rr, uu, _, _ = _reference(c, **kw)
        return (rr * c["dx_out"].to(D)).sum() + (uu * c["du"].to(D)).sum()
    gen, h = torch.Generator(device="cuda").manual_seed(9), 1e-5
    for k, g in names.items():
        base = _d(c[k])
        v = torch.randn(base.shape, generator=gen, device="cuda", dtype=D)
        diff = (loss(**{k: base + h * v}) - loss(**{k: base - h * v})) / (2 * h)
        got = (out[g].to(D) * v).sum()
        # fp32 roundings of the forward outputs and the gradient: below 200 E of the terms' size; differences: h^2
        size = torch.sqrt((out[g].to(D) ** 2 * v ** 2).sum())
        assert (got - diff).abs() <= 200 * E * size + 1e-7 * (1 + diff.abs()), k


def test_backward_with_parts_left_out(cuda_device):
    T, d = 70, 264
    c = _case(T, d, BF16, BF16, True, 32, seed=6)
    r, u = torch.empty(T, d, device="cuda"), torch.empty(T, d, dtype=BF16, device="cuda")
    kp, kr = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    pb.pi_block_norm_forward(c["norm"], c["x"], c["y"], r, u, kp, kr)
    ws = pb.make_block_norm_workspace(c["norm"], T)
    n, dx, dy = c["norm"], torch.empty(T, d, device="cuda"), torch.empty_like(c["y"])
    # only the stream's gradient arrives: dx = alpha dx_out
    pb.pi_block_norm_backward(n, None, None, None, None, None, c["dx_out"], dx, None, ws)
    assert torch.equal(dx, torch.tensor(0.9, device="cuda") * c["dx_out"])
    # only u's
    pb.pi_block_norm_backward(n, r, c["y"], kp, kr, c["du"], None, dx, dy, ws)
    zero = torch.zeros(T, d, device="cuda")
    dx2, dy2 = torch.empty_like(dx), torch.empty_like(dy)
    pb.pi_block_norm_backward(n, r, c["y"], kp, kr, c["du"], zero, dx2, dy2, ws)
    assert torch.equal(dx, dx2) and torch.equal(dy, dy2)
    # a parameter's gradient alone
    full = _run_backward(c, T, d, kp, kr, r)
    for k in ("dw_post", "dw_pre", "dgate"):
        g = torch.empty_like(full[k])
        pb.pi_block_norm_backward(n, r, c["y"], kp, kr, c["du"], c["dx_out"], None, None, ws, **{k: g})
        assert torch.equal(g, full[k]), k


def test_zero_rows_and_no_tokens(cuda_device):
    d = 72
    n = pb.BlockNorm(d, y_dtype=F16, u_dtype=F16, post_norm=True)
    x, y = torch.zeros(3, d, device="cuda"), torch.zeros(3, d, dtype=F16, device="cuda")
    r, u, kr = torch.empty_like(x), torch.empty_like(y), torch.empty(3, device="cuda")
    pb.pi_block_norm_forward(n, x, y, r, u, rstd_pre=kr)
    assert torch.all(r == 0) and torch.all(u == 0) and torch.all((kr - 1000).abs() < 0.01)
    e = x[:0]
    pb.pi_block_norm_forward(n, e, y[:0], r[:0], u[:0])
    ws = pb.make_block_norm_workspace(n, 0)
    dw = torch.ones(d, device="cuda")
    pb.pi_block_norm_backward(n, e, y[:0], kr[:0], kr[:0], y[:0], e, r[:0], y[:0], ws, dw_pre=dw,
                              flags=pb.PI_GRAD_ACCUMULATE)
    assert torch.all(dw == 1)
    pb.pi_block_norm_backward(n, e, y[:0], kr[:0], kr[:0], y[:0], e, r[:0], y[:0], ws, dw_pre=dw)
    assert torch.all(dw == 0)


def test_non_finite_rows_stay_apart(cuda_device):
    c = _case(9, 264, F16, F16, True, 0, seed=8)
    r, u = torch.empty(9, 264, device="cuda"), torch.empty(9, 264, dtype=F16, device="cuda")
    pb.pi_block_norm_forward(c["norm"], c["x"], c["y"], r, u)
    x, y = c["x"].clone(), c["y"].clone()
    x[2, 0], y[5, 100] = float("nan"), float("inf")
    r2, u2 = torch.empty_like(r), torch.empty_like(u)
    pb.pi_block_norm_forward(c["norm"], x, y, r2, u2)
    keep = [0, 1, 3, 4, 6, 7, 8]
    assert torch.equal(r2[keep], r[keep]) and torch.equal(u2[keep], u[keep])
    assert torch.isnan(u2[2]).all() and not torch.isfinite(u2[5]).all()


def test_captured_and_replayed(cuda_device):
    c = _case(200, 1032, BF16, BF16, True, 64, seed=10)
    T, d = 200, 1032
    r, u = torch.empty(T, d, device="cuda"), torch.empty(T, d, dtype=BF16, device="cuda")
    kp, kr = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    ws = pb.make_block_norm_workspace(c["norm"], T)
    dx, dy = torch.empty(T, d, device="cuda"), torch.empty_like(c["y"])
    dw = [torch.empty(d, device="cuda"), torch.empty(d, device="cuda"), torch.empty_like(c["gate"])]

    def step_():
        pb.pi_block_norm_forward(c["norm"], c["x"], c["y"], r, u, kp, kr)
        pb.pi_block_norm_backward(c["norm"], r, c["y"], kp, kr, c["du"], c["dx_out"], dx, dy, ws, *dw)
    step_()
    want = [t.clone() for t in (r, u, dx, dy, *dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_()
    for t in (r, u, dx, dy, *dw):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (r, u, dx, dy, *dw)))


def test_offsets_past_32_bits(cuda_device):
    T, d = 140_000, 16_376
    assert T * d > 2 ** 31
    n = pb.BlockNorm(d, y_dtype=F16, u_dtype=F16, post_norm=True)
    x = torch.zeros(T, d, device="cuda")
    y = torch.zeros(T, d, dtype=F16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x[-5:], y[-5:] = torch.randn(5, d, generator=gen, device="cuda"), 0.5
    u = torch.empty(T, d, dtype=F16, device="cuda")
    kr = torch.empty(T, device="cuda")
    pb.pi_block_norm_forward(n, x, y, x, u, rstd_pre=kr)
    x5 = torch.randn(5, d, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    u5, kr5 = torch.empty(5, d, dtype=F16, device="cuda"), torch.empty(5, device="cuda")
    y5 = torch.full((5, d), 0.5, dtype=F16, device="cuda")
    pb.pi_block_norm_forward(n, x5, y5, x5, u5, rstd_pre=kr5)
    assert torch.equal(u[-5:], u5) and torch.equal(x[-5:], x5) and torch.all(u[:-5] == 0)
    # the backward pass over the same rows: only the last five have a gradient
    du = torch.zeros(T, d, dtype=F16, device="cuda")
    du[-5:] = 0.25
    del y, u
    ws = pb.make_block_norm_workspace(n, T)
    dx, dw = torch.empty(T, d, device="cuda"), torch.empty(d, device="cuda")
    pb.pi_block_norm_backward(n, x, None, None, kr, du, None, dx, None, ws, dw_pre=dw)
    dx5, dw5 = torch.empty(5, d, device="cuda"), torch.empty(d, device="cuda")
    pb.pi_block_norm_backward(n, x5, None, None, kr5, du[-5:].clone(), None, dx5, None, ws, dw_pre=dw5)
    assert torch.equal(dx[-5:], dx5) and torch.all(dx[:-5] == 0)
    assert torch.all((dw - dw5).abs() <= 16 * E * (x5 * kr5[:, None]).abs().sum(0) * 0.25)


def test_gate_rows_longer_than_the_batch(cuda_device):
    """tokens_per_gate up to the largest int: one row for all tokens."""
    T, d = 90, 264
    c = _case(T, d, F16, F16, True, T, seed=12)
    big = pb.BlockNorm(d, y_dtype=F16, u_dtype=F16, eps=EPS, residual_scale=c["alpha"], branch_scale=c["beta"],
                       post_norm=True, w_post=c["w_post"], w_pre=c["w_pre"], gate=c["gate"],
                       tokens_per_gate=2 ** 31 - 1)
    outs = []
    for norm in (c["norm"], big):
        r, u = torch.empty(T, d, device="cuda"), torch.empty(T, d, dtype=F16, device="cuda")
        kp, kr = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        pb.pi_block_norm_forward(norm, c["x"], c["y"], r, u, kp, kr)
        out = _run_backward(dict(c, norm=norm), T, d, kp, kr, r)
        outs.append([r, u, *out.values()])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_two_streams_at_once(cuda_device):
    """Calls on two streams with a workspace each do not disturb one another."""
    T, d = 300, 2056
    cs = [_case(T, d, BF16, BF16, True, 64, seed=s) for s in (20, 21)]
    fwd = []
    for c in cs:
        r, u = torch.empty(T, d, device="cuda"), torch.empty(T, d, dtype=BF16, device="cuda")
        kp, kr = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        pb.pi_block_norm_forward(c["norm"], c["x"], c["y"], r, u, kp, kr)
        fwd.append((kp, kr, r))
    want = [_run_backward(c, T, d, *f) for c, f in zip(cs, fwd)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cs], [None, None]
    for _ in range(5):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k] = _run_backward(cs[k], T, d, *fwd[k])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a[x], b[x]) for x in a if a[x] is not None)


def test_backward_refuses_outputs_in_its_workspace(cuda_device):
    T, d = 5, 64
    n = pb.BlockNorm(d, y_dtype=F32, u_dtype=F32)
    ws = pb.make_block_norm_workspace(n, T)
    x, kr, g = torch.ones(T, d, device="cuda"), torch.ones(T, device="cuda"), torch.ones(T, d, device="cuda")
    used = ws.view(torch.float32)
    dw = used[64:64 + d]  # the first row of partial sums
    with pytest.raises(pb.PiError):
        pb.pi_block_norm_backward(n, x, None, None, kr, g, None, torch.empty_like(x), None, ws, dw_pre=dw)
    assert torch.all(kr == 1)
