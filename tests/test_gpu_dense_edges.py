"""The dense block operators at the edges of what their documentation allows:
the largest sizes, outputs between guards, non-finite values in backward
passes, an explicit stream, graphs with forks and memsets, and the operators
in one stream with the sparse decode step, none waiting for another."""
import pytest
import torch

import dense_ref as ref
from activation_sparse_decode_gemv_b200 import binding as pb
from activation_sparse_decode_gemv_b200 import inputs
from test_gpu_block_norm import _case
from test_gpu_dense_plans import _backward, _forward, _product
from test_gpu_gated_ffn import _rand_case

pytestmark = pytest.mark.gpu

D = torch.float64
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAN, INF = float("nan"), float("inf")


def _e(*s, dt=F32):
    return torch.empty(*s, dtype=dt, device="cuda")


def _guarded(*shape, dt=F32, fill=7.0):
    """An output between 64 known values, and the check that they are untouched."""
    n = 1
    for s in shape:
        n *= s
    end = -(-n // 8) * 8 + 128
    buf = torch.full((end,), fill, dtype=dt, device="cuda")
    return buf[64:64 + n].view(*shape), lambda: bool(torch.all(buf[:64] == fill) and torch.all(buf[64 + n:] == fill))


# ---------------------------------------------------------------- largest sizes
@pytest.mark.parametrize("T,d,f", [(2 ** 24, 8, 8), (1, 2 ** 20, 8), (130, 2 ** 20, 8), (1, 8, 2 ** 20),
                                   (130, 8, 2 ** 20)])
def test_largest_blocks(cuda_device, T, d, f):
    _forward(T, d, f, BF16)
    _backward(T, d, f, BF16, F32)


@pytest.mark.parametrize("T,n,k", [(1, 2 ** 20, 16), (200, 2 ** 20, 16), (2 ** 24, 8, 16)])
def test_largest_8_bit_products(cuda_device, T, n, k):
    _product(T, n, k, F16 if T > 1 else F32, None)


@pytest.mark.parametrize("rows,k", [(70_000, 16), (2 ** 24, 16), (3, 131056)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_largest_quantiser(cuda_device, rows, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, k, generator=gen, device="cuda").to(dtype)
    q, s = _e(rows, k, dt=torch.int8), _e(rows)
    pb.pi_quantize_i8(x, q, s)
    wq, ws = ref.quantize(x.float())
    assert torch.equal(s, ws) and torch.equal(q, wq)


def test_largest_token_count_of_the_norms(cuda_device):
    T, d = 2 ** 24, 8
    gen = torch.Generator(device="cuda").manual_seed(3)
    # whole numbers: r is exact, and the last tokens' rows are those of a call on them alone
    x = torch.randint(-3, 4, (T, d), generator=gen, device="cuda").float()
    gate = torch.ones(2, d, device="cuda")
    gate[1] = 2
    norm = pb.BlockNorm(d, y_dtype=F32, u_dtype=F16, gate=gate, tokens_per_gate=2 ** 23)
    r, u, kr = _e(T, d), _e(T, d, dt=F16), _e(T)
    pb.pi_block_norm_forward(norm, x, x, r, u, rstd_pre=kr)
    assert torch.equal(r[:2 ** 23], 2 * x[:2 ** 23]) and torch.equal(r[2 ** 23:], 3 * x[2 ** 23:])
    del r, u
    ws = pb.make_block_norm_workspace(norm, T)
    dy, dg = _e(T, d), _e(2, d)
    pb.pi_block_norm_backward(norm, None, x, None, None, None, x, None, dy, ws, dgate=dg)
    assert torch.equal(dy[:2 ** 23], x[:2 ** 23]) and torch.equal(dy[2 ** 23:], 2 * x[2 ** 23:])
    want = (x.to(D) ** 2).view(2, -1, d).sum(1)  # about 2^25: partial sums of at most 2^24 tokens in fp32
    assert torch.all((dg.to(D) - want).abs() <= 2 ** -23 * 64 * want)


# ---------------------------------------------------------------- guards
@pytest.mark.parametrize("T,d", [(1, 8), (37, 1000), (130, 2056), (5, 8200), (3, 16384)])
@pytest.mark.parametrize("yt,ut,per", [(F16, BF16, 5), (F32, F32, 1), (BF16, F16, 64)])
def test_norm_outputs_stay_inside(cuda_device, T, d, yt, ut, per):
    c = _case(T, d, yt, ut, True, per, seed=31)
    outs = [_guarded(T, d), _guarded(T, d, dt=ut), _guarded(T), _guarded(T)]
    (r, _), (u, _), (kp, _), (kr, _) = outs
    pb.pi_block_norm_forward(c["norm"], c["x"], c["y"], r, u, kp, kr)
    ws = pb.make_block_norm_workspace(c["norm"], T)
    size = ws.numel()
    big = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")  # the workspace, with room behind it
    big[:256] = 0
    outs += [_guarded(T, d), _guarded(T, d, dt=yt), _guarded(d), _guarded(d), _guarded(*c["gate"].shape)]
    pb.pi_block_norm_backward(c["norm"], r, c["y"], kp, kr, c["du"], c["dx_out"], outs[4][0], outs[5][0], big[:size],
                              outs[6][0], outs[7][0], outs[8][0])
    for k, (_, fine) in enumerate(outs):
        assert fine(), k
    assert torch.all(big[size:] == 77) and torch.all(big[:256] == 0)


def test_quantiser_outputs_stay_inside(cuda_device):
    for rows, k in ((1, 16), (33, 272), (5, 8192)):
        q, fq = _guarded(rows, k, dt=torch.int8, fill=7)
        s, fs = _guarded(rows)
        pb.pi_quantize_i8(torch.randn(rows, k, device="cuda"), q, s)
        assert fq() and fs()


def test_ffn_workspace_stays_inside(cuda_device):
    for T in (3, 300):
        u, wg, wu, wd, dy = _rand_case(T, 264, 1032, F16, 5)
        layer = pb.GatedFfnLayer(wg, wu, wd)
        size = pb.pi_gated_ffn_workspace_size(layer, T, True)
        big = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
        big[:256] = 0
        y, g, p = torch.empty_like(u), _e(T, 1032, dt=F16), _e(T, 1032, dt=F16)
        pb.pi_gated_ffn_forward(layer, u, y, big[:size], gate=g, up=p)
        pb.pi_gated_ffn_backward(layer, u, g, p, dy, big[:size], y, *(torch.empty_like(wg) for _ in range(3)))
        assert torch.all(big[size:] == 77) and torch.all(big[:256] == 0)


# ---------------------------------------------------------------- non-finite values in backward passes
@pytest.mark.parametrize("T", [3, 100, 600])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_non_finite_gradients_of_the_block_stay_apart(cuda_device, T, bad):
    d, f, dtype = 264, 520, BF16
    u, wg, wu, wd, dy = _rand_case(T, d, f, dtype, 11)
    layer = pb.GatedFfnLayer(wg, wu, wd)
    ws = pb.make_gated_ffn_workspace(layer, T, True)
    y, g, p = torch.empty_like(u), _e(T, f, dt=dtype), _e(T, f, dt=dtype)
    pb.pi_gated_ffn_forward(layer, u, y, ws, gate=g, up=p)

    def back(u=u, g=g, p=p, dy=dy):
        o = [torch.empty_like(u)] + [torch.empty_like(wg) for _ in range(3)]
        pb.pi_gated_ffn_backward(layer, u, g, p, dy, ws, *o)
        return o
    clean = back()

    def with_bad(t, at):
        t = t.clone()
        t[at] = bad
        return t
    rows, cols, neurons = (torch.arange(n, device="cuda") for n in (T, d, f))
    # u enters the matrices' gradients alone: its column of two of them
    du, dwg, dwu, dwd = back(u=with_bad(u, (1, 5)))
    assert torch.equal(du, clean[0]) and torch.equal(dwd, clean[3])
    for got, want in ((dwg, clean[1]), (dwu, clean[2])):
        assert not torch.isfinite(got[:, 5]).any() and torch.equal(got[:, cols != 5], want[:, cols != 5])
    # the kept gate: its token's row of du, its neuron's row of the matrices' gradients
    du, *dw = back(g=with_bad(g, (1, 9)))
    assert not torch.isfinite(du[1]).any() and torch.equal(du[rows != 1], clean[0][rows != 1])
    for got, want in zip(dw, clean[1:]):
        assert not torch.isfinite(got[9]).any() and torch.equal(got[neurons != 9], want[neurons != 9])
    # dy: its token's row of du, its column of dW2T (all of the other two)
    du, dwg, dwu, dwd = back(dy=with_bad(dy, (T - 1, 7)))
    assert not torch.isfinite(du[T - 1]).any() and torch.equal(du[rows != T - 1], clean[0][rows != T - 1])
    assert not torch.isfinite(dwd[:, 7]).any() and torch.equal(dwd[:, cols != 7], clean[3][:, cols != 7])
    assert pb.pi_get_device_status(ws) == 0


@pytest.mark.parametrize("T,d", [(9, 264), (9, 8200)])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_non_finite_gradients_of_the_norms_stay_apart(cuda_device, T, d, bad):
    c = _case(T, d, F32, F32, True, 3, seed=8)
    r, u, kp, kr = _e(T, d), _e(T, d), _e(T), _e(T)
    pb.pi_block_norm_forward(c["norm"], c["x"], c["y"], r, u, kp, kr)
    ws = pb.make_block_norm_workspace(c["norm"], T)

    def back(**kw):
        a = dict(c, r=r, **kw)
        o = [_e(T, d), _e(T, d), _e(d), _e(d), torch.empty_like(c["gate"])]
        pb.pi_block_norm_backward(c["norm"], a["r"], a["y"], kp, kr, a["du"], a["dx_out"], o[0], o[1], ws, *o[2:])
        return o
    clean = back()
    rows, cols = torch.arange(T, device="cuda"), torch.arange(d, device="cuda")
    for name in ("du", "dx_out"):
        t = c[name].clone()
        t[4, 11] = bad  # gate row 1
        dx, dy, dwp, dw, dg = back(**{name: t})
        for got, want in ((dx, clean[0]), (dy, clean[1])):
            assert not torch.isfinite(got[4, 11]) and torch.equal(got[rows != 4], want[rows != 4])
        assert torch.equal(dg[[0, 2]], clean[4][[0, 2]]) and not torch.isfinite(dg[1, 11])
        assert not torch.isfinite(dwp[11])
        assert torch.equal(dw[cols != 11], clean[3][cols != 11]) and bool(torch.isfinite(dw[11])) == (name == "dx_out")


# ---------------------------------------------------------------- gates
@pytest.mark.parametrize("T,per", [(20_000, 1), (20_000, 3), (20_000, 133), (20_000, 2500), (20_000, 2501),
                                   (20_000, 19_999), (4097, 4096), (777, 776)])
def test_gate_rows_of_any_length(cuda_device, T, per):
    """dgate and dw_post of whole numbers are exact, whichever blocks share a gate row.  Rows behind the last token's
    are left as they were."""
    d = 72
    gen = torch.Generator(device="cuda").manual_seed(T + per)
    n = lambda *s: torch.randint(-2, 3, s, generator=gen, device="cuda").float()  # noqa: E731
    rows = -(-T // per)
    gate, y, g = n(rows + 2, d), n(T, d), n(T, d)
    norm = pb.BlockNorm(d, y_dtype=F32, u_dtype=F32, gate=gate, tokens_per_gate=per)
    ws = pb.make_block_norm_workspace(norm, T)
    dg, dy = torch.full((rows + 2, d), 7.0, device="cuda"), _e(T, d)
    pb.pi_block_norm_backward(norm, None, y, None, None, None, g, None, dy, ws, dgate=dg)
    at = torch.arange(T, device="cuda") // per
    want = torch.zeros(rows, d, dtype=D, device="cuda").index_add_(0, at, (y * g).to(D))
    assert torch.equal(dg[:rows].to(D), want) and torch.all(dg[rows:] == 7)
    assert torch.equal(dy, g * gate[at])
    pb.pi_block_norm_backward(norm, None, y, None, None, None, g, None, None, ws, dgate=dg, flags=pb.PI_GRAD_ACCUMULATE)
    assert torch.equal(dg[:rows].to(D), 2 * want) and torch.all(dg[rows:] == 7)


# ---------------------------------------------------------------- streams and graphs
def _chain(T, dtype=F16):
    """Everything of this library in one stream: each call reads what the one before has written."""
    d, f = 512, 2048
    cfg = inputs.CONFIGS["opt7b_f16"].scaled(d=d, f=f, r=128)
    sparse = pb.FfnLayer.from_tensors(inputs.make_layer(cfg, 0, seed=1).to(torch.device("cuda")))
    u0, wg, wu, wd, dy = _rand_case(T, d, f, dtype, 77)
    dense = pb.GatedFfnLayer(wg, wu, wd)
    norm = pb.BlockNorm(d, y_dtype=F32, u_dtype=dtype, post_norm=True, branch_scale=0.5)
    norm2 = pb.BlockNorm(d, y_dtype=dtype, u_dtype=dtype)
    wq, sw = _e(d, d, dt=torch.int8), _e(d)
    pb.pi_quantize_i8(wg[:d], wq, sw)
    b = {"x": torch.empty(T, d, device="cuda"), "u": _e(T, d, dt=dtype), "y": _e(T, d, dt=dtype), "ys": _e(T, d),
         "g": _e(T, f, dt=dtype), "p": _e(T, f, dt=dtype), "q": _e(T, d, dt=torch.int8), "s": _e(T), "kp": _e(T),
         "kr": _e(T), "du": _e(T, d, dt=dtype), "dw": _e(f, d), "dx": _e(T, d), "dyb": _e(T, d), "dn": _e(d)}
    ws = [pb.make_workspace([sparse], T), pb.make_gated_ffn_workspace(dense, T, True),
          pb.make_block_norm_workspace(norm, T), pb.make_matmul_i8_workspace(T, d, d)]
    x0 = torch.randn(T, d, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")

    def run(between=lambda: None):
        b["x"].copy_(x0)
        steps = [lambda: pb.pi_block_norm_forward(norm2, b["x"], None, None, b["u"]),
                 lambda: pb.pi_decode_ffn(sparse, b["u"], b["ys"], ws[0]),
                 lambda: pb.pi_block_norm_forward(norm, b["x"], b["ys"], b["x"], b["u"], b["kp"], b["kr"]),
                 lambda: pb.pi_gated_ffn_forward(dense, b["u"], b["y"], ws[1], gate=b["g"], up=b["p"]),
                 lambda: pb.pi_gated_ffn_backward(dense, b["u"], b["g"], b["p"], b["y"], ws[1], b["du"], dw_up=b["dw"]),
                 lambda: pb.pi_block_norm_backward(norm, b["x"], b["ys"], b["kp"], b["kr"], b["du"], None, b["dx"],
                                                   b["dyb"], ws[2], dw_pre=b["dn"]),
                 lambda: pb.pi_quantize_i8(b["dx"], b["q"], b["s"]),
                 lambda: pb.pi_matmul_i8(b["q"], b["s"], wq, sw, b["ys"], ws[3]),
                 lambda: pb.pi_block_norm_forward(norm, b["x"], b["ys"], b["x"], b["u"]),
                 lambda: pb.pi_decode_ffn(sparse, b["u"], b["ys"], ws[0]),
                 lambda: pb.pi_block_norm_forward(norm, b["x"], b["ys"], b["x"], b["u"])]
        for s in steps:
            s()
            between()
    return run, b, ws


@pytest.mark.parametrize("T", [1, 4, 20])
def test_calls_in_a_row_wait_for_what_they_read(cuda_device, T):
    run, b, ws = _chain(T)
    run(torch.cuda.synchronize)
    want = {k: v.clone() for k, v in b.items()}
    for _ in range(20):
        run()
    torch.cuda.synchronize()
    assert all(torch.equal(b[k], want[k]) for k in b), [k for k in b if not torch.equal(b[k], want[k])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
        run()
    for v in b.values():
        v.zero_()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(b[k], want[k]) for k in b), [k for k in b if not torch.equal(b[k], want[k])]
    assert all(pb.pi_get_device_status(w) == 0 for w in ws)


@pytest.mark.parametrize("T", [2, 300])
def test_captured_with_forks_joins_and_memsets(cuda_device, T):
    """Both branches of a fork write what the call after the join reads; outputs are cleared inside the graph."""
    d, f = 264, 1032
    jobs = []
    for k in range(2):
        u, wg, wu, wd, _ = _rand_case(T, d, f, F16, 60 + k)
        layer = pb.GatedFfnLayer(wg, wu, wd)
        jobs.append((layer, u, torch.empty_like(u), pb.make_gated_ffn_workspace(layer, T)))
    x, r, u2 = torch.randn(T, d, device="cuda"), _e(T, d), _e(T, d, dt=F16)
    norm = pb.BlockNorm(d, y_dtype=F16, u_dtype=F16)
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        for _, _, y, _ in jobs:
            y.zero_()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            pb.pi_gated_ffn_forward(*jobs[1][:3], jobs[1][3])
        pb.pi_gated_ffn_forward(*jobs[0][:3], jobs[0][3])
        main.wait_stream(side)
        pb.pi_block_norm_forward(norm, x, jobs[1][2], r, u2)
        pb.pi_block_norm_forward(norm, r, jobs[0][2], r, u2)
    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in (r, u2, jobs[0][2], jobs[1][2])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(10):
        r.zero_(), u2.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (r, u2, jobs[0][2], jobs[1][2])))


def test_an_explicit_stream(cuda_device):
    """stream=: the work goes there, whatever the current stream is."""
    side = torch.cuda.Stream()
    x, u = torch.randn(4, 512, device="cuda"), torch.zeros(4, 512, dtype=F16, device="cuda")
    norm = pb.BlockNorm(512)
    want = torch.empty_like(u)
    pb.pi_block_norm_forward(norm, x, None, None, want)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms of work before it
    pb.pi_block_norm_forward(norm, x, None, None, u, stream=side)
    early = u.clone()  # on the current stream: does not wait for the side stream
    torch.cuda.current_stream().synchronize()
    assert torch.all(early == 0)
    side.synchronize()
    assert torch.equal(u, want)


# ---------------------------------------------------------------- no branch
@pytest.mark.parametrize("T,d", [(5, 264), (3, 8200)])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_without_a_branch_its_parameters_are_not_used(cuda_device, T, d, bad):
    """y = None: r = residual_scale x, whatever the branch's gate and weights hold."""
    gate, w = torch.full((T, d), bad, device="cuda"), torch.full((d,), bad, device="cuda")
    norm = pb.BlockNorm(d, y_dtype=F32, u_dtype=F32, post_norm=True, w_post=w, gate=gate, tokens_per_gate=1,
                        residual_scale=2.0, branch_scale=0.5)
    plain = pb.BlockNorm(d, u_dtype=F32, residual_scale=2.0)
    x = torch.randn(T, d, device="cuda")
    r, u, r0, u0 = (_e(T, d) for _ in range(4))
    pb.pi_block_norm_forward(norm, x, None, r, u)
    pb.pi_block_norm_forward(plain, x, None, r0, u0)
    assert torch.equal(r, 2 * x) and torch.equal(u, u0) and torch.equal(r, r0)
