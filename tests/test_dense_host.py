"""Argument checks of the dense block operators, on the CPU: the library
refuses before any launch (made-up device addresses are never read), and the
binding refuses what the C ABI cannot see.  Also the plain forms that the GPU
tests use, against torch's automatic differentiation."""
import ctypes as C
import os

import pytest
import torch

import dense_ref as ref
from activation_sparse_decode_gemv_b200 import binding as pb

OK, ARG, UNSUP, ALIGN, WS = pb.PI_OK, pb.PI_ERR_INVALID_ARG, pb.PI_ERR_UNSUPPORTED, pb.PI_ERR_MISALIGNED, \
    pb.PI_ERR_WORKSPACE
vp = C.c_void_p
A, B_, C_, D_, E_, F_, G_, H_ = (vp(0x100000000 * (i + 1)) for i in range(8))


@pytest.fixture(scope="module")
def lib():
    if not os.environ.get("PI_FFN_LIB"):  # another build given: use it as is
        from activation_sparse_decode_gemv_b200 import build
        build.build()
    return pb.lib()


def _gated(lib, **kw):
    base = dict(d_model=64, d_ffn=128, act=pb.PI_GATE_SILU, dtype=pb.PI_DT_F16, w_gate=0x1000, w_up=0x2000,
                w_down_t=0x3000)
    base.update(kw)
    h = vp()
    rc = lib.pi_gated_ffn_create(C.byref(pb.pi_gated_ffn_desc(**base)), C.byref(h))
    return rc, h


def test_gated_ffn_create(lib):
    def rc(**kw):
        r, h = _gated(lib, **kw)
        assert (r == OK) == bool(h)
        lib.pi_gated_ffn_destroy(h)
        return r
    assert rc() == OK and rc(dtype=pb.PI_DT_BF16, act=pb.PI_GATE_GELU) == OK
    assert rc(d_model=0) == ARG and rc(d_ffn=-8) == ARG
    assert rc(act=3) == ARG and rc(act=-1) == ARG and rc(dtype=3) == ARG
    assert rc(w_gate=None) == ARG and rc(w_up=None) == ARG and rc(w_down_t=None) == ARG
    assert rc(dtype=pb.PI_DT_F32) == UNSUP
    assert rc(d_model=60) == UNSUP and rc(d_ffn=100) == UNSUP and rc(d_model=2 ** 20 + 8) == UNSUP
    assert rc(w_up=0x2008) == ALIGN
    assert lib.pi_gated_ffn_create(None, C.byref(vp())) == ARG
    lib.pi_gated_ffn_destroy(None)


def test_gated_ffn_calls(lib):
    _, h = _gated(lib)
    n = C.c_size_t()
    size = lib.pi_gated_ffn_workspace_size
    assert size(h, 10, 0, C.byref(n)) == OK and n.value == 256 + 10 * 128 * 2
    assert size(h, 10, 1, C.byref(n)) == OK and n.value == 256 + 3 * 10 * 128 * 2
    assert size(None, 10, 0, C.byref(n)) == ARG and size(h, -1, 0, C.byref(n)) == UNSUP
    assert size(h, 2 ** 24 + 1, 0, C.byref(n)) == UNSUP and size(h, 1, 0, None) == ARG
    fwd = lib.pi_gated_ffn_forward
    assert fwd(None, A, 1, B_, None, None, C_, 1 << 20, None) == ARG
    assert fwd(h, None, 1, B_, None, None, C_, 1 << 20, None) == ARG
    assert fwd(h, A, 1, None, None, None, C_, 1 << 20, None) == ARG
    assert fwd(h, A, -1, B_, None, None, C_, 1 << 20, None) == UNSUP
    assert fwd(h, vp(8), 1, B_, None, None, C_, 1 << 20, None) == ALIGN
    assert fwd(h, A, 1, B_, vp(4), None, C_, 1 << 20, None) == ALIGN
    assert fwd(h, A, 1, B_, None, None, None, 1 << 20, None) == WS
    assert fwd(h, A, 1, B_, None, None, C_, 256 + 255, None) == WS
    assert fwd(h, A, 1, B_, None, None, vp(0x1008), 1 << 20, None) == ALIGN
    assert fwd(h, None, 0, None, None, None, None, 0, None) == OK  # no tokens: nothing is read
    # outputs over inputs, each other or the workspace
    assert fwd(h, A, 1, A, None, None, C_, 1 << 20, None) == ARG
    assert fwd(h, A, 2, B_, vp(B_.value + 128), None, C_, 1 << 20, None) == ARG
    assert fwd(h, A, 1, B_, D_, D_, C_, 1 << 20, None) == ARG
    assert fwd(h, A, 1, B_, C_, None, C_, 1 << 20, None) == ARG
    bwd = lib.pi_gated_ffn_backward
    ok = [h, A, B_, C_, D_, 4, E_, F_, G_, H_, pb.PI_DT_F32, 0, vp(0x9000), 1 << 20, None]

    def b(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return bwd(*a)
    assert b(_0=None) == ARG and b(_1=None) == ARG and b(_2=None) == ARG and b(_3=None) == ARG and b(_4=None) == ARG
    assert b(_5=-1) == UNSUP and b(_10=7) == ARG and b(_10=pb.PI_DT_BF16) == UNSUP and b(_11=2) == ARG
    assert b(_6=D_) == ARG and b(_6=A) == ARG and b(_8=F_) == ARG and b(_9=vp(E_.value + 64)) == ARG
    assert b(_7=vp(0x9100)) == ARG  # over the workspace
    assert b(_7=vp(0x18)) == ALIGN and b(_12=None) == WS and b(_13=256 + 3 * 1024 - 1) == WS
    lib.pi_gated_ffn_destroy(h)


def _norm(**kw):
    base = dict(d_model=64, y_dtype=pb.PI_DT_F16, u_dtype=pb.PI_DT_F16, post_norm=1, eps=1e-6, residual_scale=1.0,
                branch_scale=1.0, w_post=0x1000, w_pre=0x2000, gate=0x3000, tokens_per_gate=4)
    base.update(kw)
    return C.byref(pb.pi_block_norm_desc(**base))


def test_block_norm_calls(lib):
    def fwd(desc=None, x=A, y=B_, T=4, r=C_, u=D_, kp=None, kr=None):
        return lib.pi_block_norm_forward(desc or _norm(), x, y, T, r, u, kp, kr, None)
    inf, nan = float("inf"), float("nan")
    for kw in (dict(d_model=0), dict(y_dtype=3), dict(u_dtype=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=nan),
               dict(eps=inf), dict(residual_scale=nan), dict(branch_scale=inf), dict(post_norm=0),
               dict(tokens_per_gate=0), dict(tokens_per_gate=-3)):
        assert fwd(_norm(**kw)) == ARG, kw
    assert fwd(_norm(d_model=60)) == UNSUP and fwd(_norm(d_model=16392)) == UNSUP
    assert fwd(_norm(w_pre=0x2004)) == ALIGN and fwd(_norm(gate=0x3008)) == ALIGN
    assert lib.pi_block_norm_forward(None, A, B_, 4, C_, D_, None, None, None) == ARG
    assert fwd(x=None) == ARG and fwd(r=None, u=None) == ARG
    assert fwd(u=None, kr=E_) == ARG and fwd(y=None, kp=E_) == ARG
    assert fwd(_norm(post_norm=0, w_post=None), kp=E_) == ARG
    assert fwd(T=-1) == UNSUP and fwd(T=2 ** 24 + 1) == UNSUP
    assert fwd(x=vp(8)) == ALIGN and fwd(kr=vp(0x24)) == ALIGN
    # outputs over inputs: the stream in place is allowed (not tried here), nothing else
    assert fwd(r=vp(A.value + 16)) == ARG and fwd(u=A) == ARG and fwd(r=B_) == ARG and fwd(u=vp(B_.value + 32)) == ARG
    assert fwd(u=C_) == ARG
    assert fwd(x=None, y=None, T=0, r=None, u=None) == OK

    ws = vp(0x9000)

    def bwd(desc=None, r=A, y=B_, kp=vp(0x100), kr=vp(0x200), du=C_, g=D_, T=4, dx=E_, dy=F_, dwp=G_, dw=H_, dg=None,
            flags=0, ws=ws, n=1 << 30):
        return lib.pi_block_norm_backward(desc or _norm(), r, y, kp, kr, du, g, T, dx, dy, dwp, dw, dg, flags, ws, n,
                                          None)
    assert bwd(du=None, g=None) == ARG and bwd(r=None) == ARG and bwd(kr=None) == ARG and bwd(kp=None) == ARG
    assert bwd(y=None) == ARG and bwd(du=None) == ARG  # dw_pre without u's gradient
    assert bwd(_norm(post_norm=0, w_post=None)) == ARG and bwd(_norm(gate=None), dg=vp(0x300)) == ARG
    assert bwd(flags=2) == ARG and bwd(T=-1) == UNSUP and bwd(dx=vp(8)) == ALIGN
    assert bwd(dx=A) == ARG and bwd(dx=vp(D_.value + 16)) == ARG and bwd(dy=A) == ARG and bwd(dy=C_) == ARG
    assert bwd(dy=vp(B_.value + 16)) == ARG and bwd(dx=F_) == ARG
    assert bwd(ws=None) == WS and bwd(ws=vp(0x9008)) == ALIGN
    n = C.c_size_t()
    assert lib.pi_block_norm_workspace_size(_norm(), -1, C.byref(n)) == UNSUP
    assert lib.pi_block_norm_workspace_size(_norm(), 1, None) == ARG
    assert lib.pi_block_norm_workspace_size(_norm(d_model=4), 1, C.byref(n)) == UNSUP


def test_outputs_over_weights_and_parameters(lib):
    _, h = _gated(lib, w_gate=A.value, w_up=B_.value, w_down_t=C_.value)
    last = 64 * 128 * 2 - 16  # the last 16 bytes of a weight
    fwd, ws = lib.pi_gated_ffn_forward, vp(0x9000)
    for w in (A, B_, C_):
        p = vp(w.value + last)
        assert fwd(h, D_, 1, p, None, None, ws, 1 << 20, None) == ARG
        assert fwd(h, D_, 1, E_, p, None, ws, 1 << 20, None) == ARG
        assert fwd(h, D_, 1, E_, None, p, ws, 1 << 20, None) == ARG
        assert fwd(h, D_, 1, E_, None, None, p, 1 << 20, None) == ARG
        for at in range(4):
            out = [None] * 4
            out[at] = p
            assert lib.pi_gated_ffn_backward(h, D_, E_, F_, G_, 1, *out, pb.PI_DT_F16, 0, ws, 1 << 20, None) == ARG
    lib.pi_gated_ffn_destroy(h)

    def fwd(r=C_, u=D_, kp=E_, kr=F_):
        return lib.pi_block_norm_forward(_norm(), A, B_, 4, r, u, kp, kr, None)
    for w in (0x1000, 0x2000, 0x3000):
        assert fwd(r=vp(w)) == ARG and fwd(u=vp(w + 240)) == ARG and fwd(kp=vp(w)) == ARG and fwd(kr=vp(w)) == ARG
    assert fwd(kp=F_) == ARG and fwd(kp=C_) == ARG and fwd(kr=D_) == ARG and fwd(kr=A) == ARG

    def bwd(dx=E_, dy=F_, dwp=G_, dw=H_, dg=vp(0x300), T=4):
        return lib.pi_block_norm_backward(_norm(), A, B_, vp(0x100), vp(0x200), C_, D_, T, dx, dy, dwp, dw, dg, 0,
                                          vp(0x9000), 1 << 30, None)
    for w in (0x1000, 0x2000, 0x3000):
        p = vp(w + 240)
        assert bwd(dx=p) == ARG and bwd(dy=p) == ARG and bwd(dwp=p) == ARG and bwd(dw=p) == ARG and bwd(dg=p) == ARG
    assert bwd(dwp=H_) == ARG and bwd(dw=E_) == ARG and bwd(dg=G_) == ARG and bwd(dwp=A) == ARG and bwd(dw=D_) == ARG
    assert bwd(dx=vp(0x200)) == ARG and bwd(dw=vp(0x100)) == ARG
    assert bwd(dg=vp(0x3100), T=5) == ARG  # the gate's second row


def test_matmul_i8_calls(lib):
    qz = lib.pi_quantize_i8
    assert qz(None, 0, 4, 64, A, B_, None) == ARG and qz(A, 0, 4, 64, None, C_, None) == ARG
    assert qz(A, 3, 4, 64, B_, C_, None) == ARG and qz(A, 0, 4, 0, B_, C_, None) == ARG
    assert qz(A, 0, 4, 40, B_, C_, None) == UNSUP and qz(A, 0, -1, 64, B_, C_, None) == UNSUP
    assert qz(A, 0, 1, 131072, B_, C_, None) == UNSUP and qz(vp(8), 0, 4, 64, B_, C_, None) == ALIGN
    assert qz(A, 0, 4, 64, A, C_, None) == ARG and qz(A, 0, 4, 64, B_, vp(B_.value + 16), None) == ARG
    assert qz(None, 0, 0, 64, None, None, None) == OK
    n = C.c_size_t()
    assert lib.pi_matmul_i8_workspace_size(4, 100, 64, C.byref(n)) == OK and n.value >= 256
    assert lib.pi_matmul_i8_workspace_size(4, 100, 60, C.byref(n)) == UNSUP
    assert lib.pi_matmul_i8_workspace_size(4, 0, 64, C.byref(n)) == ARG
    assert lib.pi_matmul_i8_workspace_size(4, 100, 64, None) == ARG
    ok = [A, B_, C_, D_, None, 4, 100, 64, E_, 0, F_, 1 << 20, None]

    def mm(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return lib.pi_matmul_i8(*a)
    for i in (0, 1, 2, 3, 8):
        assert mm(**{f"_{i}": None}) == ARG
        assert mm(**{f"_{i}": vp(0x18)}) == ALIGN
    assert mm(_5=-1) == UNSUP and mm(_6=0) == ARG and mm(_7=72) == UNSUP and mm(_7=131072) == UNSUP
    assert mm(_8=A) == ARG and mm(_8=C_) == ARG and mm(_4=E_) == ARG and mm(_10=E_) == ARG
    assert mm(_9=5) == ARG and mm(_10=None) == WS and mm(_11=255) == WS and mm(_10=vp(0x18)) == ALIGN
    assert mm(_0=None, _1=None, _5=0, _8=None, _10=None) == OK


def _raises(fn, match):
    with pytest.raises(ValueError, match=match):
        fn()


def test_binding_checks(lib):
    h, b = torch.float16, torch.bfloat16
    w = torch.zeros(128, 64, dtype=h)
    _raises(lambda: pb.GatedFfnLayer(w.float(), w, w), "w_gate")
    _raises(lambda: pb.GatedFfnLayer(w, w.to(b), w), "w_up: dtype")
    _raises(lambda: pb.GatedFfnLayer(w, w, w[:64]), "w_down_t: shape")
    _raises(lambda: pb.GatedFfnLayer(w, w, torch.zeros(64, 128, dtype=h).t()), "w_down_t: must be contiguous")
    _raises(lambda: pb.GatedFfnLayer(w, w, w, act="tanh"), "act")
    layer = pb.GatedFfnLayer(w, w, w)
    u, g, ws = torch.zeros(4, 64, dtype=h), torch.zeros(4, 128, dtype=h), torch.zeros(65536, dtype=torch.uint8)
    _raises(lambda: pb.pi_gated_ffn_forward(layer, u[:, :32], u, ws), "u: shape")
    _raises(lambda: pb.pi_gated_ffn_forward(layer, u.float(), u, ws), "u: dtype")
    _raises(lambda: pb.pi_gated_ffn_forward(layer, u, u[:3], ws), "y: shape")
    _raises(lambda: pb.pi_gated_ffn_forward(layer, u, u.clone(), ws, gate=u), "gate: shape")
    _raises(lambda: pb.pi_gated_ffn_forward(layer, u, u.clone(), ws), "must be a CUDA tensor")
    back = lambda **kw: pb.pi_gated_ffn_backward(layer, u, g, g, u, ws, **kw)  # noqa: E731
    _raises(lambda: back(dw_gate=w.to(b)), r"dw_\*: dtype")
    _raises(lambda: back(dw_gate=w, dw_up=w.float()), "dw_up: dtype")
    _raises(lambda: back(du=g), "du: shape")
    _raises(lambda: back(), "must be a CUDA tensor")
    f = torch.zeros(4, 64)
    _raises(lambda: pb.BlockNorm(64, y_dtype=torch.int8), "y_dtype")
    _raises(lambda: pb.BlockNorm(64, w_pre=torch.zeros(63)), "w_pre: shape")
    _raises(lambda: pb.BlockNorm(64, gate=f), "tokens_per_gate")
    _raises(lambda: pb.BlockNorm(64, gate=torch.zeros(64), tokens_per_gate=4), "gate")
    n = pb.BlockNorm(64, y_dtype=h, u_dtype=h, gate=f[:2], tokens_per_gate=1)
    _raises(lambda: pb.pi_block_norm_forward(n, f, u, f, u), "gate: 2 rows")
    n = pb.BlockNorm(64, y_dtype=h, u_dtype=h)
    _raises(lambda: pb.pi_block_norm_forward(n, f, f, f, u), "y: dtype")
    _raises(lambda: pb.pi_block_norm_forward(n, f, u, f[:2], u), "x_out: shape")
    _raises(lambda: pb.pi_block_norm_forward(n, f, u, f, u), "must be a CUDA tensor")
    _raises(lambda: pb.pi_block_norm_backward(n, f, u, None, None, None, None, f, u, ws), "du or dx_out")
    _raises(lambda: pb.pi_block_norm_backward(n, f, u, None, f[0, :4], u, None, f, u, ws, dgate=f), "no gate")
    _raises(lambda: pb.pi_block_norm_backward(n, f, u, None, f[0, :3], u, None, f, u, ws), "rstd_pre: shape")
    q = torch.zeros(4, 64, dtype=torch.int8)
    _raises(lambda: pb.pi_quantize_i8(q, q, f[0, :4]), "x: ")
    _raises(lambda: pb.pi_quantize_i8(f, f, f[0, :4]), "q: dtype")
    _raises(lambda: pb.pi_quantize_i8(f, q, f[0, :3]), "scales: shape")
    _raises(lambda: pb.pi_quantize_i8(f, q, f[0, :4]), "must be a CUDA tensor")
    s = f[0, :4]
    _raises(lambda: pb.pi_matmul_i8(q, s, q[:, :32], s, f[:, :4], ws), "expected")
    _raises(lambda: pb.pi_matmul_i8(q, s, q, s, q[:, :4].contiguous(), ws), "y: dtype")
    _raises(lambda: pb.pi_matmul_i8(q, s, q, s, f[:, :4], ws), "y: must be contiguous")
    _raises(lambda: pb.pi_matmul_i8(q, s, q, s, torch.zeros(4, 4), ws, bias=f[0, :3]), "bias: shape")
    _raises(lambda: pb.pi_matmul_i8(q, s, q, s, torch.zeros(4, 4), ws), "must be a CUDA tensor")


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_plain_gradients_agree_with_automatic_differentiation(act):
    gen = torch.Generator().manual_seed(0)
    u, wg, wu, wd = (torch.randn(*s, generator=gen, dtype=ref.D) for s in ((5, 8), (16, 8), (16, 8), (16, 8)))
    dy = torch.randn(5, 8, generator=gen, dtype=ref.D)
    ts = [t.requires_grad_() for t in (u, wg, wu, wd)]
    y, g, p, _ = ref.ffn_forward(act, *ts)
    want = torch.autograd.grad((y * dy).sum(), ts)
    got = ref.ffn_backward(act, u, g, p, dy, wg, wu, wd)[:4]
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)


def test_plain_quantiser_is_the_definition():
    x = torch.tensor([[1.0, -0.5, 0.25, 0.0], [0, 0, 0, 0], [2.0, float("inf"), 0, 1], [127, 63.5, -62.5, 0.5]])
    q, s = ref.quantize(x)
    assert q.tolist() == [[127, -64, 32, 0], [0, 0, 0, 0], [0, 0, 0, 0], [127, 64, -62, 0]]
    assert s[1] == 0 and torch.isnan(s[2]) and s[3] == 1
