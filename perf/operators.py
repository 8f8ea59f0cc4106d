"""Workloads of the dense block operators: the gated feed-forward block with
its gradients, the fused norms around a block with their gradients, and the
8-bit integer product with a scale per token and per output channel.

``run`` computes an operator in its plain form (elementary torch operations in
fp32, rounded once at the end), or, where ``own`` is true, by the calls that a
user makes of this framework.  ``exact`` evaluates the definitions in fp64.

Shapes are those of the framework's FFN layers (d_model x d_ffn: 4096 x 16384,
5120 x 13824, 7168 x 28672, 8192 x 28672) or generic, odd and ragged ones.
"""
import math

import torch

own = False

HALF = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def _ffn(name, tokens, d, f, dtype, act, op="ffn_fwd", save=False):
    return {"name": name, "op": op, "tokens": tokens, "d": d, "f": f, "dtype": dtype, "act": act, "save": save}


def _norm(name, op, tokens, d, y_dtype, u_dtype, post, tokens_per_gate):
    return {"name": name, "op": op, "tokens": tokens, "d": d, "y_dtype": y_dtype, "u_dtype": u_dtype, "post": post,
            "tokens_per_gate": tokens_per_gate}


def _i8(name, tokens, k, n, dtype, out, bias):
    return {"name": name, "op": "i8", "tokens": tokens, "k": k, "n": n, "dtype": dtype, "out": out, "bias": bias}


def listed():
    return [
        # decode, between two layers of a stack: residual add and the next layer's norm of one token
        _norm("norm_fwd_1tok", "norm_fwd", 1, 8192, "f32", "f16", False, 0),
        # prompt of 8 sequences: post-norm, a gate row per sequence, residual add, pre-norm
        _norm("norm_fwd_8k", "norm_fwd", 8192, 5120, "bf16", "bf16", True, 1024),
        # training step: the gradients of the same, one gate for all tokens
        _norm("norm_bwd_4k", "norm_bwd", 4096, 7168, "bf16", "bf16", True, 4096),
        # ragged: short sequences of an odd length, a small odd width
        _norm("norm_bwd_ragged", "norm_bwd", 777, 1000, "f16", "f16", True, 111),
        # one token through a dense layer (all neurons): the serving form
        _ffn("ffn_fwd_1tok", 1, 5120, 13824, "f16", "silu"),
        # a decode batch of an odd size, ReLU gate
        _ffn("ffn_fwd_45tok", 45, 4096, 16384, "f16", "relu"),
        # a prompt through the largest layer
        _ffn("ffn_fwd_prompt", 2048, 8192, 28672, "bf16", "silu"),
        # a training step's forward pass: the pre-activations are kept for the backward pass
        _ffn("ffn_fwd_train", 4096, 5120, 13824, "bf16", "silu", save=True),
        # its backward pass: the gradients of the input and of the three matrices
        _ffn("ffn_bwd_train", 4096, 5120, 13824, "bf16", "silu", op="ffn_bwd"),
        # fine-tuning on one short sequence of a small odd-sized layer
        _ffn("ffn_bwd_ragged", 333, 1032, 2760, "f16", "gelu", op="ffn_bwd"),
        # one token through an 8-bit up projection: the serving form
        _i8("i8_1tok", 1, 8192, 28672, "f16", "f32", False),
        # a prompt through an 8-bit projection with a bias, an odd number of tokens
        _i8("i8_prompt", 2011, 5120, 13824, "bf16", "bf16", True),
    ]


def _log_int(rng, lo, hi, multiple=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / multiple)) * multiple))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "ffn_fwd", "ffn_fwd", "ffn_bwd", "i8", "i8"])
    dtype = rng.choice(["f16", "bf16"])
    if op in ("norm_fwd", "norm_bwd"):
        d = _log_int(rng, 64, 16384, 8)
        tokens = _log_int(rng, 1, min(16384, 42_000_000 // d))
        per = rng.choice([0, tokens, 1, _log_int(rng, 1, tokens)])
        y_dtype, u_dtype = rng.choice([(dtype, dtype), ("f32", dtype), ("f32", "f32")])
        c = _norm("", op, tokens, d, y_dtype, u_dtype, rng.random() < 0.7, per)
    elif op == "i8":
        k, n = _log_int(rng, 64, 14336, 16), _log_int(rng, 64, 28672)
        tokens = _log_int(rng, 1, 4096)
        c = _i8("", tokens, k, n, dtype, rng.choice([dtype, "f32"]), rng.random() < 0.5)
    else:
        d, f = _log_int(rng, 256, 8192, 8), _log_int(rng, 512, 28672, 8)
        most = (2048 * 8192 * 28672) // (d * f) // (2 if op == "ffn_bwd" else 1)
        tokens = _log_int(rng, 1, max(1, min(8192, most)))
        c = _ffn("", tokens, d, f, dtype, rng.choice(["silu", "silu", "relu", "gelu"]), op,
                 op == "ffn_fwd" and rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": case, "op": case["op"]}
    T = case["tokens"]
    if case["op"] in ("norm_fwd", "norm_bwd"):
        d, yt, ut = case["d"], HALF[case["y_dtype"]], HALF[case["u_dtype"]]
        # the residual stream has grown over the layers below; the block's output is of another size
        s["x"] = normal(T, d, std=3.0)
        s["y"] = normal(T, d, std=0.5, dtype=yt)
        s["w_pre"] = 1.0 + normal(d, std=0.1)
        s["w_post"] = 1.0 + normal(d, std=0.1) if case["post"] else None
        per = case["tokens_per_gate"]
        s["gate"] = normal(-(-T // per), d, std=0.5) if per else None
        s["scales"] = (1.0, 0.7)  # of the residual stream and of the block's output
        s["eps"] = 1e-6
        if case["op"] == "norm_bwd":
            # what a training program has from the forward pass: the new stream and the norms' factors
            s["x"], _, s["r_post"], s["r_pre"] = _norm_forward(s)
            s["du"] = normal(T, d, std=0.3, dtype=ut)
            s["dx_out"] = normal(T, d, std=0.2)
    elif case["op"] == "i8":
        k, n = case["k"], case["n"]
        # activations have a few large channels; weights are quantised once, per output channel
        channel = torch.exp(0.8 * torch.randn(k, generator=g, device="cuda"))
        s["x"] = (torch.randn(T, k, generator=g, device="cuda") * channel).to(HALF[case["dtype"]])
        w = normal(n, k, std=0.02)
        s["ws"] = w.abs().amax(1) / 127.0
        s["wq"] = torch.round(w / s["ws"][:, None]).to(torch.int8)
        s["bias"] = normal(n, std=0.1) if case["bias"] else None
    else:
        d, f, t = case["d"], case["f"], HALF[case["dtype"]]
        s["u"] = normal(T, d, dtype=t)  # a normalised input
        s["wg"], s["wu"], s["wd"] = (normal(f, d, std=0.02, dtype=t) for _ in range(3))
        if case["op"] == "ffn_bwd":
            # what the forward pass has kept, and the gradient of the block's output
            s["gate"], s["up"] = s["u"] @ s["wg"].t(), s["u"] @ s["wu"].t()
            s["dy"] = normal(T, d, std=0.5, dtype=t)
    if own:
        _handles(s, case)
    return s


def _handles(s, case):
    """The handle, workspace and output buffers that a user's program keeps."""
    from activation_sparse_decode_gemv_b200 import binding as pb
    T = case["tokens"]

    def out(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if case["op"] in ("norm_fwd", "norm_bwd"):
        d, yt, ut = case["d"], HALF[case["y_dtype"]], HALF[case["u_dtype"]]
        s["norm"] = pb.BlockNorm(d, y_dtype=yt, u_dtype=ut, eps=s["eps"], residual_scale=s["scales"][0],
                                 branch_scale=s["scales"][1], post_norm=case["post"], w_post=s["w_post"],
                                 w_pre=s["w_pre"], gate=s["gate"], tokens_per_gate=case["tokens_per_gate"])
        if case["op"] == "norm_fwd":
            s["out"] = (out(T, d, dtype=torch.float32), out(T, d, dtype=ut),
                        out(T, dtype=torch.float32) if case["post"] else None, out(T, dtype=torch.float32))
        else:
            s["ws"] = pb.make_block_norm_workspace(s["norm"], T)
            s["out"] = (out(T, d, dtype=torch.float32), out(T, d, dtype=yt),
                        out(d, dtype=torch.float32) if case["post"] else None, out(d, dtype=torch.float32),
                        None if s["gate"] is None else torch.empty_like(s["gate"]))
    elif case["op"] == "i8":
        s["q"], s["qs"] = out(T, case["k"], dtype=torch.int8), out(T, dtype=torch.float32)
        s["work"] = pb.make_matmul_i8_workspace(T, case["n"], case["k"])
        s["out"] = out(T, case["n"], dtype=HALF[case["out"]])
    else:
        d, f, t = case["d"], case["f"], HALF[case["dtype"]]
        back = case["op"] == "ffn_bwd"
        s["layer"] = pb.GatedFfnLayer(s["wg"], s["wu"], s["wd"], act=case["act"])
        s["ws"] = pb.make_gated_ffn_workspace(s["layer"], T, backward=back)
        if back:
            s["out"] = (out(T, d, dtype=t), out(f, d, dtype=t), out(f, d, dtype=t), out(f, d, dtype=t))
        else:
            s["out"] = (out(T, d, dtype=t),) + ((out(T, f, dtype=t), out(T, f, dtype=t)) if case["save"] else ())


# ---------------------------------------------------------------- plain forms
def _act(name, g):
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "relu":
        return torch.clamp_min(g, 0.0)
    return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))


def _act_grad(name, g):
    if name == "silu":
        p = torch.sigmoid(g)
        return p * (1.0 + g * (1.0 - p))
    if name == "relu":
        return (g > 0).to(g.dtype)
    return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)


def _ffn_forward(s):
    t, u = s["u"].dtype, s["u"].float()
    g, p = u @ s["wg"].float().t(), u @ s["wu"].float().t()
    y = (_act(s["case"]["act"], g) * p) @ s["wd"].float()
    return (y.to(t), g.to(t), p.to(t)) if s["case"]["save"] else (y.to(t),)


def _ffn_backward(s):
    t, act = s["u"].dtype, s["case"]["act"]
    u, g, p, dy = s["u"].float(), s["gate"].float(), s["up"].float(), s["dy"].float()
    a = _act(act, g)
    da = dy @ s["wd"].float().t()
    dp = da * a
    dg = da * p * _act_grad(act, g)
    du = dg @ s["wg"].float() + dp @ s["wu"].float()
    return du.to(t), (dg.t() @ u).to(t), (dp.t() @ u).to(t), ((a * p).t() @ dy).to(t)


def _gate_rows(s):
    """The gate row of each token: row t // tokens_per_gate."""
    T, per = s["case"]["tokens"], s["case"]["tokens_per_gate"]
    return torch.arange(T, device="cuda") // per


def _norm_forward(s):
    x, y = s["x"], s["y"].float()
    r_post = None
    if s["case"]["post"]:
        r_post = torch.rsqrt((y * y).mean(1) + s["eps"])
        y = y * r_post[:, None] * s["w_post"]
    if s["gate"] is not None:
        y = y * s["gate"][_gate_rows(s)]
    r = s["scales"][0] * x + s["scales"][1] * y
    r_pre = torch.rsqrt((r * r).mean(1) + s["eps"])
    u = (r * r_pre[:, None] * s["w_pre"]).to(HALF[s["case"]["u_dtype"]])
    return r, u, r_post, r_pre


def _norm_backward(s):
    r, y, du, d = s["x"], s["y"].float(), s["du"].float(), s["case"]["d"]
    n = r * s["r_pre"][:, None]
    dw_pre = (du * n).sum(0)
    dn = du * s["w_pre"]
    dr = s["dx_out"] + s["r_pre"][:, None] * (dn - n * (dn * n).sum(1, keepdim=True) / d)
    m = y * s["r_post"][:, None] if s["case"]["post"] else y
    b = m * s["w_post"] if s["case"]["post"] else m
    db = s["scales"][1] * dr
    dgate = None
    if s["gate"] is not None:
        rows = _gate_rows(s)
        dgate = torch.zeros_like(s["gate"]).index_add_(0, rows, db * b)
        db = db * s["gate"][rows]
    dw_post = None
    if s["case"]["post"]:
        dw_post = (db * m).sum(0)
        db = db * s["w_post"]
        db = s["r_post"][:, None] * (db - m * (db * m).sum(1, keepdim=True) / d)
    return s["scales"][0] * dr, db.to(s["y"].dtype), dw_post, dw_pre, dgate


def _i8_product(s):
    x = s["x"].float()
    xs = x.abs().amax(1)
    xs = xs / torch.full_like(xs, 127.0)  # a tensor: by a number, torch multiplies with its rounded inverse
    q = torch.clamp(torch.round(torch.nan_to_num(x / xs[:, None])), -127, 127)
    y = (q @ s["wq"].float().t()) * xs[:, None] * s["ws"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(HALF[s["case"]["out"]])


# ---------------------------------------------------------------- one pass
def run(s):
    if not own:
        return {"norm_fwd": _norm_forward, "norm_bwd": _norm_backward, "ffn_fwd": _ffn_forward,
                "ffn_bwd": _ffn_backward, "i8": _i8_product}[s["op"]](s)
    from activation_sparse_decode_gemv_b200 import binding as pb
    out = s["out"]
    if s["op"] == "norm_fwd":
        pb.pi_block_norm_forward(s["norm"], s["x"], s["y"], out[0], out[1], rstd_post=out[2], rstd_pre=out[3])
    elif s["op"] == "norm_bwd":
        pb.pi_block_norm_backward(s["norm"], s["x"], s["y"], s["r_post"], s["r_pre"], s["du"], s["dx_out"], out[0],
                                  out[1], s["ws"], dw_post=out[2], dw_pre=out[3], dgate=out[4])
    elif s["op"] == "ffn_fwd":
        keep = {"gate": out[1], "up": out[2]} if s["case"]["save"] else {}
        pb.pi_gated_ffn_forward(s["layer"], s["u"], out[0], s["ws"], **keep)
    elif s["op"] == "ffn_bwd":
        pb.pi_gated_ffn_backward(s["layer"], s["u"], s["gate"], s["up"], s["dy"], s["ws"], du=out[0], dw_gate=out[1],
                                 dw_up=out[2], dw_down_t=out[3])
    else:
        pb.pi_quantize_i8(s["x"], s["q"], s["qs"])
        pb.pi_matmul_i8(s["q"], s["qs"], s["wq"], s["ws"], out, s["work"], bias=s["bias"])
    return out


def work(case):
    T, size = case["tokens"], {"f16": 2, "bf16": 2, "f32": 4}
    if case["op"] in ("norm_fwd", "norm_bwd"):
        d, yb, ub = case["d"], size[case["y_dtype"]], size[case["u_dtype"]]
        per, post = case["tokens_per_gate"], case["post"]
        gate = 4 * d * -(-T // per) if per else 0
        params, stats = 4 * d * (2 if post else 1), 4 * T * (2 if post else 1)
        if case["op"] == "norm_fwd":  # x, y in; the new stream, u and the factors out
            return {"bytes": T * d * (4 + yb + 4 + ub) + params + gate + stats, "flops": 10 * T * d}
        # stream, y, du and its stream gradient in; dx and dy out; gradients of the weights and the gate
        return {"bytes": T * d * (4 + yb + ub + 4 + 4 + yb) + 2 * params + 2 * gate + stats, "flops": 25 * T * d}
    if case["op"] == "i8":
        k, n = case["k"], case["n"]
        return {"bytes": T * k * 2 + n * k + 4 * n * (2 if case["bias"] else 1) + T * n * size[case["out"]],
                "flops": 2 * T * k * n}
    d, f = case["d"], case["f"]
    if case["op"] == "ffn_fwd":
        return {"bytes": 2 * (3 * d * f + 2 * T * d + (2 * T * f if case["save"] else 0)), "flops": 6 * T * d * f}
    return {"bytes": 2 * (6 * d * f + 3 * T * d + 2 * T * f), "flops": 12 * T * d * f}


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    phi = {"silu": lambda z: z / (1 + torch.exp(-z)), "relu": lambda z: torch.where(z > 0, z, torch.zeros_like(z)),
           "gelu": lambda z: z * (1 - torch.special.erfc(z / math.sqrt(2)) / 2)}
    if case["op"] == "ffn_fwd":
        g = torch.einsum("td,fd->tf", s["u"].to(D), s["wg"].to(D))
        p = torch.einsum("td,fd->tf", s["u"].to(D), s["wu"].to(D))
        y = torch.einsum("tf,fd->td", phi[case["act"]](g) * p, s["wd"].to(D))
        return (y, g, p) if case["save"] else (y,)
    if case["op"] == "ffn_bwd":
        # y = sum_f phi(g) p W_f; the slope of phi in closed form
        slope = {"silu": lambda z: 1 / (1 + torch.exp(-z)) + z * torch.exp(-z) / (1 + torch.exp(-z)) ** 2,
                 "relu": lambda z: torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z)),
                 "gelu": lambda z: 1 - torch.special.erfc(z / math.sqrt(2)) / 2
                 + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)}
        g, p, u, dy = (s[k].to(D) for k in ("gate", "up", "u", "dy"))
        back = torch.einsum("td,fd->tf", dy, s["wd"].to(D))
        along_g, along_p = back * slope[case["act"]](g) * p, back * phi[case["act"]](g)
        du = torch.einsum("tf,fd->td", along_g, s["wg"].to(D)) + torch.einsum("tf,fd->td", along_p, s["wu"].to(D))
        return (du, torch.einsum("tf,td->fd", along_g, u), torch.einsum("tf,td->fd", along_p, u),
                torch.einsum("tf,td->fd", phi[case["act"]](g) * p, dy))
    if case["op"] == "i8":
        # by definition the stored scale and the quotient are fp32; ties of the quotient go to even
        x = s["x"].to(D)
        scale = (s["x"].to(D).abs().max(dim=1).values / 127).to(torch.float32).to(D)
        ratio = (x / scale[:, None]).to(torch.float32).to(D)
        code = torch.where(scale[:, None] > 0, ratio.round(), torch.zeros_like(x))
        y = torch.einsum("tk,nk->tn", code, s["wq"].to(D)) * scale[:, None] * s["ws"].to(D)[None]
        return y if s["bias"] is None else y + s["bias"].to(D)
    T, d = case["tokens"], case["d"]
    one = torch.ones((), dtype=D, device="cuda")
    y = s["y"].to(D)
    w_pre = s["w_pre"].to(D)
    w_post = s["w_post"].to(D) if case["post"] else one
    per = case["tokens_per_gate"]
    gate = s["gate"].to(D).repeat_interleave(per, 0)[:T] if per else one
    alpha, beta = s["scales"]
    if case["op"] == "norm_fwd":
        k_post = 1 / torch.sqrt(y.pow(2).sum(1) / d + s["eps"]) if case["post"] else None
        branch = y if k_post is None else y * k_post[:, None] * w_post
        r = alpha * s["x"].to(D) + beta * gate * branch
        k_pre = 1 / torch.sqrt(r.pow(2).sum(1) / d + s["eps"])
        return r, r * k_pre[:, None] * w_pre, k_post, k_pre
    r, du = s["x"].to(D), s["du"].to(D)
    k_pre = s["r_pre"].to(D)[:, None]
    # d/dr of r k(r): k (I - k^2 r r^T / d), applied to w_pre * du
    v = w_pre * du
    dr = s["dx_out"].to(D) + k_pre * v - k_pre ** 3 * r * (v * r).sum(1, keepdim=True) / d
    k_post = s["r_post"].to(D)[:, None] if case["post"] else one
    unit = y * k_post
    dgate = None
    if per:
        rows = beta * dr * unit * w_post
        pad = torch.zeros(s["gate"].shape[0] * per - T, d, dtype=D, device="cuda")
        dgate = torch.cat([rows, pad]).view(-1, per, d).sum(1)
    v = beta * dr * gate
    dw_post = None
    if case["post"]:
        dw_post = (v * unit).sum(0)
        v = v * w_post
        v = k_post * v - k_post ** 3 * y * (v * y).sum(1, keepdim=True) / d
    return alpha * dr, v, dw_post, (du * r * k_pre).sum(0), dgate
