"""The operators around the attention of a transformer block, as they are measured.

    linear      y = act(x W + b) + r, forward (with the pre-activation kept for training) and backward
    out_proj    the same product read straight from attention's [B, H, N, d_k] output, and its backward
    linear_q8   the product of e4m3 rows with e4m3 weights, scales, bias, activation and residual
    rms_norm    h = x + r, y = h / rms(h) * g, forward and backward
    rms_norm_q8 the same with y in e4m3 and one scale a row

`run` computes them with elementary torch operations in 32 bits, rounded once at the end; with
`own` set it calls self_attention_gb300 instead.  Matrices are bf16 (or e4m3 with fp32 scales),
vectors (bias, norm weight, scales, 1/rms) fp32.
"""
import math

import torch

own = False

EPS = 1e-6
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
Q8_MAX = 448.0       # the largest e4m3 value
AMAX_FLOOR = 1e-30   # a row of zeros gets the scale of this


# ------------------------------------------------------------------ cases
def listed():
    return [
        # serving, one token: the up projection of a 16 x 128 head model (long text); weight streaming
        {"name": "linear one token", "op": "linear", "M": 1, "K": 2048, "N": 8192, "act": "silu",
         "bias": True, "res": False, "keep_z": False},
        # training, high-resolution ViT-L (8 x 4096 tokens, D = 1024): the MLP's up projection
        {"name": "linear vit-l up", "op": "linear", "M": 32768, "K": 1024, "N": 4096, "act": "gelu",
         "bias": True, "res": False, "keep_z": True},
        # its backward pass
        {"name": "linear bwd vit-l up", "op": "linear_bwd", "M": 32768, "K": 1024, "N": 4096, "act": "gelu",
         "bias": True},
        # a short ragged batch with odd widths
        {"name": "linear bwd ragged", "op": "linear_bwd", "M": 1111, "K": 1000, "N": 520, "act": "silu",
         "bias": True},
        # one 224 x 224 image, ViT-B: attention's output projection added to the residual stream
        {"name": "out_proj one image", "op": "out_proj", "B": 1, "H": 12, "T": 196, "d": 64, "N": 768,
         "bias": True, "res": True},
        # the backward of the same projection over the ViT-B attention block's batch
        {"name": "out_proj bwd vit-b", "op": "out_proj_bwd", "B": 32, "H": 12, "T": 576, "d": 64, "N": 768,
         "bias": True},
        # serving in 8 bits: one token, and a prompt of 2 x 16384 tokens (long text)
        {"name": "linear_q8 one token", "op": "linear_q8", "M": 1, "K": 8192, "N": 2048, "act": "none",
         "bias": False, "res": True},
        {"name": "linear_q8 long text", "op": "linear_q8", "M": 32768, "K": 2048, "N": 8192, "act": "gelu_tanh",
         "bias": True, "res": False},
        # the norm ahead of attention, high-resolution ViT-L, and its backward over the ViT-B batch
        {"name": "rms_norm vit-l", "op": "rms_norm", "M": 32768, "D": 1024, "res": True},
        {"name": "rms_norm bwd vit-b", "op": "rms_norm_bwd", "M": 18432, "D": 768, "res": True},
        # the norm that feeds the 8-bit product: a few sequences' next tokens, and the long prompt
        {"name": "rms_norm_q8 decode", "op": "rms_norm_q8", "M": 7, "D": 2048, "res": True},
        {"name": "rms_norm_q8 long text", "op": "rms_norm_q8", "M": 32768, "D": 2048, "res": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_bwd", "out_proj", "out_proj_bwd", "linear_q8", "rms_norm",
                     "rms_norm_bwd", "rms_norm_q8"))
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("out_proj", "out_proj_bwd"):
        d = rng.choice((64, 128))
        H, B = rng.randint(2, 16 if d == 64 else 8), rng.randint(1, 32)
        T = _log_int(rng, 1, max(2, min(4096, 32768 // B)))
        c = {"op": op, "B": B, "H": H, "T": T, "d": d, "N": 8 * _log_int(rng, 12, 128), "bias": flag()}
        if op == "out_proj":
            c["res"] = flag()
        return c
    if op.startswith("rms_norm"):
        return {"op": op, "M": _log_int(rng, 1, 32768), "D": 8 * _log_int(rng, 8, 256), "res": flag()}
    step = 16 if op == "linear_q8" else 8
    c = {"op": op, "M": _log_int(rng, 1, 32768), "K": step * _log_int(rng, 64 // step, 4096 // step),
         "N": step * _log_int(rng, 64 // step, 4096 // step), "act": rng.choice(ACTS), "bias": flag()}
    if op == "linear_bwd":   # two products: half the rows
        c["M"] = min(c["M"], 16384)
    else:
        c["res"] = flag()
    if op == "linear":
        c["keep_z"] = c["act"] != "none" and flag()
    return c


# ------------------------------------------------------------------ inputs
def _q8(x):
    """Rows of x as e4m3 and the scale of each."""
    s = x.float().abs().amax(-1).clamp_min(AMAX_FLOOR)
    q = (x.float() * (Q8_MAX / s).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q, s / Q8_MAX


def prepare(case, seed):
    c = dict(case)
    op = c["op"]
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": c}
    if op in ("linear", "linear_bwd"):
        M, K, N = c["M"], c["K"], c["N"]
        s["x"] = randn(M, K)
        s["w"] = randn(K, N, std=K ** -0.5)
        if op == "linear":
            s["bias"] = randn(N, std=0.5, dtype=torch.float32) if c["bias"] else None
            s["res"] = randn(M, N) if c["res"] else None
        else:
            s["z"] = randn(M, N) if c["act"] != "none" else None   # what the forward kept
            s["dy"] = randn(M, N)
    elif op in ("out_proj", "out_proj_bwd"):
        B, H, T, d, N = c["B"], c["H"], c["T"], c["d"], c["N"]
        s["o"] = randn(B, H, T, d, std=0.5)
        s["w"] = randn(H * d, N, std=(H * d) ** -0.5)
        if op == "out_proj":
            s["bias"] = randn(N, std=0.5, dtype=torch.float32) if c["bias"] else None
            s["res"] = randn(B, T, N) if c["res"] else None
        else:
            s["dy"] = randn(B, T, N)
    elif op == "linear_q8":
        M, K, N = c["M"], c["K"], c["N"]
        s["xq"], s["xs"] = _q8(randn(M, K))
        s["wq"], s["ws"] = _q8(randn(N, K, std=K ** -0.5))   # [N, K]: one scale an output column
        s["bias"] = randn(N, std=0.5, dtype=torch.float32) if c["bias"] else None
        s["res"] = randn(M, N) if c["res"] else None
    else:
        M, D = c["M"], c["D"]
        s["g"] = 1.0 + randn(D, std=0.1, dtype=torch.float32)
        if op == "rms_norm_bwd":
            s["h"] = randn(M, D)
            s["rstd"] = torch.rsqrt(s["h"].double().square().mean(-1) + EPS).float()
            s["dy"] = randn(M, D)
            s["dh"] = randn(M, D) if c["res"] else None
        else:
            s["x"] = randn(M, D)
            s["res"] = randn(M, D) if c["res"] else None
    return s


# ------------------------------------------------------------------ the plain forms
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * (0.5 ** 0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * (0.5 ** 0.5))) + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    if act == "gelu_tanh":
        c = (2.0 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _plain_linear(x, w, bias, res, act, keep_z):
    z = x.float() @ w.float()
    if bias is not None:
        z = z + bias
    y = _act(z, act)
    if res is not None:
        y = y + res.float()
    y = y.to(torch.bfloat16)
    return (y, z.to(torch.bfloat16)) if keep_z else (y,)


def _plain_linear_bwd(x, w, dy, z, act, bias):
    dz = dy.float()
    if z is not None:
        dz = dz * _act_slope(z.float(), act)
    dx = (dz @ w.float().t()).to(torch.bfloat16)
    dw = (x.float().t() @ dz).to(torch.bfloat16)
    return (dx, dw, dz.sum(0)) if bias else (dx, dw)


def _plain_norm(x, res, g):
    h = x.float() if res is None else x.float() + res.float()
    rstd = torch.rsqrt(h.square().mean(-1) + EPS)
    return h, rstd, h * rstd.unsqueeze(-1) * g


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "linear":
        return _plain_linear(s["x"], s["w"], s["bias"], s["res"], c["act"], c["keep_z"])
    if op == "linear_bwd":
        return _plain_linear_bwd(s["x"], s["w"], s["dy"], s["z"], c["act"], c["bias"])
    if op == "out_proj":
        x = s["o"].transpose(1, 2).reshape(c["B"], c["T"], -1)
        return _plain_linear(x, s["w"], s["bias"], s["res"], "none", False)
    if op == "out_proj_bwd":
        B, H, T, d = c["B"], c["H"], c["T"], c["d"]
        x = s["o"].transpose(1, 2).reshape(B * T, H * d)
        out = _plain_linear_bwd(x, s["w"], s["dy"].view(B * T, -1), None, "none", c["bias"])
        return (out[0].view(B, T, H, d).transpose(1, 2).contiguous(),) + tuple(out[1:])
    if op == "linear_q8":
        z = s["xq"].float() @ s["wq"].float().t()
        z = z * s["xs"].unsqueeze(1) * s["ws"]
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(z, c["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return (y.to(torch.bfloat16),)
    if op == "rms_norm":
        h, rstd, y = _plain_norm(s["x"], s["res"], s["g"])
        out = (y.to(torch.bfloat16), rstd)
        return out + (h.to(torch.bfloat16),) if c["res"] else out
    if op == "rms_norm_q8":
        h, _, y = _plain_norm(s["x"], s["res"], s["g"])
        a = y.abs().amax(-1).clamp_min(AMAX_FLOOR)
        out = ((y * (Q8_MAX / a).unsqueeze(-1)).to(torch.float8_e4m3fn), a / Q8_MAX)
        return out + (h.to(torch.bfloat16),) if c["res"] else out
    # rms_norm_bwd
    xhat = s["h"].float() * s["rstd"].unsqueeze(-1)
    dy = s["dy"].float()
    t = dy * s["g"]
    dx = s["rstd"].unsqueeze(-1) * (t - xhat * (t * xhat).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(torch.bfloat16), (dy * xhat).sum(0)


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    import self_attention_gb300 as sa
    c = s["case"]
    op = c["op"]
    if op == "linear":
        out = sa.linear_forward(s["x"], s["w"], s["bias"], s["res"], c["act"], keep_z=c["keep_z"])
        return out if c["keep_z"] else (out,)
    if op == "linear_bwd":
        dx, dw, db = sa.linear_backward(s["x"], s["w"], s["dy"], s["z"], c["act"], bias=c["bias"])
        return (dx, dw, db) if c["bias"] else (dx, dw)
    if op == "out_proj":
        return (sa.out_proj_forward(s["o"], s["w"], s["bias"], s["res"]),)
    if op == "out_proj_bwd":
        do, dw, db = sa.out_proj_backward(s["o"], s["w"], s["dy"], bias=c["bias"])
        return (do, dw, db) if c["bias"] else (do, dw)
    if op == "linear_q8":
        return (sa.linear_q8(s["xq"], s["xs"], s["wq"], s["ws"], s["bias"], s["res"], c["act"]),)
    if op == "rms_norm":
        y, h, rstd = sa.rms_norm_forward(s["x"], s["g"], s["res"], EPS)
        return (y, rstd, h) if c["res"] else (y, rstd)
    if op == "rms_norm_q8":
        q, scale, h = sa.rms_norm_q8(s["x"], s["g"], s["res"], EPS)
        return (q, scale, h) if c["res"] else (q, scale)
    return sa.rms_norm_backward(s["dy"], s["h"], s["g"], s["rstd"], s["dh"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ work
def work(case):
    c = dict(case)
    op = c["op"]
    if op in ("out_proj", "out_proj_bwd"):
        c.update(M=c["B"] * c["T"], K=c["H"] * c["d"], act="none")
    if op.startswith("rms_norm"):
        n = c["M"] * c["D"]
        if op == "rms_norm_bwd":
            return {"bytes": 2 * n * (4 if c["res"] else 3) + 4 * c["M"] + 8 * c["D"], "flops": 8 * n}
        out = 1 if op == "rms_norm_q8" else 2
        return {"bytes": n * (out + (6 if c["res"] else 2)) + 4 * c["M"] + 4 * c["D"], "flops": 5 * n}
    M, K, N = c["M"], c["K"], c["N"]
    if op in ("linear", "out_proj"):
        b = 2 * (M * K + K * N + M * N) + 4 * N * c["bias"] + 2 * M * N * (c["res"] + c.get("keep_z", False))
        return {"bytes": b, "flops": 2 * M * K * N}
    if op == "linear_q8":
        b = M * K + K * N + 4 * (M + N) + 2 * M * N * (1 + c["res"]) + 4 * N * c["bias"]
        return {"bytes": b, "flops": 2 * M * K * N}
    kept = c["act"] != "none"
    b = 2 * (2 * M * K + 2 * K * N + M * N * (2 if kept else 1)) + 4 * N * c["bias"]
    return {"bytes": b, "flops": 4 * M * K * N}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _exact_f(z, act):
    """act and its derivative, each from its own formula."""
    if act == "relu":
        return z.clamp_min(0.0), torch.heaviside(z, torch.zeros_like(z))
    if act == "gelu":
        return z * _phi(z), _phi(z) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        k, a = math.sqrt(2.0 / math.pi), 0.044715
        p = torch.sigmoid(2.0 * k * (z + a * z ** 3))       # (1 + tanh u) / 2 = sigmoid(2 u)
        return z * p, p + z * p * (1.0 - p) * 2.0 * k * (1.0 + 3.0 * a * z ** 2)
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1.0 - p)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    f = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in s.items()}
    if op in ("linear", "out_proj", "linear_q8"):
        if op == "linear_q8":
            x, w = f["xq"] * f["xs"][:, None], (f["wq"] * f["ws"][:, None]).T
        elif op == "out_proj":
            x, w = torch.einsum("bhtd->bthd", f["o"]).flatten(2), f["w"]
        else:
            x, w = f["x"], f["w"]
        z = torch.matmul(x, w)
        if f["bias"] is not None:
            z += f["bias"]
        y = _exact_f(z, c.get("act", "none"))[0]
        if f["res"] is not None:
            y = y + f["res"]
        return [y, z] if c.get("keep_z") else [y]
    if op == "linear_bwd":
        dz = f["dy"] if f["z"] is None else f["dy"] * _exact_f(f["z"], c["act"])[1]
        out = [torch.einsum("mn,kn->mk", dz, f["w"]), torch.einsum("mk,mn->kn", f["x"], dz)]
        return out + [torch.einsum("mn->n", dz)] if c["bias"] else out
    if op == "out_proj_bwd":
        w = f["w"].view(c["H"], c["d"], -1)
        do = torch.einsum("btn,hdn->bhtd", f["dy"], w)
        dw = torch.einsum("bhtd,btn->hdn", f["o"], f["dy"]).flatten(0, 1)
        return [do, dw, f["dy"].sum((0, 1))] if c["bias"] else [do, dw]
    if op == "rms_norm_bwd":
        D, r = c["D"], f["rstd"][:, None]
        u = f["dy"] * f["g"]
        dx = r * u - f["h"] * r ** 3 * (u * f["h"]).sum(1, keepdim=True) / D
        if f["dh"] is not None:
            dx = dx + f["dh"]
        return [dx, torch.einsum("md,md,m->d", f["dy"], f["h"], f["rstd"])]
    h = f["x"] if f["res"] is None else f["x"] + f["res"]
    rms = ((h ** 2).sum(1) / c["D"] + EPS).sqrt()
    y = h / rms[:, None] * f["g"]
    if op == "rms_norm":
        return [y, 1.0 / rms, h] if c["res"] else [y, 1.0 / rms]
    scale = torch.clamp(y.abs().max(1).values, min=AMAX_FLOOR) / Q8_MAX
    q = y / scale[:, None]            # before its rounding to 8 bits
    return [q, scale, h] if c["res"] else [q, scale]
