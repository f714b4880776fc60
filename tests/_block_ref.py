"""Plain 64-bit implementations of the linear layers and the norm, with the error bounds the GPU
tests hold the kernels to.  Written from the formulas, on whatever device the tensors are on.

Bounds, per element.  u8 = 2^-8 is half a bf16 step relative to the value; a sum of n products in
fp32, in any order and with each addition off by up to a whole step (2^-23: tensor cores may
truncate), is off by at most (n + 8) 2^-23 times the sum of the products' magnitudes.  The
activations' slopes are at most 1.13 in magnitude, and their own fp32 evaluation is off by at most
2^-20 (|z| + 1) (a few fp32 operations, and 1.5e-7 from the approximation of the normal
distribution function); the slopes' by 2^-19 (1 + |z|) likewise.
"""
import math

import torch

U8 = 2.0 ** -8
STEP = 2.0 ** -23
SLOPE = 1.13
Q8_MAX, AMAX_FLOOR = 448.0, 1e-30
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def act(z, name):
    if name == "relu":
        return torch.relu(z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    return torch.ones_like(z)


def linear(x, w, bias=None, residual=None, name="none"):
    """(y, z, tolerance of y, tolerance of z) for 2-D x."""
    x, w = x.double(), w.double()
    z, a = x @ w, x.abs() @ w.abs()
    if bias is not None:
        z, a = z + bias.double(), a + bias.double().abs()
    y, tol_z = act(z, name), (x.shape[1] + 8) * STEP * a
    tol_y = SLOPE * tol_z + (0 if name in ("none", "relu") else 2.0 ** -20 * (z.abs() + 1))
    if residual is not None:
        y = y + residual.double()
        tol_y = tol_y + STEP * (y.abs() + residual.double().abs())
    return y, z, tol_y + U8 * (y.abs() + tol_y), tol_z + U8 * (z.abs() + tol_z)


def linear_bwd(x, w, dy, z=None, name="none"):
    """{name: (value, tolerance)} of dx, dw, dbias for 2-D x."""
    x, w, dy = x.double(), w.double(), dy.double()
    if z is None:
        dz, e = dy, torch.zeros_like(dy)
    else:
        z = z.double()
        dz = dy * act_slope(z, name)
        # the slope's evaluation, then (for the products) its bf16 rounding
        e = dy.abs() * (2.0 ** -19 * (1 + z.abs()) if name != "relu" else 0.0) + STEP * dz.abs()
    er = e if z is None else e + U8 * (dz.abs() + e)
    out = {}
    for key, v, a, err, n in (
            ("dx", dz @ w.T, dz.abs() @ w.abs().T, er @ w.abs().T, w.shape[1]),
            ("dw", x.T @ dz, x.abs().T @ dz.abs(), x.abs().T @ er, x.shape[0])):
        t = err + (n + 8) * STEP * (a + err)
        out[key] = (v, t + U8 * (v.abs() + t))
    out["db"] = (dz.sum(0), e.sum(0) + (x.shape[0] + 8) * STEP * dz.abs().sum(0))
    return out


def heads_to_rows(o):
    """[B, H, N, d] -> [B N, H d]."""
    B, H, N, d = o.shape
    return o.permute(0, 2, 1, 3).reshape(B * N, H * d)


def rows_to_heads(x, B, H, N, d):
    return x.view(B, N, H, d).permute(0, 2, 1, 3)


def rms_norm(x, weight, residual=None, eps=1e-6):
    """(y, h, rstd) in 64 bits."""
    h = x.double() if residual is None else x.double() + residual.double()
    rstd = 1 / torch.sqrt((h * h).mean(-1) + eps)
    return h * rstd.unsqueeze(-1) * weight.double(), h, rstd


def rms_norm_bwd(dy, h, weight, rstd, dh=None):
    """{name: (value, tolerance)} of dx, dweight for 2-D h, from the kept h and rstd."""
    dy, h, weight, r = dy.double(), h.double(), weight.double(), rstd.double().unsqueeze(-1)
    D = h.shape[1]
    g, n = dy * weight, h * r
    c, ca = (g * n).mean(-1, keepdim=True), (g * n).abs().mean(-1, keepdim=True)
    dx = r * (g - n * c)
    # a mean of D products, then a handful of fp32 operations
    tol = r * n.abs() * ca * (D + 16) * STEP + 16 * STEP * r * (g.abs() + (n * c).abs())
    if dh is not None:
        dx = dx + dh.double()
        tol = tol + STEP * (dx.abs() + dh.double().abs())
    dw = (dy * n).sum(0)
    return {"dx": (dx, tol + U8 * (dx.abs() + tol)),
            "dweight": (dw, (h.shape[0] + 16) * STEP * (dy * n).abs().sum(0))}


def check(name, got, ref, tol):
    """Every element of `got` within its own tolerance of `ref`."""
    assert tuple(got.shape) == tuple(ref.shape), f"{name}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    d = (got.double() - ref).abs()
    bad = ~(d <= tol)
    if bool(bad.any()):
        i = int((d / tol.clamp_min(1e-300)).nan_to_num(posinf=1e30, nan=1e30).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} elements out of tolerance; worst at flat "
                             f"{i}: got {got.reshape(-1)[i].item()}, expected {ref.reshape(-1)[i].item()}, "
                             f"tolerance {tol.reshape(-1)[i].item()}")
