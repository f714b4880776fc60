"""The linear layers and the norm without a GPU: every bad argument is refused with the documented
status before the device is touched, and the plain 64-bit formulas the GPU tests compare with agree
with differences of one another."""
import pytest
import torch

import self_attention_gb300 as sa
import _block_ref as ref
from self_attention_gb300.build import build


@pytest.fixture(scope="module")
def lib():
    return sa.load_library(build())


# Fake, never-dereferenced device addresses, 256 MB apart.
X, W, BIAS, RES, Y, Z, DX, DW, DB, WS = (0x10000000 * (i + 1) for i in range(10))


def test_linear_argument_errors(lib):
    def fwd(x=X, w=W, bias=BIAS, res=RES, y=Y, z=Z, M=16, K=64, N=32, act=2):
        return lib.attn_linear(x, w, bias, res, y, z, M, K, N, act, None)

    assert fwd(M=-1) == 1
    for bad in (0, -8, 4, 60, 1 << 20):
        assert fwd(K=bad) == 1 and fwd(N=bad) == 1
    assert fwd(M=0x7fffffff, K=1 << 19) == 1            # 2^50 elements
    assert fwd(act=-1) == 1 and fwd(act=5) == 1
    assert fwd(M=0, x=0, w=0, y=0) == 0                 # no rows: nothing to do
    assert fwd(x=0) == 1 and fwd(w=0) == 1 and fwd(y=0) == 1
    for k in ("x", "w", "bias", "res", "y", "z"):
        assert fwd(**{k: X + 8 if k == "x" else 0xF0000008}) == 3
    assert fwd(y=X) == 1 and fwd(y=W + 16) == 1 and fwd(y=BIAS) == 1 and fwd(z=RES) == 1
    assert fwd(y=Z) == 1
    assert fwd(y=RES + 64) == 1                         # over a part of the residual
    assert fwd(y=RES, z=RES + 512) == 1                 # y may be the residual, z may not overlap it


def test_out_proj_argument_errors(lib):
    def fwd(o=X, w=W, bias=0, res=0, y=Y, B=2, H=2, N=8, d=64, n_out=32):
        return lib.attn_out_proj(o, w, bias, res, y, B, H, N, d, n_out, None)

    assert fwd(d=32) == 2 and fwd(d=96) == 2
    for k in ("B", "H", "N"):
        assert fwd(**{k: 0}) == 1
    assert fwd(n_out=12) == 1 and fwd(n_out=0) == 1
    assert fwd(B=1 << 16, N=1 << 16) == 1               # rows past the int range
    assert fwd(H=1 << 14) == 1
    assert fwd(o=0) == 1 and fwd(y=0) == 1
    assert fwd(o=X + 2) == 3
    assert fwd(y=X) == 1


def test_linear_bwd_workspace_and_argument_errors(lib):
    need = sa.attn_linear_bwd_workspace_size(16, 64, 32, 2)
    assert need >= 16 * 32 * 2 + 32 * 4
    assert 0 < sa.attn_linear_bwd_workspace_size(16, 64, 32, 0) < need     # no dz to keep
    assert sa.attn_linear_bwd_workspace_size(16, 60, 32, 2) == 0
    assert sa.attn_linear_bwd_workspace_size(16, 64, 32, 7) == 0
    assert sa.attn_linear_bwd_workspace_size(-1, 64, 32, 0) == 0
    assert sa.attn_out_proj_bwd_workspace_size(2, 2, 8, 96, 32) == 0
    assert sa.attn_out_proj_bwd_workspace_size(2, 2, 8, 64, 32) > 0

    def bwd(x=X, w=W, dy=Y, z=Z, dx=DX, dw=DW, db=DB, ws=WS, nbytes=need, M=16, K=64, N=32, act=2):
        return lib.attn_linear_bwd(x, w, dy, z, dx, dw, db, ws, nbytes, M, K, N, act, None)

    assert bwd(K=60) == 1 and bwd(act=9) == 1 and bwd(M=-1) == 1
    assert bwd(x=0) == 1 and bwd(dy=0) == 1 and bwd(z=0) == 1 and bwd(w=0) == 1
    assert bwd(ws=0) == 6 and bwd(nbytes=need - 1) == 6 and bwd(ws=WS + 16) == 6
    assert bwd(dx=DX + 4) == 3 and bwd(db=DB + 8) == 3
    assert bwd(dx=X) == 1 and bwd(dw=W) == 1 and bwd(db=Z) == 1 and bwd(dx=DW) == 1 and bwd(db=WS + 64) == 1

    n2 = sa.attn_out_proj_bwd_workspace_size(2, 2, 8, 64, 32)

    def obwd(o=X, dy=Y, do=DX, nbytes=n2, d=64):
        return lib.attn_out_proj_bwd(o, W, dy, do, DW, DB, WS, nbytes, 2, 2, 8, d, 32, None)

    assert obwd(d=80) == 2 and obwd(nbytes=n2 - 1) == 6 and obwd(do=X) == 1 and obwd(dy=0) == 1


def test_q8_argument_errors(lib):
    def fwd(x=X, xs=BIAS, w=W, ws=RES, y=Y, M=16, K=64, N=32, act=0):
        return lib.attn_linear_q8(x, xs, w, ws, 0, 0, y, M, K, N, act, None)

    assert fwd(K=72) == 1 and fwd(K=0) == 1 and fwd(N=12) == 1 and fwd(M=-1) == 1 and fwd(act=6) == 1
    assert fwd(xs=0) == 1 and fwd(ws=0) == 1 and fwd(x=0) == 1
    assert fwd(xs=BIAS + 4) == 3 and fwd(x=X + 8) == 3
    assert fwd(y=W) == 1 and fwd(y=BIAS) == 1

    def quant(x=X, q=Y, s=Z, M=16, D=64):
        return lib.attn_quantize_q8(x, q, s, M, D, None)

    assert quant(D=60) == 1 and quant(M=-1) == 1 and quant(x=0) == 1 and quant(s=0) == 1
    assert quant(q=X) == 1 and quant(s=Y + 256) == 1 and quant(q=Y + 8) == 3 and quant(M=0, x=0, q=0, s=0) == 0


def test_rms_norm_argument_errors(lib):
    import ctypes
    f = ctypes.c_float

    def fwd(x=X, res=RES, w=W, y=Y, h=Z, r=DB, M=16, D=64, eps=1e-6):
        return lib.attn_rms_norm(x, res, w, y, h, r, M, D, f(eps), None)

    assert fwd(D=60) == 1 and fwd(D=0) == 1 and fwd(M=-1) == 1
    assert fwd(eps=-1e-6) == 1 and fwd(eps=float("nan")) == 1 and fwd(eps=float("inf")) == 1
    assert fwd(x=0) == 1 and fwd(w=0) == 1 and fwd(y=0) == 1
    assert fwd(res=0) == 1                              # h without a residual
    assert fwd(x=X + 4) == 3 and fwd(r=DB + 4) == 3
    assert fwd(y=X) == 1 and fwd(y=Z) == 1 and fwd(h=RES + 16) == 1 and fwd(h=W) == 1 and fwd(r=W) == 1
    assert fwd(M=0, x=0, y=0) == 0
    assert lib.attn_rms_norm_q8(X, RES, W, Y, 0, Z, 16, 64, f(1e-6), None) == 1      # no scale
    assert lib.attn_rms_norm_q8(X, RES, W, Y, DB, Z, 16, 60, f(1e-6), None) == 1     # D % 8
    assert lib.attn_rms_norm_q8(X, RES, W, Y, DB, Y + 512, 16, 64, f(1e-6), None) == 1

    need = sa.attn_rms_norm_bwd_workspace_size(16, 64)
    assert need > 0 and sa.attn_rms_norm_bwd_workspace_size(16, 60) == 0

    def bwd(dy=Y, h=X, w=W, r=DB, dh=RES, dx=DX, dw=DW, ws=WS, n=need, D=64):
        return lib.attn_rms_norm_bwd(dy, h, w, r, dh, dx, dw, ws, n, 16, D, None)

    assert bwd(D=12) == 1 and bwd(dy=0) == 1 and bwd(r=0) == 1 and bwd(dx=0) == 1 and bwd(dw=0) == 1
    assert bwd(n=need - 1) == 6 and bwd(ws=0) == 6 and bwd(ws=WS + 128) == 6
    assert bwd(dx=DX + 8) == 3
    assert bwd(dx=X) == 1 and bwd(dx=RES + 16) == 1 and bwd(dw=W) == 1 and bwd(dx=WS) == 1


def test_in_place_goes_by_operand(lib):
    """Only the operand that an output may lie over excuses it: y over a residual that is x as well would
    overwrite rows of x that other tiles still read."""
    import ctypes
    assert lib.attn_linear(X, W, BIAS, X, X, 0, 16, 64, 64, 0, None) == 1
    assert lib.attn_linear(X, RES, BIAS, RES, RES, 0, 64, 64, 64, 0, None) == 1
    assert lib.attn_out_proj(X, W, 0, X, X, 2, 2, 8, 64, 128, None) == 1
    assert lib.attn_linear_q8(X, BIAS, X, RES, 0, X, X, 16, 64, 32, 0, None) == 1
    f = ctypes.c_float(1e-6)
    assert lib.attn_rms_norm(X, RES, X, Y, X, DB, 1, 64, f, None) == 1
    need = sa.attn_rms_norm_bwd_workspace_size(16, 64)
    assert lib.attn_rms_norm_bwd(DX, X, W, DB, DX, DX, DW, WS, need, 16, 64, None) == 1
    assert lib.attn_rms_norm_bwd(Y, DX, W, DB, DX, DX, DW, WS, need, 16, 64, None) == 1


@pytest.mark.parametrize("name", ref.ACTS)
def test_slopes_against_differences(name):
    """act_slope is the slope of act: central differences, whose own error is the third derivative
    times step^2 / 6 and the 64-bit rounding over the step."""
    z = torch.linspace(-9, 9, 4001, dtype=torch.float64) + 1e-4     # no sample within a step of relu's kink
    step = 1e-5
    d = (ref.act(z + step, name) - ref.act(z - step, name)) / (2 * step)
    assert float((d - ref.act_slope(z, name)).abs().max()) < 1e-9


def test_gradients_of_the_formulas_against_differences():
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, dy = r(6, 8), r(8, 16), r(16), r(6, 16)
    for name in ref.ACTS:
        z = x @ w + b
        if name == "relu":
            assert float(z.abs().min()) > 1e-4
        grads = ref.linear_bwd(x, w, dy, z, name)
        loss = lambda x, w, b: (ref.act(x @ w + b, name) * dy).sum()  # noqa: E731
        for key, at in (("dx", 0), ("dw", 1), ("db", 2)):
            args = [x, w, b]
            v, e = torch.randn(args[at].shape, generator=g, dtype=torch.float64), 1e-6
            up, dn = list(args), list(args)
            up[at], dn[at] = args[at] + e * v, args[at] - e * v
            diff = (loss(*up) - loss(*dn)) / (2 * e)
            assert abs(float(diff - (grads[key][0] * v).sum())) < 1e-6
    x, res, w, dy, dh = r(5, 24), r(5, 24), r(24), r(5, 24), r(5, 24)
    y, h, rstd = ref.rms_norm(x, w, res, 1e-3)

    def loss(x, res, w):
        y, h, _ = ref.rms_norm(x, w, res, 1e-3)
        return (y * dy).sum() + (h * dh).sum()

    grads = ref.rms_norm_bwd(dy, h, w, rstd, dh)
    for key, at in (("dx", 0), ("dx", 1), ("dweight", 2)):
        args = [x, res, w]
        v, e = torch.randn(args[at].shape, generator=g, dtype=torch.float64), 1e-6
        up, dn = list(args), list(args)
        up[at], dn[at] = args[at] + e * v, args[at] - e * v
        diff = (loss(*up) - loss(*dn)) / (2 * e)
        assert abs(float(diff - (grads[key][0] * v).sum())) < 1e-6


def test_tensor_level_refusals_without_a_gpu(lib):
    """The compiled binding loads without a GPU and refuses what are no CUDA tensors with a ValueError,
    unknown activations by name, and never reaches the device."""
    x, w, v = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, 32, dtype=torch.bfloat16), torch.zeros(64)
    for bad in (lambda: sa.linear_forward(x, w), lambda: sa.linear_forward(None, w), lambda: sa.linear_forward(3, w),
                lambda: sa.linear_backward(x, w, x), lambda: sa.out_proj_forward(x, w), lambda: sa.out_proj_backward(x, w, x),
                lambda: sa.linear_q8(x, v, w, v), lambda: sa.rms_norm_forward(x, v), lambda: sa.rms_norm_q8(x, v),
                lambda: sa.rms_norm_backward(x, x, v, v), lambda: sa.quantize_q8(x), lambda: sa.quantize_q8("x"),
                lambda: sa.linear_forward(x, w, activation="swish"), lambda: sa.quantize_q8(x, stream=0)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        sa._binding().quantize_q8(x, x)
