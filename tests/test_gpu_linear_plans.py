"""Every kernel that the linear layers' plans choose from, element by element against 64 bits within derived
bounds (see _block_ref), at the sizes of _linear_plans."""
import zlib

import pytest
import torch

import self_attention_gb300 as sa
import _block_ref as ref
import _linear_plans as plans

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_attention_gb300.build import build
    sa.load_library(build())


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


@pytest.mark.parametrize("M,K,N", plans.FORWARD)
def test_forward(M, K, N):
    """With and without bias, activation, residual and z, each in both states beside the others' both."""
    g = _gen(M, K, N)
    x, w = _randn(g, M, K), _randn(g, K, N, std=K ** -0.5)
    bias, res = _randn(g, N, dtype=torch.float32), _randn(g, M, N)
    for name, b, r, keep in (("none", None, None, False), ("gelu", bias, None, True), ("relu", bias, res, False),
                             ("silu", None, res, True), ("gelu_tanh", bias, res, True), ("none", None, res, False)):
        out = sa.linear_forward(x, w, b, r, name, keep_z=keep)
        y, z, ty, tz = ref.linear(x, w, b, r, name)
        ref.check(f"y {name}", out[0] if keep else out, y, ty)
        if keep:
            ref.check(f"z {name}", out[1], z, tz)
    assert sa.attn_get_device_status() == 0


@pytest.mark.parametrize("M,K,N", plans.Q8)
def test_q8(M, K, N):
    """Rows and columns with scales far apart."""
    g = _gen(M, K, N, "q8")
    xq, xs = sa.quantize_q8(_randn(g, M, K) * torch.exp2(torch.randint(-6, 7, (M, 1), generator=g, device="cuda")).bfloat16())
    wq, ws = sa.quantize_q8(_randn(g, N, K, std=K ** -0.5))
    bias, res = _randn(g, N, dtype=torch.float32), _randn(g, M, N)
    x = xq.double() * xs.double()[:, None]
    w = (wq.double() * ws.double()[:, None]).T
    for name, b, r in (("none", None, None), ("gelu_tanh", bias, None), ("silu", bias, res), ("none", None, res)):
        y, _, ty, _ = ref.linear(x, w, b, r, name)
        ref.check(f"y {name}", sa.linear_q8(xq, xs, wq, ws, b, r, name), y, ty)
    assert sa.attn_get_device_status() == 0


@pytest.mark.parametrize("B,H,N,d,n_out", plans.HEADS)
def test_out_proj(B, H, N, d, n_out):
    g = _gen(B, H, N, d, n_out)
    o, w = _randn(g, B, H, N, d), _randn(g, H * d, n_out, std=(H * d) ** -0.5)
    bias, res = _randn(g, n_out, dtype=torch.float32), _randn(g, B, N, n_out)
    rows = ref.heads_to_rows(o)
    for b, r in ((None, None), (bias, res), (None, res)):
        y, _, ty, _ = ref.linear(rows, w, b, None if r is None else r.view(B * N, n_out))
        ref.check("y", sa.out_proj_forward(o, w, b, r).view(B * N, n_out), y, ty)
    assert sa.attn_get_device_status() == 0


@pytest.mark.parametrize("M,K,N", plans.BACKWARD)
def test_backward(M, K, N):
    """Without an activation (the plan the size is there for) and with one, and each gradient alone."""
    g = _gen(M, K, N, "bwd")
    x, w, dy, z = _randn(g, M, K), _randn(g, K, N, std=K ** -0.5), _randn(g, M, N), _randn(g, M, N, std=2.0)
    for name in ("none", "gelu"):
        kept = None if name == "none" else z
        got = sa.linear_backward(x, w, dy, kept, name)
        want = ref.linear_bwd(x, w, dy, kept, name)
        for key, t in zip(("dx", "dw", "db"), got):
            ref.check(f"{key} {name}", t, *want[key])
        for i, key in enumerate(("dx", "dw", "db")):
            alone = sa.linear_backward(x, w, dy, kept, name, bias=i == 2, need_dx=i == 0, need_dw=i == 1)
            assert [t is not None for t in alone] == [i == 0, i == 1, i == 2]
            ref.check(f"{key} {name} alone", alone[i], *want[key])
    assert sa.attn_get_device_status() == 0


@pytest.mark.parametrize("B,H,N,d,n_out", plans.HEADS_BACKWARD)
def test_out_proj_backward(B, H, N, d, n_out):
    g = _gen(B, H, N, d, n_out, "bwd")
    o, w, dy = _randn(g, B, H, N, d), _randn(g, H * d, n_out, std=(H * d) ** -0.5), _randn(g, B, N, n_out)
    do, dw, db = sa.out_proj_backward(o, w, dy)
    want = ref.linear_bwd(ref.heads_to_rows(o), w, dy.view(B * N, n_out))
    ref.check("do", do, *(ref.rows_to_heads(t, B, H, N, d) for t in want["dx"]))
    ref.check("dw", dw, *want["dw"])
    ref.check("db", db, *want["db"])
    assert sa.attn_get_device_status() == 0
