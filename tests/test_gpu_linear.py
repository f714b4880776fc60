"""The linear layers (attn_linear, attn_out_proj, attn_linear_q8) and their backward on the GPU,
against plain 64-bit implementations within derived bounds (see _block_ref)."""
import zlib

import pytest
import torch

import self_attention_gb300 as sa
import _block_ref as ref

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


def _status_ok():
    assert sa.attn_get_device_status() == 0


# one row to several tiles, one under and one over each tile edge, widths that end inside a tile
SHAPES = [(1, 8, 8), (1, 64, 128), (1, 2048, 512), (2, 72, 1032), (3, 1000, 24), (7, 136, 264),
          (16, 256, 256), (17, 512, 128), (33, 4096, 136), (64, 128, 320), (65, 64, 72), (127, 200, 504),
          (128, 1024, 384), (129, 192, 256), (196, 768, 768), (255, 264, 640), (256, 320, 128),
          (257, 256, 520), (300, 1032, 248), (577, 128, 1024), (1111, 1000, 520), (2049, 64, 8),
          (1500, 8, 2056)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_forward(M, K, N):
    g = _gen(M, K, N)
    x, w = _randn(g, M, K), _randn(g, K, N, std=K ** -0.5)
    bias, res = _randn(g, N, dtype=torch.float32), _randn(g, M, N)
    for name, b, r, keep in (("none", None, None, False), ("gelu", bias, None, True), ("relu", bias, res, False),
                             ("silu", None, res, True), ("gelu_tanh", bias, res, False), ("none", bias, res, True)):
        out = sa.linear_forward(x, w, b, r, name, keep_z=keep)
        y, z, ty, tz = ref.linear(x, w, b, r, name)
        ref.check(f"y {name}", out[0] if keep else out, y, ty)
        if keep:
            ref.check(f"z {name}", out[1], z, tz)
    _status_ok()


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_backward(M, K, N):
    g = _gen(M, K, N, "bwd")
    x, w, dy, z = _randn(g, M, K), _randn(g, K, N, std=K ** -0.5), _randn(g, M, N), _randn(g, M, N, std=2.0)
    for name in ref.ACTS:
        got = sa.linear_backward(x, w, dy, None if name == "none" else z, name)
        want = ref.linear_bwd(x, w, dy, None if name == "none" else z, name)
        for key, t in zip(("dx", "dw", "db"), got):
            ref.check(f"{key} {name}", t, *want[key])
    dx, dw, db = sa.linear_backward(x, w, dy, bias=False, need_dx=False)
    assert dx is None and db is None
    ref.check("dw alone", dw, *ref.linear_bwd(x, w, dy)["dw"])
    dx, dw, db = sa.linear_backward(x, w, dy, z, "gelu", bias=False, need_dw=False)
    assert dw is None and db is None
    ref.check("dx alone", dx, *ref.linear_bwd(x, w, dy, z, "gelu")["dx"])
    _status_ok()


HEADS = [(1, 1, 1, 64, 8), (1, 12, 196, 64, 768), (3, 2, 130, 128, 264), (5, 3, 63, 64, 136), (2, 5, 257, 64, 320),
         (33, 2, 7, 64, 128), (2, 16, 300, 128, 512), (1, 1, 513, 128, 1024)]


@pytest.mark.parametrize("B,H,N,d,n_out", HEADS)
def test_out_proj(B, H, N, d, n_out):
    g = _gen(B, H, N, d, n_out)
    o, w = _randn(g, B, H, N, d), _randn(g, H * d, n_out, std=(H * d) ** -0.5)
    bias, res, dy = _randn(g, n_out, dtype=torch.float32), _randn(g, B, N, n_out), _randn(g, B, N, n_out)
    rows = ref.heads_to_rows(o)
    for b, r in ((None, None), (bias, res), (None, res)):
        y, _, ty, _ = ref.linear(rows, w, b, None if r is None else r.view(B * N, n_out))
        ref.check("y", sa.out_proj_forward(o, w, b, r).view(B * N, n_out), y, ty)
    do, dw, db = sa.out_proj_backward(o, w, dy)
    want = ref.linear_bwd(rows, w, dy.view(B * N, n_out))
    ref.check("do", do, *(ref.rows_to_heads(t, B, H, N, d) for t in want["dx"]))
    ref.check("dw", dw, *want["dw"])
    ref.check("db", db, *want["db"])
    _status_ok()


Q8_SHAPES = [(1, 16, 8), (1, 8192, 256), (2, 144, 1032), (7, 1008, 24), (16, 256, 256), (33, 512, 136),
             (64, 4096, 128), (128, 128, 384), (129, 192, 264), (196, 768, 768), (256, 336, 128), (257, 256, 520),
             (300, 1040, 248), (1111, 1008, 520), (2049, 64, 8)]


@pytest.mark.parametrize("M,K,N", Q8_SHAPES)
def test_linear_q8(M, K, N):
    g = _gen(M, K, N, "q8")
    xq, xs = sa.quantize_q8(_randn(g, M, K))
    wq, ws = sa.quantize_q8(_randn(g, N, K, std=K ** -0.5))
    bias, res = _randn(g, N, dtype=torch.float32), _randn(g, M, N)
    # the products of the values that the 8 bits stand for are exact: the bound of a bf16 product,
    # and two more roundings for the scales
    x = xq.double() * xs.double()[:, None]
    w = (wq.double() * ws.double()[:, None]).T
    for name, b, r in (("none", None, None), ("gelu_tanh", bias, None), ("silu", bias, res), ("none", None, res)):
        y, _, ty, _ = ref.linear(x, w, b, r, name)
        ref.check(f"y {name}", sa.linear_q8(xq, xs, wq, ws, b, r, name), y, ty)
    _status_ok()


def test_linear_leading_dimensions_and_empty():
    g = _gen("lead")
    x, w, bias = _randn(g, 3, 5, 64), _randn(g, 64, 40), _randn(g, 40, dtype=torch.float32)
    y = sa.linear_forward(x, w, bias, None, "gelu")
    assert y.shape == (3, 5, 40)
    assert torch.equal(y.view(15, 40), sa.linear_forward(x.view(15, 64), w, bias, None, "gelu"))
    assert sa.linear_forward(x[1, 2], w, bias, None, "gelu").shape == (40,)
    # no rows: nothing to do forward, zero gradients of the parameters backward
    e = x[:0]
    y, z = sa.linear_forward(e, w, bias, None, "gelu", keep_z=True)
    assert y.shape == (0, 5, 40)
    dx, dw, db = sa.linear_backward(e, w, y, z, "gelu")
    assert dx.shape == e.shape and not bool(dw.any()) and not bool(db.any())
    q, s = sa.quantize_q8(e)
    wq, ws = sa.quantize_q8(w.t().contiguous())
    assert sa.linear_q8(q, s, wq, ws).shape == (0, 5, 40)
    _status_ok()


@pytest.mark.parametrize("M", [5, 300])
def test_non_finite_rows_stay_in_their_rows(M):
    """A NaN or an infinity in one row of x (or dy) reaches that row of the output alone."""
    g = _gen("nan", M)
    x, w, res = _randn(g, M, 200), _randn(g, 200, 136, std=0.1), _randn(g, M, 136)
    clean = sa.linear_forward(x, w, None, res, "gelu")
    xb = x.clone()
    xb[2, 7], xb[4, 199] = float("nan"), float("inf")
    y = sa.linear_forward(xb, w, None, res, "gelu")
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[[2, 4]] = False
    assert torch.equal(y[keep], clean[keep])
    assert bool(y[2].isnan().all()) and not bool(y[4].isfinite().all())
    dy = _randn(g, M, 136)
    dxc, _, _ = sa.linear_backward(x, w, dy)
    dyb = dy.clone()
    dyb[2, 100] = float("nan")
    dx, dw, db = sa.linear_backward(x, w, dyb)
    keep[4] = True
    assert torch.equal(dx[keep], dxc[keep])
    assert bool(dx[2].isnan().all()) and bool(dw[:, 100].isnan().all()) and bool(db[100].isnan())
    assert bool(dw[:, :100].isfinite().all()) and bool(db[:100].isfinite().all())


@pytest.mark.parametrize("M,K,N", [(3, 72, 136), (130, 128, 264), (300, 200, 72)])
def test_writes_stay_inside_and_in_place_residual(M, K, N):
    """Rows before and behind the outputs are left as they were, and y may be the residual itself."""
    g = _gen("guard", M, K, N)
    x, w, res, bias = _randn(g, M, K), _randn(g, K, N), _randn(g, M, N), _randn(g, N, dtype=torch.float32)
    want = sa.linear_forward(x, w, bias, res, "silu")
    big = torch.full((M + 16, N), 7.0, dtype=torch.bfloat16, device="cuda")
    zbig = big.clone()
    sa.attn_linear(x, w, bias, res, big[8:], zbig[8:], M, K, N, sa.ACTIVATIONS["silu"])
    assert torch.equal(big[8:8 + M], want)
    for t in (big, zbig):
        assert bool((t[:8] == 7).all()) and bool((t[8 + M:] == 7).all())
    inplace = res.clone()
    sa.attn_linear(x, w, bias, inplace, inplace, None, M, K, N, sa.ACTIVATIONS["silu"])
    assert torch.equal(inplace, want)
    dy, z = _randn(g, M, N), _randn(g, M, N)
    dx, dw, db = sa.linear_backward(x, w, dy, z, "silu")
    gx = torch.full((M + 16, K), 7.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.full((K + 16, N), 7.0, dtype=torch.bfloat16, device="cuda")
    gb = torch.full((N + 16,), 7.0, device="cuda")
    nbytes = sa.attn_linear_bwd_workspace_size(M, K, N, 4)
    ws = torch.full((nbytes + 256,), 77, dtype=torch.uint8, device="cuda")
    sa.attn_linear_bwd(x, w, dy, z, gx[8:], gw[8:], gb[8:], ws, nbytes, M, K, N, 4)
    for got, t, n in ((gx, dx, M), (gw, dw, K), (gb, db, N)):
        assert torch.equal(got[8:8 + n], t)
        assert bool((got[:8] == 7).all()) and bool((got[8 + n:] == 7).all())
    assert bool((ws[nbytes:] == 77).all())


@pytest.mark.parametrize("M,K,N", [(1, 2048, 512), (40, 512, 264), (700, 320, 520)])
def test_reproducible_and_captured(M, K, N):
    """The same call twice, on another stream, and captured and replayed on new inputs: the same bits."""
    g = _gen("graph", M, K, N)
    x, w, dy, z = _randn(g, M, K), _randn(g, K, N), _randn(g, M, N), _randn(g, M, N)
    bias, res = _randn(g, N, dtype=torch.float32), _randn(g, M, N)
    xq, xs = sa.quantize_q8(_randn(g, M, K))
    wq, ws = sa.quantize_q8(_randn(g, N, K))

    def run(stream=None):
        return (sa.linear_forward(x, w, bias, res, "gelu", stream=stream),
                *sa.linear_backward(x, w, dy, z, "gelu", stream=stream),
                sa.linear_q8(xq, xs, wq, ws, bias, res, stream=stream))

    first = run()
    for a, b in zip(first, run()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = run(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = run()
        graphs.append((gr, out))
    x.copy_(_randn(g, M, K))
    dy.copy_(_randn(g, M, N))
    for gr, _ in graphs:
        gr.replay()
    again = run()
    for _, out in graphs:
        for a, b in zip(again, out):
            assert torch.equal(a, b)
    _status_ok()


def test_autograd_matches_the_formulas():
    g = _gen("autograd")
    x, w = _randn(g, 4, 33, 128).requires_grad_(), _randn(g, 128, 72, std=0.1).requires_grad_()
    bias, res = _randn(g, 72, dtype=torch.float32).requires_grad_(), _randn(g, 4, 33, 72).requires_grad_()
    dy = _randn(g, 4, 33, 72)
    y = sa.linear(x, w, bias, res, "gelu")
    _, z = sa.linear_forward(x.detach(), w.detach(), bias.detach(), None, "gelu", keep_z=True)
    y.backward(dy)
    want = ref.linear_bwd(x.detach().view(-1, 128), w.detach(), dy.view(-1, 72), z.view(-1, 72), "gelu")
    ref.check("dx", x.grad.view(-1, 128), *want["dx"])
    ref.check("dw", w.grad, *want["dw"])
    ref.check("db", bias.grad, *want["db"])
    assert torch.equal(res.grad, dy)
    # a non-contiguous incoming gradient, and only some inputs asked for
    x.grad = w.grad = None
    sa.linear(x, w.detach(), None, None, "silu").sum().backward()
    _, z = sa.linear_forward(x.detach(), w.detach(), None, None, "silu", keep_z=True)
    want = ref.linear_bwd(x.detach().view(-1, 128), w.detach(), torch.ones(132, 72, device="cuda"), z.view(-1, 72), "silu")
    ref.check("dx", x.grad.view(-1, 128), *want["dx"])
    o = _randn(g, 2, 3, 50, 64).requires_grad_()
    wo = _randn(g, 192, 72).requires_grad_()
    dyo = _randn(g, 2, 50, 72)
    sa.out_proj(o, wo).backward(dyo)
    want = ref.linear_bwd(ref.heads_to_rows(o.detach()), wo.detach(), dyo.view(100, 72))
    ref.check("do", o.grad, *(ref.rows_to_heads(t, 2, 3, 50, 64) for t in want["dx"]))
    ref.check("dwo", wo.grad, *want["dw"])
    _status_ok()


def test_refusals_by_tensor():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, 32, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(32, device="cuda")
    for bad in (lambda: sa.linear_forward(x.float(), w), lambda: sa.linear_forward(x.t(), w),
                lambda: sa.linear_forward(x, w.t()), lambda: sa.linear_forward(x, w, b.bfloat16()),
                lambda: sa.linear_forward(x, w, b[:16]), lambda: sa.linear_forward(x, w, b, x),
                lambda: sa.linear_forward(x, w, activation="swish"), lambda: sa.linear_forward(x.cpu(), w),
                lambda: sa.linear_forward(x, w.cpu()), lambda: sa.linear_backward(x, w, x),
                lambda: sa.linear_backward(x, w, torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"),
                                           activation="gelu"),
                lambda: sa.out_proj_forward(x, w), lambda: sa.linear_q8(x, b, w, b),
                lambda: sa.quantize_q8(x.float())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sa.AttnError) as e:      # a width that is no multiple of 8
        sa.linear_forward(torch.zeros(4, 60, dtype=torch.bfloat16, device="cuda"), w[:60].contiguous())
    assert e.value.code == 1
    with pytest.raises(sa.AttnError) as e:      # rows that do not start on 16 bytes
        y = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
        sa.attn_linear(x.view(-1)[1:], w, None, None, y, None, 3, 64, 32, 0)
    assert e.value.code == 3


@pytest.mark.parametrize("M,K,N", [(1, 8, 8), (70, 16, 20008), (65, 520, 72), (513, 64, 264), (640, 1032, 1000),
                                   (2049, 264, 4104)])
def test_bias_gradient_of_few_and_many_rows(M, K, N):
    """By whole columns, by slices of rows and in a pass of its own; with and without the other gradients."""
    g = _gen("bias", M, K, N)
    x, w, dy = _randn(g, M, K), _randn(g, K, N, std=0.05), _randn(g, M, N)
    want = ref.linear_bwd(x, w, dy)
    for need_dx, need_dw in ((True, True), (False, True), (True, False), (False, False)):
        dx, dw, db = sa.linear_backward(x, w, dy, need_dx=need_dx, need_dw=need_dw)
        ref.check("db", db, *want["db"])
        assert torch.equal(db, sa.linear_backward(x, w, dy, need_dx=need_dx, need_dw=need_dw)[2])
        if need_dx:
            ref.check("dx", dx, *want["dx"])
        if need_dw:
            ref.check("dw", dw, *want["dw"])
