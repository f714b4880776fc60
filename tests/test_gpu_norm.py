"""The root-mean-square norm (attn_rms_norm, its 8-bit form and its backward) on the GPU, against
plain 64-bit implementations within derived bounds (see _block_ref)."""
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


SHAPES = [(1, 8), (1, 2048), (2, 16), (3, 248), (7, 2048), (33, 256), (64, 264), (129, 768), (200, 1000),
          (1000, 1024), (513, 1032), (70, 2056), (37, 4096), (20, 4104), (9, 8192), (5, 8200), (11, 16384),
          (3, 16392), (4, 40000), (6001, 64), (2, 65544), (2500, 2048), (400, 2056)]


@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("with_res", [False, True])
def test_rms_norm(M, D, with_res):
    g = _gen(M, D, with_res)
    x, w = _randn(g, M, D), 1 + _randn(g, D, std=0.2, dtype=torch.float32)
    res = _randn(g, M, D, std=2.0) if with_res else None
    y, h, rstd = sa.rms_norm_forward(x, w, res, 1e-5)
    ry, rh, rr = ref.rms_norm(x, w, res, 1e-5)
    # h is exact in fp32 up to half a step; the mean of D squares is off by (D + 8) steps, its
    # inverse root by half of that and a few operations
    tr = ((D + 8) / 2 + 8) * ref.STEP
    ref.check("rstd", rstd, rr, tr * rr)
    t = (tr + 4 * ref.STEP) * ry.abs()
    ref.check("y", y, ry, t + ref.U8 * (ry.abs() + t))
    if with_res:
        ref.check("h", h, rh, ref.U8 * rh.abs() * (1 + ref.STEP) + ref.STEP * rh.abs())
    else:
        assert h is x


@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("with_dh", [False, True])
def test_rms_norm_backward(M, D, with_dh):
    g = _gen(M, D, with_dh, "bwd")
    h, dy, w = _randn(g, M, D), _randn(g, M, D), 1 + _randn(g, D, std=0.2, dtype=torch.float32)
    dh = _randn(g, M, D) if with_dh else None
    rstd = ref.rms_norm(h, w)[2].float()
    dx, dw = sa.rms_norm_backward(dy, h, w, rstd, dh)
    want = ref.rms_norm_bwd(dy, h, w, rstd, dh)
    ref.check("dx", dx, *want["dx"])
    ref.check("dweight", dw, *want["dweight"])
    again = sa.rms_norm_backward(dy, h, w, rstd, dh)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def _check_q8(q, scale, y, ty):
    """q scale against y: half an e4m3 step (2^-4 relative, or half of 2^-9 of the scale below the
    normal range), where the kernel's own y may be off by ty."""
    amax = y.abs().amax(-1)
    s = amax.clamp_min(ref.AMAX_FLOOR) / ref.Q8_MAX
    ref.check("scale", scale, s, ty.amax(-1) / ref.Q8_MAX + 4 * ref.STEP * s)
    deq = q.double() * scale.double().unsqueeze(-1)
    tol = ty + 2.0 ** -4 * (y.abs() + ty) + 2.0 ** -10 * s.unsqueeze(-1) + 8 * ref.STEP * y.abs()
    ref.check("q", deq, y, tol)
    assert bool((q.double().abs().amax(-1)[amax > 1e-20] == 448).all())


@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("with_res", [False, True])
def test_rms_norm_q8(M, D, with_res):
    g = _gen(M, D, with_res, "q8")
    x, w = _randn(g, M, D), 1 + _randn(g, D, std=0.2, dtype=torch.float32)
    res = _randn(g, M, D) if with_res else None
    q, scale, h = sa.rms_norm_q8(x, w, res, 1e-5)
    y, rh, _ = ref.rms_norm(x, w, res, 1e-5)
    _check_q8(q, scale, y, ((D + 8) / 2 + 12) * ref.STEP * y.abs())
    if with_res:
        ref.check("h", h, rh, ref.U8 * rh.abs() * (1 + ref.STEP) + ref.STEP * rh.abs())
    xq, xs = sa.quantize_q8(x)
    _check_q8(xq, xs, x.double(), torch.zeros_like(y))


def test_rows_of_zeros_tiny_and_non_finite_values():
    D = 512
    g = _gen("rows")
    x = _randn(g, 6, D)
    x[1] = 0
    x[2] *= 2.0 ** -60
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    w = torch.ones(D, device="cuda")
    y, _, rstd = sa.rms_norm_forward(x, w, None, 1e-6)
    assert not bool(y[1].any()) and abs(rstd[1].item() - 1000.0) < 1e-2
    assert bool(y[3].isnan().all()) and not bool(y[4].isfinite().all())
    clean = [0, 1, 2, 5]
    ry = ref.rms_norm(x, w, None, 1e-6)[0]
    ref.check("y", y[clean], ry[clean], ref.U8 * 1.01 * ry[clean].abs() + 1e-30)
    q, s, _ = sa.rms_norm_q8(x, w, None, 1e-6)
    assert not bool(q[1].double().any()) and bool((s[[3, 4]].isnan()).all())
    assert bool(s[clean].isfinite().all()) and bool(q[clean].double().isfinite().all())
    q, s = sa.quantize_q8(x)
    assert not bool(q[1].double().any()) and bool((s[[3, 4]].isnan()).all())
    _check_q8(q[clean], s[clean], x[clean].double(), torch.zeros_like(ry[clean]))
    # a zero row with eps = 0 has no norm
    y, _, rstd = sa.rms_norm_forward(x[1:2].contiguous(), w, None, 0.0)
    assert bool(rstd.isinf().all()) and bool(y.isnan().all())


def test_in_place_and_guards():
    g = _gen("inplace")
    M, D = 37, 776
    x, res, w = _randn(g, M, D), _randn(g, M, D), 1 + _randn(g, D, std=0.2, dtype=torch.float32)
    y, h, rstd = sa.rms_norm_forward(x, w, res)
    for which in ("x", "residual"):
        a, b = x.clone(), res.clone()
        buf = torch.full((M + 8, D), 7.0, dtype=torch.bfloat16, device="cuda")
        sa.attn_rms_norm(a, b, w, buf[4:], a if which == "x" else b, None, M, D, 1e-6)
        assert torch.equal(a if which == "x" else b, h)
        assert torch.equal(buf[4:4 + M], y) and bool((buf[:4] == 7).all()) and bool((buf[4 + M:] == 7).all())
    dy, dh = _randn(g, M, D), _randn(g, M, D)
    dx, dw = sa.rms_norm_backward(dy, h, w, rstd, dh)
    n = sa.attn_rms_norm_bwd_workspace_size(M, D)
    ws = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
    buf, dw2 = torch.full((M + 8, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.empty_like(dw)
    buf[4:4 + M] = dh
    sa.attn_rms_norm_bwd(dy, h, w, rstd, buf[4:], buf[4:], dw2, ws, n, M, D)
    assert torch.equal(buf[4:4 + M], dx) and torch.equal(dw, dw2)
    assert bool((buf[:4] == 7).all()) and bool((buf[4 + M:] == 7).all()) and bool((ws[n:] == 77).all())


def test_empty_streams_graphs_and_autograd():
    g = _gen("misc")
    D = 256
    w = (1 + _randn(g, D, std=0.2, dtype=torch.float32)).requires_grad_()
    e = torch.empty(0, D, dtype=torch.bfloat16, device="cuda")
    y, h, rstd = sa.rms_norm_forward(e, w.detach(), e)
    assert y.shape == (0, D) and rstd.shape == (0,)
    dx, dw = sa.rms_norm_backward(y, h, w.detach(), rstd)
    assert dx.shape == (0, D) and not bool(dw.any())
    x, res = _randn(g, 3, 50, D), _randn(g, 3, 50, D)
    want = sa.rms_norm_forward(x, w.detach(), res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sa.rms_norm_forward(x, w.detach(), res, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = sa.rms_norm_forward(x, w.detach(), res)
        bwd = sa.rms_norm_backward(res, got[1], w.detach(), got[2], x)
    x.copy_(_randn(g, 3, 50, D))
    gr.replay()
    want = sa.rms_norm_forward(x, w.detach(), res)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(sa.rms_norm_backward(res, want[1], w.detach(), want[2], x), bwd))
    # autograd: y and h both used, then h alone, then no residual
    xg, rg = x.detach().requires_grad_(), res.detach().requires_grad_()
    dy, dh = _randn(g, 3, 50, D), _randn(g, 3, 50, D)
    y, h = sa.rms_norm(xg, w, rg)
    torch.autograd.backward([y, h], [dy, dh])
    ref_b = ref.rms_norm_bwd(dy.view(-1, D), h.detach().view(-1, D), w.detach(), want[2].view(-1), dh.view(-1, D))
    ref.check("dx", xg.grad.view(-1, D), *ref_b["dx"])
    ref.check("dw", w.grad, *ref_b["dweight"])
    assert torch.equal(xg.grad, rg.grad)
    xg.grad = rg.grad = w.grad = None
    y, h = sa.rms_norm(xg, w, rg)
    h.backward(dh)
    assert torch.equal(xg.grad, dh) and torch.equal(rg.grad, dh) and not bool(w.grad.any())
    xg.grad = None
    sa.rms_norm(xg, w).backward(dy)
    rstd = ref.rms_norm(x.view(-1, D), w.detach())[2].float()
    want = ref.rms_norm_bwd(dy.view(-1, D), x.view(-1, D), w.detach(), rstd)["dx"]
    ref.check("dx", xg.grad.view(-1, D), want[0], want[1] * (1 + 2.0 ** -6) + 2.0 ** -14)


def test_refusals_by_tensor():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (lambda: sa.rms_norm_forward(x, w.bfloat16()), lambda: sa.rms_norm_forward(x, w[:32]),
                lambda: sa.rms_norm_forward(x.t(), w), lambda: sa.rms_norm_forward(x, w, x[:2]),
                lambda: sa.rms_norm_forward(x.cpu(), w), lambda: sa.rms_norm_backward(x, x, w, w),
                lambda: sa.rms_norm_q8(x.half(), w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sa.rms_norm_forward(x, w, eps=float("nan")), lambda: sa.rms_norm_forward(x, w, eps=-1.0),
                lambda: sa.rms_norm_forward(x[:, :60].contiguous(), w[:60].contiguous()),
                lambda: sa.quantize_q8(x[:, :60].contiguous())):
        with pytest.raises(sa.AttnError) as e:
            bad()
        assert e.value.code == 1


@pytest.mark.parametrize("M,D", [(1, 64), (5, 8), (33, 64), (1000, 72), (7, 128), (777, 128), (100_003, 64), (40_001, 128),
                                 (30_001, 200), (20_003, 256), (13_001, 392), (10_007, 512)])
def test_short_rows(M, D):
    """Several rows a warp, and several a thread where there are many; numbers of rows that end inside both."""
    for flag in (False, True):
        test_rms_norm(M, D, flag)
        test_rms_norm_q8(M, D, flag)
        test_rms_norm_backward(M, D, flag)


@pytest.mark.parametrize("M,D", [(45, 64), (45, 128), (90_001, 64), (50_001, 128)])
def test_short_rows_do_not_see_one_another(M, D):
    """A NaN or an infinity stays in its row, and nothing is written behind the last."""
    g = _gen("alone", M, D)
    x, dy, w = _randn(g, M, D), _randn(g, M, D), 1 + _randn(g, D, std=0.2, dtype=torch.float32)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[torch.tensor([0, 3, 9, M // 2, M - 1], device="cuda")] = True
    x2, dy2 = x.clone(), dy.clone()
    x2[bad, 5] = float("nan")
    dy2[bad, 1] = float("inf")
    (y, _, rstd), (q, scale, _) = sa.rms_norm_forward(x, w), sa.rms_norm_q8(x, w)
    (y2, _, rstd2), (q2, scale2, _) = sa.rms_norm_forward(x2, w), sa.rms_norm_q8(x2, w)
    assert torch.equal(y[~bad], y2[~bad]) and torch.equal(rstd[~bad], rstd2[~bad]) and bool(rstd2[bad].isnan().all())
    assert torch.equal(q[~bad].float(), q2[~bad].float()) and torch.equal(scale[~bad], scale2[~bad])
    assert bool(scale2[bad].isnan().all())
    dx, dx2 = sa.rms_norm_backward(dy, x, w, rstd)[0], sa.rms_norm_backward(dy2, x, w, rstd)[0]
    assert torch.equal(dx[~bad], dx2[~bad]) and bool((~dx2[bad].isfinite()).any(-1).all())

    rows = 40   # behind the last
    full = [torch.full((M + rows, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    stat = torch.full((M + rows,), 7.0, device="cuda")
    sa.attn_rms_norm(x, x, w, full[0], full[1], stat, M, D, 1e-6)
    n = sa.attn_rms_norm_bwd_workspace_size(M, D)
    dw, ws = torch.empty(D, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda")
    sa.attn_rms_norm_bwd(dy, x, w, rstd, None, full[2], dw, ws, n, M, D)
    torch.cuda.synchronize()
    for t in (*full, stat):
        assert bool((t[M:] == 7.0).all())
    assert torch.equal(full[2][:M], dx)
