"""Rotary positions on the GPU, against the formula in 64 bits within derived bounds (see _cache_ref), their
gradient against the formula's and against differences."""
import math
import zlib

import pytest
import torch

import self_attention_gb300 as sa
import _cache_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_attention_gb300.build import build
    sa.load_library(build())


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("B,H,N,d,rotated", [(1, 1, 1, 64, 64), (1, 16, 1, 128, 128), (2, 3, 7, 64, 16),
                                             (3, 5, 33, 128, 48), (1, 2, 1000, 128, 128), (2, 17, 129, 64, 32),
                                             (40, 24, 5, 128, 112), (2, 12, 1500, 64, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("where", ["none", "shared", "each"])
def test_rotary(B, H, N, d, rotated, interleaved, where):
    g = _gen(B, H, N, d, rotated, interleaved, where)
    x = _randn(g, B, H, N, d)
    turns, f = sa.rotary_turns(rotated), ref.frequencies(rotated)
    positions = None
    at = torch.arange(N).expand(B, N)
    if where == "shared":
        positions = torch.randint(-5, 1 << 20, (N,), generator=g, device="cuda", dtype=torch.int32)
        at = positions.cpu().expand(B, N)
    elif where == "each":
        positions = torch.randint(-(2 ** 31), 2 ** 31 - 1, (B, N), generator=g, device="cuda", dtype=torch.int32)
        at = positions.cpu()
    amplitude = 1.0 if where == "none" else 1.25
    y = sa.rotary_forward(x, turns, positions, interleaved, amplitude)
    # the angle of a 64-bit product is itself off by 2^-52 of the angle at positions this far
    want, tol = ref.turned(x.cpu(), at, f, interleaved, amplitude)
    far = 2.0 ** -52 * float(at.abs().max()) * 4
    ref.check("y", y, want, tol + far * x.cpu().double().abs().amax())
    assert torch.equal(y[..., rotated:], x[..., rotated:])
    dx = sa.rotary_backward(x, turns, positions, interleaved, amplitude)
    want, tol = ref.turned(x.cpu(), at, f, interleaved, amplitude, -1.0)
    ref.check("dx", dx, want, tol + far * x.cpu().double().abs().amax())


def test_positions_far_out_are_exact():
    """At position 2^31 - 1 the fastest pair has turned 3.4e8 times; an fp32 angle would be off by 100 radians."""
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[..., :32] = 1
    at = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device="cuda")
    y = sa.rotary_forward(x, sa.rotary_turns(64), at)[0, 0, 0].double().cpu()
    # turns a position as integers over 2^64, as exact as Python's
    for j, t in enumerate(sa.rotary_turns(64, device="cpu").tolist()):
        turn = (t * (2 ** 31 - 1) % 2 ** 64) / 2 ** 64
        assert abs(y[j] - math.cos(2 * math.pi * turn)) < 2.0 ** -8 * 1.01
        assert abs(y[j + 32] - math.sin(2 * math.pi * turn)) < 2.0 ** -8 * 1.01


@pytest.mark.parametrize("method", ["none", "positions", "base", "parts"])
def test_scaled_frequencies(method):
    g = _gen(method)
    x = _randn(g, 2, 3, 50, 128)
    rotated, factor, trained = 96, 4.0, 2048
    j = torch.arange(rotated // 2, dtype=torch.float64)
    f = ref.frequencies(rotated)
    if method == "positions":
        f = f / factor
    if method == "base":
        f = (10000.0 * factor ** (rotated / (rotated - 2))) ** (-2 * j / rotated)
        assert abs(f[-1] / ref.frequencies(rotated)[-1] - 1 / factor) < 1e-12 and f[0] == 1
    if method == "parts":
        ramp = ((trained * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = ramp * f + (1 - ramp) * f / factor
        assert f[0] == 1 and abs(f[-1] / ref.frequencies(rotated)[-1] - 1 / factor) < 1e-12
    at = torch.arange(10000, 10050, dtype=torch.int32)
    y = sa.rotary_forward(x, sa.rotary_turns(rotated, method=method, factor=factor, trained=trained), at.cuda())
    want, tol = ref.turned(x.cpu(), at.expand(2, 50), f)
    ref.check("y", y, want, tol + 2.0 ** -36)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(interleaved):
    """Against differences: rotary is linear, so that <dy, R e> for a unit e is the gradient's element."""
    g = _gen("grad", interleaved)
    x = _randn(g, 2, 2, 5, 64).requires_grad_()
    dy = _randn(g, 2, 2, 5, 64)
    at = torch.tensor([3, 1, 4, 1, 59], dtype=torch.int32, device="cuda")
    turns, f = sa.rotary_turns(32), ref.frequencies(32)
    y = sa.rotary(x, turns, at, interleaved, 1.5)
    y.backward(dy)
    base, step = x.detach().cpu().double(), 2.0 ** -3
    want = torch.zeros_like(base)
    for c in range(64):
        e = torch.zeros_like(base)
        e[..., c] = step
        hi, lo = (ref.turned(base + s * e, at.cpu().expand(2, 5), f, interleaved, 1.5)[0] for s in (1, -1))
        want[..., c] = (dy.cpu().double() * (hi - lo)).sum(-1) / (2 * step)
    tol = 8 * 2.0 ** -23 * 1.5 * 2 * dy.abs().amax().item() + 2.0 ** -8 * (want.abs() + 1e-6)
    ref.check("dx", x.grad, want, tol)
    with pytest.raises(RuntimeError):       # no second derivative
        x.grad = None
        y = sa.rotary(x, turns, at, interleaved)
        gx, = torch.autograd.grad(y, x, dy.requires_grad_(), create_graph=True)
        gx.sum().backward()


def test_training_through_projection_rotary_and_attention():
    """The gradients of a projection's input and weights with rotary positions ahead of attention, against PyTorch's own
    differentiation of the formulas in 64 bits: within 1e-2 of their norms, as the attention's own gradients are held."""
    g = _gen("train")
    B, N, H, d = 2, 130, 4, 64
    D = H * d
    x, dy = _randn(g, B, N, D), _randn(g, B, H, N, d)
    ws = [_randn(g, D, D, std=D ** -0.5) for _ in range(3)]
    turns, f = sa.rotary_turns(d), ref.frequencies(d).cuda()
    leaves = [t.clone().requires_grad_() for t in (x, *ws)]
    q, k, v = sa.qkv_proj(*leaves, H)
    o = sa.attention(sa.rotary(q, turns), sa.rotary(k, turns), v)
    o.backward(dy)
    plain = [t.double().requires_grad_() for t in (x, *ws)]
    heads = [(plain[0] @ w).view(B, N, H, d).transpose(1, 2) for w in plain[1:]]
    angle = torch.arange(N, device="cuda").double().view(N, 1) * f

    def turn(t):
        a, b = t[..., :d // 2], t[..., d // 2:]
        return torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1)

    p = (turn(heads[0]) @ turn(heads[1]).transpose(2, 3) / math.sqrt(d)).softmax(-1)
    (p @ heads[2]).backward(dy.double())
    for name, got, want in zip(("x", "w_q", "w_k", "w_v"), leaves, plain):
        err = (got.grad.double() - want.grad).norm() / want.grad.norm()
        assert err < 1e-2, (name, err.item())


def test_backward_captured_and_replayed():
    """The gradient in a graph, with leaves that no eager graph holds."""
    g = _gen("capture")
    x, dy = _randn(g, 2, 3, 40, 64), _randn(g, 2, 3, 40, 64)
    turns = sa.rotary_turns(64)
    want = sa.rotary_backward(dy, turns)
    leaf = x.clone().requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = sa.rotary(leaf, turns)
        grad, = torch.autograd.grad(y, leaf, dy)
    for _ in range(2):
        grad.zero_()
        graph.replay()
        assert torch.equal(grad, want)


def test_in_place_and_guards():
    g = _gen("inplace")
    B, H, N, d = 3, 5, 37, 128
    x = _randn(g, B, H, N, d)
    turns = sa.rotary_turns(64)
    y = sa.rotary_forward(x, turns)
    buf = torch.full((B + 2, H, N, d), 7.0, dtype=torch.bfloat16, device="cuda")
    buf[1:1 + B] = x
    sa.attn_rotary(buf[1:], buf[1:], None, 0, turns, B, H, N, d, 64, 0, 1.0)
    assert torch.equal(buf[1:1 + B], y) and bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())
    assert sa.rotary_forward(x[:0], turns).shape == (0, H, N, d)
    assert sa.rotary_forward(x[:, :, :0].contiguous(), turns).shape == (B, H, 0, d)


def test_non_finite_values_stay_in_their_pair():
    x = torch.ones(1, 1, 3, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 1, 3] = float("nan")
    x[0, 0, 2, 5] = float("inf")
    y = sa.rotary_forward(x, sa.rotary_turns(32), torch.tensor([1, 1, 1], dtype=torch.int32, device="cuda"))
    bad = ~y.isfinite()
    assert bad[0, 0].nonzero().tolist() == [[1, 3], [1, 19], [2, 5], [2, 21]]


def test_refusals():
    x = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    turns = sa.rotary_turns(32)
    ok = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    sa.rotary_forward(x, turns, ok)
    for bad in (ok.long(), ok[:1], ok[:, :3], ok.cpu(), ok.view(2, 4, 1), ok.t().contiguous().t()):
        with pytest.raises(ValueError):
            sa.rotary_forward(x, turns, bad)
    for bad in (x.float(), x[:, :, ::2], x[0], x.cpu(), x.transpose(1, 2)):
        with pytest.raises(ValueError):
            sa.rotary_forward(bad, turns)
    for bad in (turns.int(), turns.cpu(), turns.view(4, 4), turns.double()):
        with pytest.raises(ValueError):
            sa.rotary_forward(x, bad)
    for bad in (sa.rotary_turns(96), turns[:4], turns[:0]):       # wider than the head, not a multiple of 16, none
        with pytest.raises(sa.AttnError):
            sa.rotary_forward(x, bad.clone())
    with pytest.raises(sa.AttnError):
        sa.rotary_forward(x, turns, None, False, float("nan"))
    with pytest.raises(sa.AttnError):
        sa.rotary_forward(torch.zeros(1, 1, 1, 96, dtype=torch.bfloat16, device="cuda"), turns)
    for kw in (dict(rotated=8), dict(rotated=40), dict(rotated=32, method="no"), dict(rotated=32, base=1.0),
               dict(rotated=32, factor=0.0), dict(rotated=32, method="parts"),
               dict(rotated=32, method="parts", trained=100, low=2.0, high=2.0)):
        with pytest.raises(ValueError):
            sa.rotary_turns(**kw)
