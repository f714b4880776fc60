"""A block written with the public autograd operators alone trains: every leaf gets its gradient."""
import zlib

import pytest
import torch

import self_attention_gb300 as sa
import _block_ref as ref
from test_gpu_block import _block64, _params, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_attention_gb300.build import build
    sa.load_library(build())


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


@pytest.mark.parametrize("B,N,D,H,F", [(2, 130, 256, 4, 1000), (3, 196, 768, 12, 776)])
def test_every_leaf_of_a_block_gets_its_gradient(B, N, D, H, F):
    """Bounds as in test_gpu_block: three times the sum of the block's independent bf16 roundings."""
    g = _gen(B, N, D, H, F)
    p, x, dy = _params(g, D, F), _randn(g, B, N, D), _randn(g, B, N, D)
    leaves = {k: t.requires_grad_() for k, t in {**p, "x": x}.items()}
    n1 = sa.rms_norm(x, p["g1"])
    q, k, v = sa.qkv_proj(n1, p["wq"], p["wk"], p["wv"], H)
    h = sa.out_proj(sa.attention(q, k, v), p["wo"], p["bo"], residual=x)
    n2 = sa.rms_norm(h, p["g2"])
    y = sa.linear(sa.linear(n2, p["w1"], p["b1"], activation="gelu"), p["w2"], p["b2"], residual=h)
    y.backward(dy)
    leaves64 = {k: t.detach().double().requires_grad_() for k, t in leaves.items()}
    y64 = _block64(leaves64["x"], leaves64, H)
    y64.backward(dy.double())
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(y.detach(), y64.detach()) < 0.021
    for k, t in leaves.items():
        assert t.grad is not None, k
        assert t.grad.dtype == t.dtype and rel(t.grad, leaves64[k].grad) < 0.03, k
    assert sa.attn_get_device_status() == 0


def test_qkv_proj_with_and_without_a_graph():
    g = _gen("qkv")
    x = _randn(g, 2, 70, 128)
    ws = [_randn(g, 128, 128, std=0.1) for _ in range(3)]
    plain = sa.qkv_proj(x, *ws, 2)
    assert not any(t.requires_grad for t in plain)
    leaf = x.clone().requires_grad_()
    with torch.no_grad():
        assert not any(t.requires_grad for t in sa.qkv_proj(leaf, *ws, 2))
    got = sa.qkv_proj(leaf, *ws, 2)
    for a, b in zip(plain, got):
        assert torch.equal(a, b)
    douts = [_randn(g, 2, 2, 70, 64) for _ in range(3)]
    want = sa.qkv_proj_backward(x, *ws, *douts)
    torch.autograd.backward(got, douts)
    assert torch.equal(leaf.grad, want[0])
    # only a weight asked for, an output unused, a gradient with other strides
    wk = ws[1].clone().requires_grad_()
    _, k, _ = sa.qkv_proj(x, ws[0], wk, ws[2], 2)
    k.transpose(1, 2).backward(douts[1].transpose(1, 2))
    zero = torch.zeros_like(douts[0])
    assert torch.equal(wk.grad, sa.qkv_proj_backward(x, *ws, zero, douts[1], zero)[2].bfloat16())
    # on a stream given by object and by handle
    for by_handle in (False, True):
        st = torch.cuda.Stream()
        leaf.grad = None
        st.wait_stream(torch.cuda.current_stream())
        out = sa.qkv_proj(leaf, *ws, 2, stream=st.cuda_stream if by_handle else st)
        torch.cuda.current_stream().wait_stream(st)
        torch.autograd.backward(out, douts)
        torch.cuda.synchronize()
        assert torch.equal(leaf.grad, want[0])
    # a second derivative is refused, as the other operators do
    q, _, _ = sa.qkv_proj(leaf, *ws, 2)
    (gx,) = torch.autograd.grad(q.float().sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.float().sum().backward()
    assert sa.attn_get_device_status() == 0


def test_qkv_proj_against_the_formula_and_differences():
    """The products' gradients in 64 bits, and the 64-bit formula against a central difference."""
    g = _gen("qkv64")
    B, N, D, H = 1, 66, 128, 1
    x, ws = _randn(g, B, N, D).requires_grad_(), [_randn(g, D, D, std=0.1).requires_grad_() for _ in range(3)]
    douts = [_randn(g, B, H, N, D // H) for _ in range(3)]
    torch.autograd.backward(sa.qkv_proj(x, *ws, H), douts)
    x64, w64, d64 = x.detach().double(), [w.detach().double() for w in ws], [d.double().view(B * N, D) for d in douts]
    dx = sum(d @ w.T for d, w in zip(d64, w64))
    sums = sum(d.abs() @ w.abs().T for d, w in zip(d64, w64))
    tol = (3 * D + 8) * ref.STEP * sums
    ref.check("dx", x.grad.view(B * N, D), dx, tol + ref.U8 * (dx.abs() + tol))
    for w, d in zip(ws, d64):
        want = x64.view(-1, D).T @ d
        tol = (N + 8) * ref.STEP * (x64.view(-1, D).abs().T @ d.abs())
        ref.check("dw", w.grad, want, tol + ref.U8 * (want.abs() + tol))      # summed in fp32, rounded to w's type
    v, e = torch.randn(B * N, D, generator=g, device="cuda", dtype=torch.float64), 1e-4
    loss = lambda t: sum(((t @ w) * d).sum() for w, d in zip(w64, d64))  # noqa: E731
    diff = (loss(x64.view(-1, D) + e * v) - loss(x64.view(-1, D) - e * v)) / (2 * e)
    assert abs(float(diff - (dx * v).sum())) < 1e-6 * float((dx * v).abs().sum())


def test_a_block_captured_and_replayed():
    """Forward and backward of norm, QKV projection, attention and output projection in one graph, replayed on new
    inputs: what the eager pass gives (its sums of dQ and dW may meet in another order: a bf16 step)."""
    g = _gen("capture")
    B, N, D, H = 2, 100, 128, 2
    x, dy = _randn(g, B, N, D), _randn(g, B, N, D)
    leaves = [t.requires_grad_() for t in (x, 1 + _randn(g, D, std=0.1, dtype=torch.float32),
                                           *(_randn(g, D, D, std=0.1) for _ in range(4)))]

    def step():
        x, gain, wq, wk, wv, wo = leaves
        q, k, v = sa.qkv_proj(sa.rms_norm(x, gain), wq, wk, wv, H)
        y = sa.out_proj(sa.attention(q, k, v), wo, None, x)
        return (y.detach(), *torch.autograd.grad(y, leaves, dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        with torch.no_grad():
            x.copy_(_randn(g, B, N, D))
            dy.copy_(_randn(g, B, N, D))
        graph.replay()
        for a, b in zip(got, step()):
            assert float((a.double() - b.double()).norm()) <= 2 * ref.U8 * float(b.double().norm())
    assert sa.attn_get_device_status() == 0
