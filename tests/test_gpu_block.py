"""The operators of a transformer block as they are used together: norm, QKV projection, attention,
output projection onto the residual stream, norm, and the two linear layers of the MLP; training
(forward and backward) in bf16, and the MLP of a few tokens in 8 bits."""
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


class _QkvProj(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, wq, wk, wv, H):
        ctx.save_for_backward(x, wq, wk, wv)
        return sa.qkv_proj(x, wq, wk, wv, H)

    @staticmethod
    def backward(ctx, dq, dk, dv):
        return (*sa.qkv_proj_backward(*ctx.saved_tensors, dq.contiguous(), dk.contiguous(), dv.contiguous()), None)


def _params(g, D, F):
    p = {"g1": 1 + _randn(g, D, std=0.1, dtype=torch.float32), "g2": 1 + _randn(g, D, std=0.1, dtype=torch.float32),
         "bo": _randn(g, D, std=0.1, dtype=torch.float32), "b1": _randn(g, F, std=0.1, dtype=torch.float32),
         "b2": _randn(g, D, std=0.1, dtype=torch.float32)}
    for n, shape in (("wq", (D, D)), ("wk", (D, D)), ("wv", (D, D)), ("wo", (D, D)), ("w1", (D, F)), ("w2", (F, D))):
        p[n] = _randn(g, *shape, std=shape[0] ** -0.5)
    return p


def _block(x, p, H):
    n1 = sa.rms_norm(x, p["g1"])
    q, k, v = _QkvProj.apply(n1, p["wq"], p["wk"], p["wv"], H)
    h1 = sa.out_proj(sa.attention(q, k, v), p["wo"], p["bo"], x)
    u = sa.linear(sa.rms_norm(h1, p["g2"]), p["w1"], p["b1"], None, "gelu")
    return sa.linear(u, p["w2"], p["b2"], h1)


def _block64(x, p, H):
    B, N, D = x.shape
    heads = lambda t: t.view(B, N, H, D // H).transpose(1, 2)  # noqa: E731
    n1 = ref.rms_norm(x, p["g1"])[0]
    q, k, v = (heads(n1 @ p[w]) for w in ("wq", "wk", "wv"))
    a = torch.softmax(q @ k.transpose(-1, -2) / (D // H) ** 0.5, -1) @ v
    h1 = a.transpose(1, 2).reshape(B, N, D) @ p["wo"] + p["bo"] + x
    u = ref.act(ref.rms_norm(h1, p["g2"])[0] @ p["w1"] + p["b1"], "gelu")
    return u @ p["w2"] + p["b2"] + h1


@pytest.mark.parametrize("B,N,D,H,F", [(2, 130, 256, 4, 1000), (1, 1, 128, 1, 512), (3, 196, 768, 12, 776)])
def test_block_forward_and_backward(B, N, D, H, F):
    """Against the block in 64 bits.  Each of the ten or so bf16 roundings on the way to y is uniform
    within half a step (root mean square 2^-8 / sqrt 3 of the value at most) and enters about as large
    as it is, independent of the others: sqrt(10) 2^-8 / sqrt 3 = 0.7 % of y in the 2-norm, twice as
    many for a gradient 1 %; the bounds are three times that."""
    g = torch.Generator(device="cuda").manual_seed(zlib.crc32(repr((B, N, D, H, F)).encode()))
    p, x, dy = _params(g, D, F), _randn(g, B, N, D), _randn(g, B, N, D)
    leaves = {k: t.requires_grad_() for k, t in {**p, "x": x}.items()}
    y = _block(x, p, H)
    y.backward(dy)
    leaves64 = {k: t.detach().double().requires_grad_() for k, t in leaves.items()}
    y64 = _block64(leaves64["x"], leaves64, H)
    y64.backward(dy.double())
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(y.detach(), y64.detach()) < 0.021
    for k, t in leaves.items():
        if N == 1 and k in ("wq", "wk"):     # one key: the softmax is constant, the gradient zero
            assert float(t.grad.abs().max()) < 1e-3
            continue
        assert rel(t.grad, leaves64[k].grad) < 0.03, k
    assert sa.attn_get_device_status() == 0


@pytest.mark.parametrize("M,D,F", [(1, 1024, 4096), (5, 256, 1008), (150, 512, 2048)])
def test_mlp_in_8_bits(M, D, F):
    """norm -> 8 bits -> up projection with GELU -> 8 bits -> down projection onto the residual
    stream; each product against the 64-bit one of the values its inputs stand for."""
    g = torch.Generator(device="cuda").manual_seed(zlib.crc32(repr((M, D, F)).encode()))
    x, res = _randn(g, M, D), _randn(g, M, D)
    gw, b1 = 1 + _randn(g, D, std=0.1, dtype=torch.float32), _randn(g, F, std=0.1, dtype=torch.float32)
    w1 = sa.quantize_q8(_randn(g, F, D, std=D ** -0.5))
    w2 = sa.quantize_q8(_randn(g, D, F, std=F ** -0.5))
    deq = lambda q, s: q.double() * s.double()[..., None]  # noqa: E731
    nq, ns, h = sa.rms_norm_q8(x, gw, res)
    u = sa.linear_q8(nq, ns, *w1, b1, None, "gelu")
    uq, us = sa.quantize_q8(u)
    y = sa.linear_q8(uq, us, *w2, None, h)
    ry, _, ty, _ = ref.linear(deq(nq, ns), deq(*w1).T, b1, None, "gelu")
    ref.check("u", u, ry, ty)
    ry, _, ty, _ = ref.linear(deq(uq, us), deq(*w2).T, None, h)
    ref.check("y", y, ry, ty)
    assert sa.attn_get_device_status() == 0
