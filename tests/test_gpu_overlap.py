"""Chains of kernels that start while the one before them ends, each reading what that one has just written
into buffers that are used again and again with other values: the bits of the same calls one at a time."""
import zlib

import pytest
import torch

import self_attention_gb300 as sa

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


def _alone_and_chained(chain, sets, rounds=30):
    """chain(inputs, wait) enqueues its calls, calling wait() between them, and returns its outputs (of its own
    each time).  One at a time first, then all without a wait."""
    alone = []
    for s in sets:
        alone.append([t.clone() for t in chain(s, torch.cuda.synchronize)])
        torch.cuda.synchronize()
    got = [chain(sets[i % len(sets)], lambda: None) for i in range(rounds)]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        for a, b in zip(alone[i % len(sets)], out):
            assert torch.equal(a, b), i
    assert sa.attn_get_device_status() == 0


@pytest.mark.parametrize("M,K,N", [(1, 512, 256), (7, 2048, 512), (96, 256, 1024), (300, 512, 264), (2048, 256, 1032)])
def test_quantised_weights_and_rows_into_the_product(M, K, N):
    """quantize_q8 of the weights, then of the rows, then linear_q8: w_scale, x_scale and both operands have
    just been written."""
    g = _gen("q8", M, K, N)
    sets = [(_randn(g, M, K, std=2.0 ** i), _randn(g, N, K, std=2.0 ** -i)) for i in range(3)]
    bias = _randn(g, N, dtype=torch.float32)
    xq, xs = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(M, device="cuda")
    wq, ws = torch.empty(N, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(N, device="cuda")

    def chain(s, wait):
        y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        wait()
        sa.attn_quantize_q8(s[0], xq, xs, M, K)
        wait()
        sa.attn_quantize_q8(s[1], wq, ws, N, K)
        wait()
        sa.attn_linear_q8(xq, xs, wq, ws, bias, None, y, M, K, N, 0)
        wait()
        return [y]

    _alone_and_chained(chain, sets)


@pytest.mark.parametrize("M,K,D", [(1, 64, 256), (16, 256, 512), (196, 768, 768), (600, 520, 264), (3000, 128, 1032)])
def test_norm_gradient_into_a_layer(M, K, D):
    """The norm's backward writes dy (and its dweight is used as a bias), the layer before it sums dy for its
    bias gradient beside the products, and that gradient is the bias of the next product."""
    g = _gen("bwd", M, K, D)
    sets = [(_randn(g, M, D, std=2.0 ** i), _randn(g, M, D), torch.rand(M, generator=g, device="cuda") + 0.5)
            for i in range(3)]
    x, w, gain = _randn(g, M, K), _randn(g, K, D, std=0.1), torch.rand(D, generator=g, device="cuda") + 0.5
    dy, dgain = torch.empty(M, D, dtype=torch.bfloat16, device="cuda"), torch.empty(D, device="cuda")
    db = torch.empty(D, device="cuda")
    nb, lb = sa.attn_rms_norm_bwd_workspace_size(M, D), sa.attn_linear_bwd_workspace_size(M, K, D, 0)
    nws, lws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (nb, lb))

    def chain(s, wait):
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        y, n = torch.empty(M, D, dtype=torch.bfloat16, device="cuda"), torch.empty_like(dy)
        wait()
        sa.attn_rms_norm_bwd(s[0], s[1], gain, s[2], None, dy, dgain, nws, nb, M, D)
        wait()
        sa.attn_linear_bwd(x, w, dy, None, dx, dw, db, lws, lb, M, K, D, 0)
        wait()
        sa.attn_linear(x, w, db, dy, y, None, M, K, D, 0)
        wait()
        sa.attn_rms_norm(y, None, dgain, n, None, None, M, D, 1e-6)
        wait()
        return [dx, dw, y, n]

    _alone_and_chained(chain, sets)
