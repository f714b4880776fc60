"""Calls on some of a batch's rows: the rows' scales and 1/rms then start on any element."""
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


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("first", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("M,K,N", [(9, 256, 136), (300, 512, 264)])
def test_rows_from_any_on(M, K, N, first):
    """The same bits as from a copy of the rows, on the current stream, another one, and captured."""
    g = _gen(M, K, N)
    xq, xs = sa.quantize_q8(_randn(g, M, K))
    wq, ws = sa.quantize_q8(_randn(g, N, K))
    gain, dy = torch.rand(K, generator=g, device="cuda") + 0.5, _randn(g, M, K)
    _, h, rstd = sa.rms_norm_forward(_randn(g, M, K), gain)
    want = (sa.linear_q8(xq[first:].clone(), xs[first:].clone(), wq, ws),
            *sa.rms_norm_backward(dy[first:].clone(), h[first:].clone(), gain, rstd[first:].clone()))

    def run(stream=None):
        return (sa.linear_q8(xq[first:], xs[first:], wq, ws, stream=stream),
                *sa.rms_norm_backward(dy[first:], h[first:], gain, rstd[first:], stream=stream))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    results = [run(), run(side)]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results.append(run())
    graph.replay()
    for got in results:
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    assert sa.attn_get_device_status() == 0
