"""The linear layers at the most rows they take: row numbers next to 2^31."""
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


def test_the_most_rows():
    """2^31 - 256 rows of 8 columns (34 GB in, 34 GB out), each the numbers of a small pattern: every row is
    compared with its pattern's, a 64-bit reference's."""
    M, P = (1 << 31) - 256, 1 << 15
    g = torch.Generator(device="cuda").manual_seed(17)
    pattern, w = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((P, 8), (8, 8)))
    bias = torch.randn(8, generator=g, device="cuda")
    x = torch.empty(M, 8, dtype=torch.bfloat16, device="cuda")
    whole = M // P * P
    x[:whole].view(-1, P, 8).copy_(pattern)
    x[whole:] = pattern[:M - whole]
    y = sa.linear_forward(x, w, bias)
    want, _, tol, _ = ref.linear(pattern, w, bias)
    few = sa.linear_forward(pattern[:64], w, bias)
    ref.check("few rows", few, want[:64], tol[:64])
    ref.check("first", y[:P], want, tol)
    step = P * 4096
    for at in range(0, whole, step):
        part = y[at:min(at + step, whole)].view(-1, P, 8)
        assert bool((part == y[:P]).all()), at
    ref.check("last", y[whole:], want[:M - whole], tol[:M - whole])
    assert sa.attn_get_device_status() == 0
