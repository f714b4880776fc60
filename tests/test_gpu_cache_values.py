"""Values that are not finite in the cache, against the formulas in 64 bits: a single token that does not see itself, and
infinities among the cached slots, by sign and place, whichever kernel a call runs."""
import math
import zlib

import pytest
import torch

import self_attention_gb300 as sa
import _cache_ref as ref
from _cache_plans import ROOM

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), math.inf


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


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("G", [1, 4, 9, 16, 17])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("C", [150, ROOM])
def test_a_single_token_that_does_not_see_itself(G, d, value, C):
    """Its own key and value reach nothing where its mask word leaves it out, and what sees it where the word does not."""
    g = _gen("single", G, d, str(value))
    B, H, lens = 5, 2, [0, 70, 70, 0, 95]
    q = _randn(g, B, H * G, 1, d, std=2.0)
    k, v = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    words = torch.tensor([0, 0, 1, 1, -2], device="cuda").view(B, 1)
    w = torch.rand(B, H, C, generator=g, device="cuda")
    for b, n in enumerate(lens):
        k[b, :, n + 1:], v[b, :, n + 1:] = NAN, NAN
        v[b, :, n, 3], v[b, :, n, d // 2:] = value, value
        if not int(words[b]) & 1:
            k[b, :, n] = value
    o, lse, out = sa.cache_attention(q, k, v, _i32(*lens), words, weights=w)
    want_o, want_l, want_w = ref.attention(q, k, v, lens, words.cpu(), w)
    assert not bool(o[0].any()) and bool((lse[0] == -INF).all())
    ref.check("o", o, *want_o)
    ref.check("lse", lse, *want_l)
    ref.check("weights", out, *want_w)
