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


def _lay(v, lens, T, g):
    """Values that are not finite among the cached slots and the first token's: one of each kind alone in a column, the
    two infinities together, an infinity with NaN, and the same infinity twice; every chunk of columns has some."""
    B, H, _, d = v.shape
    for b, n in enumerate(lens):
        for h in range(H):
            at = torch.randint(0, n + 1, (d,), generator=g, device="cuda").tolist()      # (slot n: the first token's)
            for c in range(0, d, 3):
                kind = (c // 3 + h + b) % 7
                v[b, h, at[c], c] = (INF, -INF, NAN, INF, INF, -INF, INF)[kind]
                if kind in (3, 4, 5, 6) and at[c + 1 - (c == d - 1)] != at[c]:
                    v[b, h, at[c + 1 - (c == d - 1)], c] = (-INF, NAN, -INF, INF)[kind - 3]


# B, H, G, T, d, C, lengths
INFINITIES = [(2, 2, 1, 1, d, 130, [0, 129]) for d in (64, 128)]
INFINITIES += [(4, 2, G, T, d, C, [0, 7, 100, 299 - T]) for G, T in ((1, 1), (4, 1), (3, 3), (16, 1), (2, 8), (17, 1), (9, 20))
               for d in (64, 128) for C in (300, ROOM)]
INFINITIES += [(2, 2, 4, 1, d, ROOM, [39000, 777]) for d in (64, 128)]                       # parts, joined
INFINITIES += [(2, 2, 3, 5, d, ROOM, [39000, 777]) for d in (64, 128)]
INFINITIES += [(2, 2, 10, 5, d, ROOM, [39000, 777]) for d in (64, 128)]
INFINITIES += [(33, 3, 2, 2, d, 5000, [4990 - 151 * i for i in range(33)]) for d in (64, 128)]    # runs over several units
INFINITIES += [(40, 8, 1, 33, d, 300, [260 - 6 * i for i in range(40)]) for d in (64, 128)]      # whole units of larger tiles


def test_the_sizes_reach_every_kernel():
    plans = {sa.attn_debug_cache_plan(B, H, G, T, C, d)[:2] + (d,) for B, H, G, T, d, C, _ in INFINITIES}
    assert plans >= {(kind, rows, d) for kind in (1, 2) for rows in (8, 16) for d in (64, 128)}, plans
    assert {(3, 128), (4, 128)} <= {p[:2] for p in plans}, plans


@pytest.mark.parametrize("B,H,G,T,d,C,lens", INFINITIES, ids=lambda x: len(x) if isinstance(x, list) else x)
def test_infinities_among_the_cached_values(B, H, G, T, d, C, lens):
    """A sum of products with positive weights: infinite where one of its values is, by sign, NaN where both signs meet."""
    g = _gen("infinities", B, H, G, T, d, C)
    q = _randn(g, B, H * G, T, d)
    k, v = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    for b, n in enumerate(lens):
        k[b, :, n + T:], v[b, :, n + T:] = NAN, NAN
    clean = sa.cache_attention(q, k, v, _i32(*lens))
    _lay(v, lens, T, g)
    o, lse = sa.cache_attention(q, k, v, _i32(*lens))
    want_o, want_l = ref.attention_many(q, k, v, lens)
    ref.check("o", o, *want_o)
    ref.check("lse", lse, *want_l)
    assert bool(want_o[0].isinf().any()) and bool(want_o[0].isnan().any()) and torch.equal(lse, clean[1])
    columns = v[:, :, :1].new_zeros(B, H, 1, d)
    for b, n in enumerate(lens):
        columns[b] = (~v[b, :, :n + T].isfinite()).any(1, keepdim=True).to(v.dtype)
    same = (columns == 0).repeat_interleave(G, 1).expand_as(o)
    assert torch.equal(o[same], clean[0][same])              # the other columns are as they were
    assert sa.attn_get_device_status() == 0


def test_a_row_without_weights_stays_nan():
    """Queries that are not finite make their own rows NaN, whatever the values are."""
    g = _gen("nan rows")
    B, H, G, d, C = 2, 2, 4, 128, 1000
    q, k, v = _randn(g, B, H * G, 1, d), _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    q[0, 1, 0, 7], q[1, 6] = NAN, NAN
    v[:, :, 11, 5], v[:, :, 500, 6] = INF, -INF
    o, lse = sa.cache_attention(q, k, v, _i32(990, 30))
    bad = torch.zeros(B, H * G, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 6] = True
    assert bool(o[bad].isnan().all()) and bool(lse[bad].isnan().all())
    good = o[~bad]
    assert bool((good[..., 5] == INF).all()) and not bool(lse[~bad].isnan().any())
    seen = o[0][~bad[0]]
    assert bool((seen[..., 6] == -INF).all()) and not bool(good.isnan().any())


@pytest.mark.parametrize("G,d,C", [(1, 64, 300), (4, 128, 300), (16, 64, 300), (3, 128, ROOM), (12, 64, ROOM), (16, 128, ROOM), (20, 64, ROOM)])
def test_large_values_under_small_weights(G, d, C):
    """Weights 2^(-33 j / 4) of 16 slots that one warp takes, under values of 2^(8 j + 4): each product is held to its weight's
    rounding, not to an absolute one."""
    B, H, n = 1, 2, 16
    k, v = (torch.zeros(B, H, C, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, H * G, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0], q[..., 1] = 1, 0.25
    j = torch.arange(n, device="cuda").float()
    k[..., :n, 0], k[..., :n, 1] = -8 * j, -j                    # score j is exact: -33 j / 4
    c = torch.arange(d, device="cuda")                           # a column has one value, at slot c % 16
    v[:, :, c % n, c] = torch.exp2(8.0 * (c % n) + 4).to(torch.bfloat16)
    o, lse = sa.cache_attention(q, k, v, _i32(n - 1), scale=math.log(2.0))
    weights = torch.exp2(-33 * j.double() / 4)
    want = (weights[c % n] / weights.sum() * torch.exp2(8.0 * (c % n).double() + 4)).expand_as(o)
    # the scale, its product with log2 e and with the score are rounded (2^-24 each of at most 124 units of ln 2); the weight's
    # 2^-8 and o's
    tol = want * (3 * 124 * 2.0 ** -24 + 2.0 ** -8 + 2.0 ** -8 * 1.01)
    ref.check("o", o, want, tol)
    assert (lse.double() - math.log(weights.sum().item())).abs().max() < 1e-5
    low = c % n <= 12                                            # weights down to 2^-99: infinite values there keep their sign
    for value in (INF, -INF):
        v[:, :, (c % n)[low], c[low]] = value
        o2, lse2 = sa.cache_attention(q, k, v, _i32(n - 1), scale=math.log(2.0))
        assert bool((o2[..., low] == value).all()) and torch.equal(o2[..., ~low], o[..., ~low]) and torch.equal(lse2, lse)
