"""The cache on the GPU: append, attention of single, chained and drafted tokens, accumulated weights and eviction,
against the formulas in 64 bits within derived bounds (see _cache_ref)."""
import math
import zlib

import pytest
import torch

import self_attention_gb300 as sa
import _cache_ref as ref
from _cache_plans import BLOCKS, CASES, ODD, POISON, ROOM

pytestmark = pytest.mark.gpu
NAN = float("nan")


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


def _parents(g, B, T):
    r = torch.rand(B, T, generator=g, device="cuda").cpu()
    return [[int(r[b, t] * (t + 1)) - 1 for t in range(T)] for b in range(B)]


def _cache(g, B, H, C, d, lengths, T, behind=NAN):
    """k, v with `behind` in every slot that no token has."""
    k, v = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), C - T)
        k[b, :, n + T:], v[b, :, n + T:] = behind, behind
    return k, v


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("B,H,Hq,T,d,C,rotated", [(1, 1, 1, 1, 64, 8, 64), (3, 2, 6, 5, 128, 40, 64),
                                                  (32, 4, 16, 1, 128, 100, 128), (2, 5, 5, 300, 64, 333, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_append(B, H, Hq, T, d, C, rotated, interleaved, given):
    g = _gen(B, H, T, d, interleaved, given)
    lens = [(7 * b) % (C - T + 1) for b in range(B)]
    k, v, q = _randn(g, B, H, T, d), _randn(g, B, H, T, d), _randn(g, B, Hq, T, d)
    ck, cv = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    w = torch.rand(B, H, C, generator=g, device="cuda")
    slots = torch.full((B, H, C), -7, dtype=torch.int32, device="cuda")
    was = [t.clone() for t in (ck, cv, w, slots)]
    positions = torch.randint(0, 99999, (B, T), generator=g, device="cuda", dtype=torch.int32) if given else None
    at = positions.cpu() if given else torch.tensor(lens).view(B, 1) + torch.arange(T)
    out = sa.cache_append(k, v, ck, cv, _i32(*lens), sa.rotary_turns(rotated), positions, interleaved, 1.5, q=q,
                          weights=w, slot_positions=slots)
    f = ref.frequencies(rotated)
    ref.check("q", out, *ref.turned(q.cpu(), at, f, interleaved, 1.5))
    want, tol = ref.turned(k.cpu(), at, f, interleaved, 1.5)
    for b, n in enumerate(lens):
        ref.check("k", ck[b, :, n:n + T], want[b], tol[b])
        assert torch.equal(cv[b, :, n:n + T], v[b]) and not bool(w[b, :, n:n + T].any())
        assert torch.equal(slots[b, :, n:n + T].cpu(), at[b].int().expand(H, T))
        for t in (ck, cv, w, slots):        # nothing else is touched
            old = was[[ck is t, cv is t, w is t, slots is t].index(True)]
            assert torch.equal(t[b, :, :n], old[b, :, :n]) and torch.equal(t[b, :, n + T:], old[b, :, n + T:])


def test_append_of_rows_and_lengths_out_of_range():
    g = _gen("rows")
    B, H, T, d, C = 4, 3, 6, 64, 20
    k, v = _randn(g, B, H, T, d), _randn(g, B, H, T, d)
    ck, cv = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    was_k, was_v = ck.clone(), cv.clone()
    rows = torch.tensor([[0, 2, 5], [1, -1, 3], [6, 4, 4], [0, 1, 2]], dtype=torch.int32, device="cuda")
    lens = [3, 0, -9, 18]
    assert sa.cache_append(k, v, ck, cv, _i32(*lens), rows=rows) is None       # no turns: copied
    for b, n in enumerate(lens):
        n = max(n, 0)
        want_k, want_v = was_k[b].clone(), was_v[b].clone()
        for i, r in enumerate(rows[b].tolist()):
            if 0 <= r < T and n + i < C:
                want_k[:, n + i], want_v[:, n + i] = k[b, :, r], v[b, :, r]
        assert torch.equal(ck[b], want_k) and torch.equal(cv[b], want_v)
    ck.copy_(was_k)
    sa.cache_append(k, v, ck, cv, _i32(C, C + 5, 2 ** 31 - 1, C))             # full: nothing is written
    assert torch.equal(ck, was_k)
    sa.cache_append(k[:, :, :0].contiguous(), v[:, :, :0].contiguous(), ck, cv, _i32(0, 0, 0, 0))
    assert torch.equal(ck, was_k)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])))
@pytest.mark.parametrize("masked,room", [(False, 0), (True, 0), (True, ROOM)])
def test_attention(case, masked, room):
    B, H, G, T, d, C, lens = case
    C = max(C, room)
    g = _gen(case, masked)
    q = _randn(g, B, H * G, T, d, std=2.0)
    k, v = _cache(g, B, H, C, d, lens, T)
    tree = sa.tree_words(_parents(g, B, T)) if masked else None
    o, lse = sa.cache_attention(q, k, v, _i32(*lens), tree)
    want_o, want_l, _ = ref.attention(q, k, v, lens, tree)
    ref.check("o", o, *want_o)
    ref.check("lse", lse, *want_l)
    again = sa.cache_attention(q, k, v, _i32(*lens), tree)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])))
@pytest.mark.parametrize("some,room", [(False, 0), (True, 0), (True, ROOM)])
def test_weights(case, some, room):
    B, H, G, T, d, C, lens = case
    C = max(C, room)
    g = _gen(case, some, "weights")
    q = _randn(g, B, H * G, T, d, std=2.0)
    k, v = _cache(g, B, H, C, d, lens, T)
    w = torch.rand(B, H, C, generator=g, device="cuda")
    tree = sa.tree_words(_parents(g, B, T))
    counted = torch.tensor([(0x5A5A5A5A5A5A5A5B * (b + 1)) % 2 ** 63 for b in range(B)], device="cuda") if some else None
    was = w.clone()
    o, lse, out = sa.cache_attention(q, k, v, _i32(*lens), tree, weights=w, counted=counted)
    assert torch.equal(w, was)
    want_o, want_l, want_w = ref.attention(q, k, v, lens, tree, w, counted)
    ref.check("o", o, *want_o)
    ref.check("lse", lse, *want_l)
    ref.check("weights", out, *want_w)
    o2, lse2, out2 = sa.cache_attention(q, k, v, _i32(*lens), tree, weights=w, counted=counted, weights_out=w)
    assert out2 is w and torch.equal(out, w) and torch.equal(o, o2) and torch.equal(lse, lse2)
    plain = sa.cache_attention(q, k, v, _i32(*lens), tree)
    assert torch.equal(o, plain[0]) and torch.equal(lse, plain[1])


@pytest.mark.parametrize("B,H,G,T,d,C,ragged", BLOCKS)
@pytest.mark.parametrize("masked", [False, True])
def test_attention_over_many_blocks(B, H, G, T, d, C, ragged, masked):
    """CTAs with runs of blocks, and runs over several heads and sequences."""
    g = _gen("blocks", B, H, G, T, d, masked)
    lens = [C - T - (b * 977) % (ragged + 1) for b in range(B)]
    q = _randn(g, B, H * G, T, d, std=2.0)
    k, v = _cache(g, B, H, C, d, lens, T)
    tree = sa.tree_words(_parents(g, B, T)) if masked else None
    o, lse = sa.cache_attention(q, k, v, _i32(*lens), tree)
    assert sa.attn_get_device_status() == 0
    want_o, want_l = ref.attention_many(q, k, v, lens, tree)
    ref.check("o", o, *want_o)
    ref.check("lse", lse, *want_l)
    again = sa.cache_attention(q, k, v, _i32(*lens), tree)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("T,G,d", ODD)
@pytest.mark.parametrize("C", [150, ROOM])
def test_rows_that_see_nothing_or_odd_sets(T, G, d, C):
    """Masks that are no trees: empty rows, a row that sees only others, all bits."""
    g = _gen("odd", T, G)
    B, H = 3, 2
    lens = [0, 0, 70]
    q = _randn(g, B, H * G, T, d, std=2.0)
    k, v = _cache(g, B, H, C, d, lens, T)
    words = torch.randint(-(2 ** 63), 2 ** 63 - 1, (B, T), generator=g, device="cuda")
    words[:, 0] = 0
    words[0] = 0
    words[1, 1] = -1
    words[2, 2] = 1 << (T - 1) if T < 64 else -(2 ** 63)
    w = torch.rand(B, H, C, generator=g, device="cuda")
    o, lse, out = sa.cache_attention(q, k, v, _i32(*lens), words, weights=w)
    want_o, want_l, want_w = ref.attention(q, k, v, lens, words.cpu(), w)
    assert not bool(o[0].any()) and bool((lse[0] == -math.inf).all())
    ref.check("o", o, *want_o)
    ref.check("lse", lse, *want_l)
    ref.check("weights", out, *want_w)


@pytest.mark.parametrize("T,G,d", POISON)
@pytest.mark.parametrize("value", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("C", [300, ROOM])
def test_what_a_row_does_not_see_does_not_reach_it(T, G, d, value, C):
    """A drafted token whose key and value are not finite spoils its descendants' rows alone."""
    g = _gen("poison", T, G, d, str(value))
    B, H, n = 2, 2, [200, 3]
    q = _randn(g, B, H * G, T, d)
    k, v = _cache(g, B, H, C, d, n, T)
    parents = _parents(g, B, T)
    parents[0][1] = parents[1][1] = 0
    tree = sa.tree_words(parents)
    clean = sa.cache_attention(q, k, v, _i32(*n), tree)
    for b in range(B):
        v[b, :, n[b] + 1, 5] = value
        v[b, :, n[b] + T - 1, d - 1] = value
    o, lse = sa.cache_attention(q, k, v, _i32(*n), tree)
    assert torch.equal(lse, clean[1])
    sees = (tree.unsqueeze(-1) >> torch.tensor([1, T - 1], device="cuda") & 1).bool().view(B, 1, T, 2)
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[..., 5] = sees[..., 0]
    bad[..., d - 1] |= sees[..., 1]
    assert torch.equal(o.isfinite(), ~bad)
    assert torch.equal(o[~bad], clean[0][~bad])
    k[0, :, n[0] + 1] = value                    # a key: the rows that see it have no weights at all
    o, lse = sa.cache_attention(q, k, v, _i32(*n), tree)
    safe = ~sees[0, 0, :, 0]
    assert torch.equal(lse[0][:, safe], clean[1][0][:, safe])
    keep = safe.view(1, T, 1) & ~bad[0]
    assert torch.equal(o[0][keep.expand_as(o[0])], clean[0][0][keep.expand_as(o[0])])


def test_lengths_out_of_range_are_taken_as_the_nearest():
    g = _gen("range")
    B, H, G, T, d, C = 4, 2, 2, 3, 64, 90
    q, k, v = _randn(g, B, H * G, T, d), _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    got = sa.cache_attention(q, k, v, _i32(-1, C, -2 ** 31, 2 ** 31 - 1))
    want = sa.cache_attention(q, k, v, _i32(0, C - T, 0, C - T))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_large_scores_and_scales():
    """Scores of thousands: one slot takes everything; a small scale: all alike."""
    g = _gen("large")
    B, H, T, d, C = 2, 2, 2, 128, 300
    q, k, v = _randn(g, B, H, T, d, std=40.0), _randn(g, B, H, C, d, std=10.0), _randn(g, B, H, C, d)
    for scale in (1.0, 1e-4):
        o, lse = sa.cache_attention(q, k, v, _i32(298, 100), scale=scale)
        want_o, want_l, _ = ref.attention(q, k, v, [298, 100], scale=scale)
        ref.check("o", o, *want_o)
        ref.check("lse", lse, *want_l)


def test_chain_is_attention_over_a_prefix():
    """A token over a cache of n is the framework's attention of its row over n + 1 keys."""
    g = _gen("prefix")
    B, H, N, d = 2, 4, 257, 64
    q, k, v = _randn(g, B, H, N, d), _randn(g, B, H, N, d), _randn(g, B, H, N, d)
    o, lse = sa.forward(q, k, v)
    one, l1 = sa.cache_attention(q[:, :, -1:].contiguous(), k, v, _i32(N - 1, N - 1))
    assert (lse[:, :, -1:] - l1).abs().max() < 1e-3
    assert (o[:, :, -1:].float() - one.float()).abs().max() < 1e-2


@pytest.mark.parametrize("G,T", [(1, 1), (2, 64)])
def test_cache_past_2_31_elements(G, T):
    """The last head of a cache of 2^32 bytes and more."""
    B, H, C, d = 1, 17, 1 << 20, 128
    n = C - T
    g = _gen("huge", G)
    k = torch.zeros(B, H, C, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(B, H, C, d, dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 2 ** 31
    q = _randn(g, B, H * G, T, d)
    v[:, -1, :, :] = 1
    k[:, -1, -T - 1, :] = 4 * q[:, -1, 0]
    v[:, -1, -T - 1, :] = 3
    o, lse = sa.cache_attention(q, k, v, _i32(n))
    s = (4 * q[:, -1, 0].double()).square().sum() / 4 / math.sqrt(d)
    z = torch.logsumexp(torch.tensor([s.item()] + [0.0] * 0), 0)
    want = torch.logaddexp(s.cpu(), torch.tensor(math.log(n), dtype=torch.float64))
    assert abs(lse[0, -1, 0].item() - want.item()) < 1e-3 * (1 + abs(want.item())) and z is not None
    share = math.exp(s.item() - want.item())
    assert abs(o[0, -1, 0].float().mean().item() - (3 * share + 1 * (1 - share))) < 3e-2
    assert not bool(o[0, 0].any())


def test_refusals():
    B, H, G, T, d, C = 2, 2, 3, 4, 64, 40
    q = torch.zeros(B, H * G, T, d, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(B, H, C, d, dtype=torch.bfloat16, device="cuda")
    v, n = k.clone(), _i32(1, 2)
    w, tree = torch.zeros(B, H, C, device="cuda"), torch.zeros(B, T, dtype=torch.int64, device="cuda")
    sa.cache_attention(q, k, v, n, tree, weights=w, counted=tree[:, 0].contiguous())
    assert len(sa.cache_attention(q, k, v, n, tree, counted=tree[:, 0].contiguous())) == 2     # of no account alone
    bad = [dict(q=q.float()), dict(q=q[0]), dict(q=q.transpose(1, 2)), dict(q=q[:, :5].contiguous()), dict(q=q.cpu()),
           dict(k=k.half()), dict(k=k[:1]), dict(v=v[:, :, :-1].contiguous()), dict(v=v.float()), dict(n=n.long()),
           dict(n=n[:1]), dict(n=n.cpu()), dict(tree=tree.int()), dict(tree=tree[:, :2].contiguous()),
           dict(weights=w.double()), dict(weights=w[..., :-1].contiguous()), dict(weights=None, weights_out=w),
           dict(weights_out=w.double()), dict(counted=n)]
    for kw in bad:
        a = dict(q=q, k=k, v=v, n=n, tree=tree, weights=w)
        a.update(kw)
        with pytest.raises(ValueError):
            sa.cache_attention(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("n"), **a)
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=math.inf)):
        with pytest.raises(sa.AttnError):
            sa.cache_attention(q, k, v, n, **kw)
    big = torch.zeros(B, H, 65, d, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(sa.AttnError):                                # more than 64 tokens
        sa.cache_attention(big, torch.zeros(B, H, 100, d, dtype=torch.bfloat16, device="cuda"),
                           torch.zeros(B, H, 100, d, dtype=torch.bfloat16, device="cuda"), n)
    with pytest.raises(sa.AttnError):                                # more tokens than slots
        sa.cache_attention(q, k[:, :, :3].contiguous(), v[:, :, :3].contiguous(), n)
    with pytest.raises(sa.AttnError):
        sa.cache_attention(*(torch.zeros(1, 1, 2, 96, dtype=torch.bfloat16, device="cuda") for _ in range(3)), _i32(0))
    for p in ([[0, 0]], [[-1, 1]], [[]], [[-1], [-1, 0]], [[-1] * 65]):
        with pytest.raises(ValueError):
            sa.tree_words(p)
    with pytest.raises(ValueError):
        sa.cache_append(q, q, k, v, n)
    new = torch.zeros(B, H, T, d, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
    for kw in (dict(rows=rows.long()), dict(rows=rows[:1]), dict(rows=rows, q=q), dict(q=q.float()),
               dict(q=q[:, :, :2].contiguous()), dict(positions=rows), dict(weights=w.half()),
               dict(slot_positions=w), dict(turns=rows)):
        with pytest.raises(ValueError):
            sa.cache_append(new, new, k, v, n, **kw)
    with pytest.raises(sa.AttnError):                                # into the tokens themselves
        sa.cache_append(new, new, new, v[:, :, :T].contiguous(), n)
    with pytest.raises(sa.AttnError):                                # k and v into one cache
        sa.cache_append(new, new, k, k, n)
    slots = torch.zeros(B, H, C, dtype=torch.int32, device="cuda")
    # no backward: what a graph is recorded for is refused, without one it is taken
    wants = q.clone().requires_grad_()
    with pytest.raises(ValueError, match="no backward"):
        sa.cache_attention(wants, k, v, n)
    with pytest.raises(ValueError, match="no backward"):
        sa.cache_append(new.clone().requires_grad_(), new, k, v, n)
    with pytest.raises(ValueError, match="no backward"):
        sa.cache_evict(k, v, w.clone().requires_grad_(), slots, n, 4)
    with torch.no_grad():
        assert not sa.cache_attention(wants, k, v, n)[0].requires_grad
    for kw in (dict(keep=0), dict(keep=-1), dict(keep=4, recent=5), dict(keep=4, recent=-1), dict(keep=2 ** 40)):
        with pytest.raises(sa.AttnError):
            sa.cache_evict(k, v, w, slots, n, **kw)
    for a in ((k, v, w.double(), slots, n), (k, v, w, slots.long(), n), (k, v, w, slots, n.long()),
              (k, v[:, :, :9].contiguous(), w, slots, n), (k, v, w[..., :9].contiguous(), slots, n)):
        with pytest.raises(ValueError):
            sa.cache_evict(*a, 4)
    with pytest.raises(sa.AttnError):
        sa.cache_evict(k, k, w, slots, n, 4)


# ------------------------------------------------------------------ eviction
def _evict_case(g, B, H, C, d):
    k, v = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    w = torch.rand(B, H, C, generator=g, device="cuda") ** 6 * 20
    pos = torch.rand(B, H, C, generator=g, device="cuda").argsort(-1).to(torch.int32)
    return k, v, w, pos


def _check_evict(k, v, w, pos, lens, keep, recent, in_place=False):
    want = ref.evict(k, v, w, pos, lens, keep, recent)
    where = dict(weights_out=w, positions_out=pos) if in_place else {}
    w2, p2, n2 = sa.cache_evict(k, v, w, pos, _i32(*lens), keep, recent, **where)
    for name, got, x in zip(("k", "v", "weights", "positions", "lengths"), (k, v, w2, p2, n2), want):
        x = x.to(got.device)
        same = (got == x) | (got.isnan() & x.isnan()) if got.is_floating_point() else got == x
        assert bool(same.all()), (name, same.logical_not().nonzero()[:5].tolist())
    return w2, p2, n2


@pytest.mark.parametrize("B,H,C,d,lens,keep,recent", [
    (1, 1, 1, 64, [1], 1, 0), (1, 1, 2, 128, [2], 1, 1), (1, 1, 2, 64, [2], 1, 0),
    (3, 2, 100, 64, [100, 64, 3], 64, 10), (2, 3, 1025, 128, [1025, 1000], 1000, 100),
    (2, 1, 5000, 64, [5000, 4097], 33, 33), (4, 2, 300, 128, [0, 300, 1, 77], 76, 0),
    (1, 2, 2500, 64, [2500], 2499, 1), (1, 1, 3000, 128, [2999], 1500, 700), (2, 2, 40, 64, [40, 39], 50, 50),
    (1, 1, 20000, 64, [19999], 9000, 100), (3, 4, 9000, 128, [9000, 1000, 8123], 999, 998), (10, 5, 4200, 64, [4200 - 7 * i for i in range(10)], 4100, 1),
    (30, 5, 1100, 64, [1100] * 30, 1000, 5), (1, 3, 16400, 128, [5], 3, 1),
    (16, 8, 3000, 128, [3000 - 11 * i for i in range(16)], 1400, 100), (4, 8, 9000, 128, [9000, 8999, 4000, 0], 4500, 50),
    (40, 4, 1100, 64, [1100 - i for i in range(40)], 1000, 5), (4, 40, 1100, 128, [1100, 1000, 501, 31], 500, 50),
    (2, 90, 5001, 128, [5001, 4000], 2400, 100), (2, 80, 8192, 64, [8192, 8000], 900, 10), (2, 80, 8193, 64, [8193, 33], 900, 10)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(B, H, C, d, lens, keep, recent, in_place):
    g = _gen(B, H, C, lens, keep, recent, in_place)
    _check_evict(*_evict_case(g, B, H, C, d), lens, keep, recent, in_place)


def test_evict_ties_and_odd_weights():
    g = _gen("ties")
    B, H, C, d = 2, 2, 2300, 64
    k, v, w, pos = _evict_case(g, B, H, C, d)
    w = (w * 2).floor().clamp_max(3.0)                       # a handful of values, most of them zero
    w[0, 0, 5], w[0, 0, 2000], w[0, 1, 7], w[1, 0, 1111] = NAN, -3.0, math.inf, -math.inf
    w[1, 1] = 0
    _check_evict(*(t.repeat(1, 40, *[1] * (t.dim() - 2)) for t in (k, v, w, pos)), [2300, 2200], 900, 50)
    _check_evict(k, v, w, pos, [2300, 2200], 900, 50)
    k, v, w, pos = _evict_case(g, B, H, C, d)
    w[0, 0] = 1e-42                                          # subnormal
    w[0, 0, 1500:] = 2e-42
    pos[1] = 3                                               # one position everywhere: all are the newest
    _check_evict(k, v, w, pos, [2300, 2300], 700, 20)


def test_evict_of_a_long_cache():
    """More slots than fit shared memory."""
    g = _gen("long")
    for B, H, C, in_place in ((1, 1, 400001, False), (1, 1, 400001, True), (1, 77, 49999, True)):
        k, v, w, pos = _evict_case(g, B, H, C, 64)           # by 8 blocks a head, by one
        _check_evict(k, v, w, pos, [C] * B, 20000, 999, in_place)
    k, v, w, pos = _evict_case(g, 1, 2, 400001, 64)          # few slots in use of many
    _check_evict(k, v, w, pos, [3000], 2000, 99)


def test_evict_of_whole_halves():
    """All that stays lies behind all that goes: as many moves as slots stay, around what a block's list holds."""
    g = _gen("halves")
    k, v, w, pos = _evict_case(g, 1, 1, 6300, 64)
    w = torch.arange(6300, device="cuda").float().repeat(1, 80, 1)
    for heads, keep in ((80, 3070), (80, 3071), (80, 3073), (160, 2000), (160, 3071)):
        ks, vs = k.repeat(1, heads, 1, 1), v.repeat(1, heads, 1, 1)
        _check_evict(ks, vs, w[:, :1].repeat(1, heads, 1), pos.repeat(1, heads, 1), [6300], keep, 0)


def test_evict_leaves_the_rest():
    """Slots that nothing moves into keep their keys and values, those behind the last among them."""
    g = _gen("rest")
    k, v, w, pos = _evict_case(g, 1, 1, 128, 64)
    k[:, :, 100:], v[:, :, 100:] = NAN, NAN
    was = k.clone()
    _check_evict(k, v, w, pos, [100], 60, 5)
    assert bool(k[:, :, 100:].isnan().all()) and torch.equal(k[:, :, 60:100], was[:, :, 60:100])


# ------------------------------------------------------------------ together
def test_decoding_with_drafts_and_eviction():
    """A prompt, drafted trees, the accepted path, eviction, the next token: each step against the formulas."""
    g = _gen("together")
    B, H, G, d, C = 2, 2, 2, 64, 256
    turns, f = sa.rotary_turns(32), ref.frequencies(32)
    ck, cv = (torch.full((B, H, C, d), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.zeros(B, H, C, device="cuda")
    slots = torch.full((B, H, C), -1, dtype=torch.int32, device="cuda")
    lengths = _i32(0, 0)
    N = 150
    k, v = _randn(g, B, H, N, d), _randn(g, B, H, N, d)
    sa.cache_append(k, v, ck, cv, lengths, turns, weights=w, slot_positions=slots)
    lengths = lengths + N
    last = torch.full((B,), N, dtype=torch.int32, device="cuda")
    for step in range(3):
        T = (1, 6, 40)[step]
        parents = _parents(g, B, T)
        tree = sa.tree_words(parents)
        depth = torch.zeros(B, T, dtype=torch.int32)
        for b in range(B):
            for t in range(T):
                depth[b, t] = depth[b, parents[b][t]] + 1 if parents[b][t] >= 0 else 0
        positions = last.view(B, 1) + depth.cuda()
        k, v, q = _randn(g, B, H, T, d), _randn(g, B, H, T, d), _randn(g, B, H * G, T, d)
        qt = sa.cache_append(k, v, ck, cv, lengths, turns, positions, q=q, weights=w, slot_positions=slots)
        ref.check("q", qt, *ref.turned(q.cpu(), positions.cpu(), f))
        want = ref.attention(qt, ck, cv, lengths.tolist(), tree, w)
        o, lse, w = sa.cache_attention(qt, ck, cv, lengths, tree, weights=w)
        for name, got, x in zip(("o", "lse", "weights"), (o, lse, w), want):
            ref.check(name, got, *x)
        path = torch.full((B, 3), -1, dtype=torch.int32)
        for b in range(B):                               # from the last token to its root
            at, line = T - 1, []
            while at >= 0:
                line.append(at)
                at = parents[b][at]
            line = line[::-1][:3]
            path[b, :len(line)] = torch.tensor(line, dtype=torch.int32)
        sa.cache_append(k, v, ck, cv, lengths, turns, positions, rows=path.cuda(), weights=w, slot_positions=slots)
        for b in range(B):
            n = int(lengths[b])
            for i, r in enumerate(path[b].tolist()):
                if r >= 0:
                    assert torch.equal(cv[b, :, n + i], v[b, :, r])
                    assert bool((slots[b, :, n + i] == positions[b, r]).all())
        taken = (path >= 0).sum(1).to(torch.int32).cuda()
        lengths, last = lengths + taken, last + taken
        w, slots, lengths = _check_evict(ck, cv, w, slots, lengths.tolist(), 120, 16, in_place=bool(step % 2))
        assert lengths.tolist() == [120, 120]


def test_captured_and_replayed_steps_on_another_stream():
    g = _gen("graph")
    B, H, G, d, C = 3, 2, 4, 128, 500
    turns = sa.rotary_turns(128)
    ck, cv = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    k, v, q = _randn(g, B, H, 1, d), _randn(g, B, H, 1, d), _randn(g, B, H * G, 1, d)
    w = torch.rand(B, H, C, generator=g, device="cuda")
    pos = torch.arange(C, dtype=torch.int32, device="cuda").repeat(B, H, 1)
    lengths = _i32(300, 10, 499)
    start = [t.clone() for t in (ck, cv, w, pos, lengths)]

    def step():
        qt = sa.cache_append(k, v, ck, cv, lengths, turns, q=q, weights=w, slot_positions=pos)
        o, lse, _ = sa.cache_attention(qt, ck, cv, lengths, weights=w, weights_out=w)
        sa.cache_evict(ck, cv, w, pos, lengths + 1, 256, 32, w, pos)
        lengths.copy_((lengths + 1).clamp_max(256))
        return o, lse

    def reset():
        for t, x in zip((ck, cv, w, pos, lengths), start):
            t.copy_(x)

    eager = []
    for _ in range(3):
        o, lse = step()
        eager.append((o.clone(), lse.clone()))
    after = [t.clone() for t in (ck, cv, w, pos, lengths)]
    reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o, lse = step()
    reset()
    for i in range(3):
        graph.replay()
        assert torch.equal(o, eager[i][0]) and torch.equal(lse, eager[i][1])
    for t, x in zip((ck, cv, w, pos, lengths), after):
        assert torch.equal(t, x)


def test_calls_at_once_on_one_cache_and_by_host_threads():
    """Captured calls of several sizes replayed over one another's streams, and eager ones from several threads."""
    import threading
    g = _gen("threads")
    B, H, d, C = 2, 2, 128, ROOM
    k, v = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    n = _i32(3000, 777)
    qs = [_randn(g, B, H * G, T, d) for G, T in ((1, 1), (4, 4), (2, 30), (4, 64))]
    want = [sa.cache_attention(q, k, v, n) for q in qs]
    graphs = []
    for q in qs:
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            out = [sa.cache_attention(q, k, v, n) for _ in range(3)]
        graphs.append((graph, s, out))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s, _out in graphs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, _, out), w in zip(graphs, want):
        for o, lse in out:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(10):
            o, lse = sa.cache_attention(qs[i], k, v, n, stream=s)
            s.synchronize()
            if not (torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(qs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and sa.attn_get_device_status() == 0


def test_between_other_kernels_that_use_tensor_memory():
    """A step of a block: the projections before and after share the SMs' tensor memory with the attention."""
    g = _gen("block")
    B, H, G, T, d, C = 4, 2, 4, 16, 64, ROOM
    D = H * G * d
    x, wq, wo = _randn(g, B, T, D), _randn(g, D, D, std=D ** -0.5), _randn(g, D, D, std=D ** -0.5)
    wk = _randn(g, D, H * d, std=D ** -0.5)
    k, v = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    n = _i32(1000, 5000, 0, 313)
    turns = sa.rotary_turns(64)

    def step():
        h, _, _ = sa.rms_norm_forward(x, torch.ones(D, device="cuda"))
        q = sa.linear_forward(h, wq).view(B, T, H * G, d).transpose(1, 2).contiguous()
        nk = sa.linear_forward(h, wk).view(B, T, H, d).transpose(1, 2).contiguous()
        qt = sa.cache_append(nk, nk, k, v, n, turns, q=q)
        o, lse = sa.cache_attention(qt, k, v, n)
        return sa.out_proj_forward(o, wo, None, x), o, lse, qt

    first = [t.clone() for t in step()]
    for _ in range(30):
        again = step()
    assert all(torch.equal(a, b) for a, b in zip(first, again)) and sa.attn_get_device_status() == 0
    want_o, want_l = ref.attention_many(first[3], k, v, n.tolist())
    ref.check("o", first[1], *want_o)
    ref.check("lse", first[2], *want_l)


def test_streams_at_once():
    """Two streams with calls in flight at once, each with its own workspace."""
    g = _gen("streams")
    B, H, G, T, d, C = 2, 2, 2, 8, 64, 3000
    q = [_randn(g, B, H * G, T, d) for _ in range(2)]
    k, v = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    n = _i32(2990, 1234)
    want = [sa.cache_attention(x, k, v, n) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[] for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            got[i].append(sa.cache_attention(q[i], k, v, n, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_what_is_written_in_place_is_seen_by_recorded_graphs():
    """A graph that saved a cache, its weights or its positions refuses a backward over what was written since."""
    g = _gen("written")
    B, H, C, d = 2, 2, 40, 64
    ck, cv, k, v = (_randn(g, B, H, n, d) for n in (C, C, 1, 1))
    w = torch.rand(B, H, C, generator=g, device="cuda")
    pos = torch.arange(C, dtype=torch.int32, device="cuda").repeat(B, H, 1)
    lengths = _i32(20, 30)
    calls = [(lambda: sa.cache_append(k, v, ck, cv, lengths, weights=w, slot_positions=pos), (ck, cv, w, pos)),
             (lambda: sa.cache_attention(k, ck, cv, lengths, weights=w, weights_out=w), (w,)),
             (lambda: sa.cache_evict(ck, cv, w, pos, lengths, 16, 4, w, pos), (ck, cv, w, pos))]
    for call, out in calls:
        others = [t for t in (ck, cv, w, pos, k, v, lengths) if not any(t is x for x in out)]
        before = [t._version for t in out], [t._version for t in others]
        leaf = torch.ones((), device="cuda", requires_grad=True)
        y = sum((leaf * t).float().sum() for t in out if t.is_floating_point())
        call()
        assert all(t._version > n for t, n in zip(out, before[0]))
        assert [t._version for t in others] == before[1]
        with pytest.raises(RuntimeError, match="inplace operation"):
            y.backward()
    with torch.inference_mode():                       # (such tensors have no version)
        ci, cj = ck.clone(), cv.clone()
        sa.cache_append(k, v, ci, cj, lengths)
