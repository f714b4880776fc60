"""The cache's calls over runs of blocks and past 2^31 elements, element by element: accumulated weights wherever the
attention runs over many blocks, and every call on the last head of a cache past 2^31 elements (and of kept scores past them).

Bounds as in _cache_ref, but for the number of additions a sum takes one after another: a chain there is no longer than what
a CTA adds up of one unit, and the parts that are joined."""
import math
import zlib

import pytest
import torch

import self_attention_gb300 as sa
import _cache_ref as ref
from _block_ref import STEP, U8
from _cache_plans import BLOCKS

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


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _many(q, k, v, lengths, tree, w, counted, chain):
    """(o, tolerance), (lse, tolerance), (weights, tolerance) in 64 bits; chain(slots): the longest run of additions."""
    B, Hq, T, d = q.shape
    H = k.shape[1]
    G = Hq // H
    f64 = dict(dtype=torch.float64, device=q.device)
    o, lse = torch.zeros(B, Hq, T, d, **f64), torch.zeros(B, Hq, T, **f64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    out, tw = w.double(), STEP * w.double().abs()
    u = torch.arange(T, device=q.device)
    for b in range(B):
        n = int(lengths[b])
        own = u.view(1, T) <= u.view(T, 1) if tree is None else (tree[b].view(T, 1) >> u & 1).bool()
        hide = torch.cat((torch.zeros(T, n, dtype=torch.bool, device=q.device), ~own), 1)
        adds = (chain(n + T) + 8) * STEP
        add = torch.ones(T, **f64) if counted is None else (counted[b] >> u & 1).double()
        for h in range(H):
            at = slice(h * G, (h + 1) * G)
            rows, kk, vv = q[b, at].double(), k[b, h, :n + T].double(), v[b, h, :n + T].double()
            s = (rows @ kk.T / math.sqrt(d)).masked_fill_(hide, -math.inf)
            a = (rows.abs() @ kk.abs().T).masked_fill_(hide, 0.0).amax(-1)
            ds = (d + 8) * STEP / math.sqrt(d) * a + 4 * STEP * s.masked_fill(hide, 0.0).abs().amax(-1) + 2.0 ** -21
            x = torch.logsumexp(s, -1)
            p = s.sub_(x.unsqueeze(-1)).exp_()
            e = (2 * ds + U8 + adds).unsqueeze(-1) * (p @ vv.abs())
            o[b, at], lse[b, at] = p @ vv, x
            to[b, at] = e + U8 * (o[b, at].abs() + e)
            tl[b, at] = ds + adds + 4 * STEP * x.abs()
            p = p * add.view(1, T, 1)
            out[b, h, :n + T] += p.sum((0, 1))
            tw[b, h, :n + T] += (p * (2 * ds + adds + (G * T + 8) * STEP).unsqueeze(-1)).sum((0, 1)) + STEP * out[b, h, :n + T].abs()
    return (o, to), (lse, tl), (out, tw)


@pytest.mark.parametrize("B,H,G,T,d,C,ragged", BLOCKS)
@pytest.mark.parametrize("some", [False, True])
def test_weights_over_many_blocks(B, H, G, T, d, C, ragged, some):
    """Kept scores and K a second time where the shares run over several heads and sequences."""
    g = _gen("weights", B, H, G, T, d, C, some)
    lens = [C - T - (b * 977) % (ragged + 1) for b in range(B)]
    q = _randn(g, B, H * G, T, d, std=2.0)
    k, v = _randn(g, B, H, C, d), _randn(g, B, H, C, d)
    for b, n in enumerate(lens):
        k[b, :, n + T:], v[b, :, n + T:] = math.nan, math.nan
    w = torch.rand(B, H, C, generator=g, device="cuda")
    tree = counted = None
    if some:
        parents = [[int(x * (t + 1)) - 1 for t, x in enumerate(row)] for row in torch.rand(B, T, generator=g, device="cuda").tolist()]
        tree = sa.tree_words(parents)
        counted = torch.randint(-(2 ** 63), 2 ** 63 - 1, (B,), generator=g, device="cuda")
    o, lse, out = sa.cache_attention(q, k, v, _i32(*lens), tree, weights=w, counted=counted)
    want = _many(q, k, v, lens, tree, w, counted, lambda slots: slots)
    for name, got, x in zip(("o", "lse", "weights"), (o, lse, out), want):
        ref.check(name, got, *x)
    again = sa.cache_attention(q, k, v, _i32(*lens), tree, weights=w, counted=counted, weights_out=w)
    assert again[2] is w and torch.equal(w, out) and torch.equal(again[0], o) and torch.equal(again[1], lse)
    assert sa.attn_get_device_status() == 0


# d, C, G, T of one sequence with 17 cached heads: 2^31 elements and more
LONG = [(128, 1 << 20, 1, 1), (128, 1 << 20, 2, 64), (64, 1 << 23, 16, 1), (64, 1 << 23, 5, 4)]
HEADS = 17


def _long(g, d, C):
    k, v = (torch.zeros(1, HEADS, C, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    for t in (k, v):
        t[:, -1].normal_(generator=g)
    return k, v


@pytest.mark.parametrize("d,C,G,T", LONG)
def test_attention_past_2_31_elements(d, C, G, T):
    """Every row of the last head, and the weights of its slots; the first heads' are the mean of nothing but zeros."""
    g = _gen("long", d, C, G, T)
    k, v = _long(g, d, C)
    q = _randn(g, 1, HEADS * G, T, d)
    n = C - T - 3
    # a slot for each row of the last head that takes most of its weight, the last slots among them
    last = q[0, -G:].reshape(G * T, d)
    at = torch.cat((torch.arange(n - G * T // 2, n), torch.randint(0, n - G * T, (G * T - G * T // 2,), generator=g, device="cuda").cpu()))
    k[0, -1, at.cuda()] = (last.float() * (1.6 if d == 128 else 2.6)).to(torch.bfloat16)
    w = torch.rand(1, HEADS, C, generator=g, device="cuda")
    o, lse, out = sa.cache_attention(q, k, v, _i32(n), weights=w)
    kind, _, ctas = sa.attn_debug_cache_plan(1, HEADS, G, T, C, d)
    assert kind in (2, 4)
    if G == 16:
        assert kind == 2 and HEADS * G * T * C > 2 ** 31             # kept scores past them too
    # by shares: of few rows a warp adds 16 slots and two terms a step of 128, of more a CTA all its slots
    share = HEADS * C // ctas + 128
    steps = share // 128 * 34 if kind == 2 else share
    want = _many(q[:, -G:], k[:, -1:], v[:, -1:], [n], None, w[:, -1:], None, lambda slots: steps + 2000)
    ref.check("o", o[:, -G:], *want[0])
    ref.check("lse", lse[:, -G:], *want[1])
    ref.check("weights", out[:, -1:], *want[2])
    assert want[0][0].abs().mean() > 0.3                              # (rows that say something)
    assert not bool(o[:, :-G].any())
    gain = (out[:, :-1] - w[:, :-1])[..., :n]                         # zeros: every slot alike, to a step of what it had
    assert (gain - G * T / n).abs().max() < 0.02 * G * T / n + 2.0 ** -22
    assert torch.equal(out[..., n + T:], w[..., n + T:])


@pytest.mark.parametrize("d,C", [(128, 1 << 20), (64, 1 << 23)])
def test_append_and_eviction_past_2_31_elements(d, C):
    g = _gen("long evict", d, C)
    k, v = _long(g, d, C)
    T = 5
    w = torch.rand(1, HEADS, C, generator=g, device="cuda")
    pos = torch.arange(C, dtype=torch.int32, device="cuda").repeat(1, HEADS, 1)
    nk, nv = _randn(g, 1, HEADS, T, d), _randn(g, 1, HEADS, T, d)
    turns, at = sa.rotary_turns(d), _i32(*range(C + 100, C + 100 + T)).view(1, T)
    n = C - T
    before = k[0, -1, :n].clone(), v[0, -1, :n].clone()
    sa.cache_append(nk, nv, k, v, _i32(n), turns, at, weights=w, slot_positions=pos)
    assert torch.equal(k[0, :, n:], sa.rotary_forward(nk, turns, at)[0]) and torch.equal(v[0, :, n:], nv[0])
    assert torch.equal(k[0, -1, :n], before[0]) and torch.equal(v[0, -1, :n], before[1]) and not bool(k[0, :-1, :n].any())
    assert not bool(w[0, :, n:].any()) and torch.equal(pos[0, :, n:], at.expand(HEADS, T))
    for keep, recent in ((C // 3, 1000), (C - 12345, 7)):
        # of each head: ranks, what stays, holes below and movers behind, both in ascending order
        L = C
        j = torch.arange(C, device="cuda")
        fresh = pos[0] > pos[0].amax(-1, keepdim=True) - recent
        rank = torch.where(fresh, math.inf, w[0])
        stays = torch.zeros(HEADS, C, dtype=torch.bool, device="cuda")
        stays.scatter_(1, rank.sort(dim=-1, descending=True, stable=True).indices[:, :keep], True)
        want_w, want_p = w.clone(), pos.clone()
        for h in range(HEADS):
            to, of = (~stays[h] & (j < keep)).nonzero()[:, 0], (stays[h] & (j >= keep)).nonzero()[:, 0]
            for t in (want_w, want_p):
                t[0, h, to] = t[0, h, of]
            if h == HEADS - 1:
                want_k, want_v = k[0, h].clone(), v[0, h].clone()
                for t in (want_k, want_v):
                    t[to] = t[of]
        want_w[..., keep:], want_p[..., keep:] = 0.0, -1
        w2, p2, n2 = sa.cache_evict(k, v, w, pos, _i32(L), keep, recent)
        assert n2.tolist() == [keep] and torch.equal(w2, want_w) and torch.equal(p2, want_p)
        assert torch.equal(k[0, -1], want_k) and torch.equal(v[0, -1], want_v)
