"""Rotary positions and the cache without a GPU: every bad argument is refused with the documented status before the
device is touched; mask words and frequencies are made on the host."""
import ctypes

import pytest
import torch

import self_attention_gb300 as sa
import _cache_plans
import _cache_ref as ref
from self_attention_gb300.build import build


@pytest.fixture(scope="module")
def lib():
    return sa.load_library(build())


# Fake, never-dereferenced device addresses, 256 MB apart.
A = [0x10000000 * (i + 1) for i in range(14)]
f = ctypes.c_float


def test_rotary_argument_errors(lib):
    for call in (lib.attn_rotary, lib.attn_rotary_bwd):
        def fwd(x=A[0], y=A[1], p=A[2], stride=0, t=A[3], B=2, H=3, N=4, d=64, r=32, i=0, a=1.0):
            return call(x, y, p, stride, t, B, H, N, d, r, i, f(a), None)
        assert fwd(d=96) == 2 and fwd(d=0) == 2
        for r in (0, -16, 8, 24, 80):
            assert fwd(r=r) == 1
        assert fwd(B=-1) == 1 and fwd(H=-1) == 1 and fwd(N=-1) == 1 and fwd(H=16385) == 1
        assert fwd(B=1 << 16, N=1 << 16) == 1 and fwd(B=1 << 10, H=1 << 14, N=1 << 12) == 1
        assert fwd(i=2) == 1 and fwd(a=float("inf")) == 1 and fwd(stride=3) == 1
        assert fwd(x=0) == 1 and fwd(y=0) == 1 and fwd(t=0) == 1
        assert fwd(x=A[0] + 8) == 3 and fwd(y=A[1] + 2) == 3 and fwd(t=A[3] + 8) == 3 and fwd(p=A[2] + 2) == 3
        assert fwd(y=A[0] + 16) == 1 and fwd(y=A[3]) == 1 and fwd(y=A[2], stride=4) == 1
        assert fwd(N=0, x=0, y=0, t=0) == 0 and fwd(B=0) == 0 and fwd(H=0) == 0


def test_append_argument_errors(lib):
    def app(k=A[0], v=A[1], ck=A[2], cv=A[3], n=A[4], t=A[5], p=A[6], rows=0, q=A[7], qo=A[8], w=A[9], s=A[10], B=2,
            H=2, Hq=4, T=5, m=5, d=64, C=32, r=64, i=0, a=1.0):
        return lib.attn_cache_append(k, v, ck, cv, n, t, p, rows, q, qo, w, s, B, H, Hq, T, m, d, C, r, i, f(a), None)
    assert app(d=80) == 2
    for bad in (dict(B=-1), dict(H=0), dict(Hq=0), dict(T=-1, m=-1), dict(C=0), dict(C=1 << 30), dict(m=4), dict(r=8),
                dict(r=80), dict(i=3), dict(a=float("nan")), dict(k=0), dict(v=0), dict(ck=0), dict(cv=0), dict(n=0),
                dict(qo=0), dict(q=0), dict(rows=A[11]), dict(H=20000), dict(rows=A[11], q=0, qo=0, T=0),
                dict(ck=A[0]), dict(cv=A[2] + 64), dict(qo=A[7] + 16), dict(w=A[10]), dict(s=A[4]), dict(ck=A[5])):
        assert app(**bad) == 1, bad
    for bad in (dict(k=A[0] + 8), dict(cv=A[3] + 4), dict(t=A[5] + 8), dict(n=A[4] + 2), dict(s=A[10] + 1)):
        assert app(**bad) == 3, bad
    assert app(T=0, m=0, k=0) == 0 and app(B=0) == 0


def test_attention_argument_errors(lib):
    need = sa.attn_cache_attention_workspace_size(2, 2, 3, 4, 40, 64, True)
    assert need > sa.attn_cache_attention_workspace_size(2, 2, 3, 4, 40, 64) >= 0
    assert sa.attn_cache_attention_workspace_size(1, 2, 1, 1, 1 << 20, 128) > 0      # split over CTAs

    def att(q=A[0], k=A[1], v=A[2], n=A[3], t=A[4], c=A[5], w=A[6], wo=A[7], o=A[8], l=A[9], ws=A[10], nb=need, B=2, H=2,
            G=3, T=4, C=40, d=64, scale=0.125):
        return lib.attn_cache_attention(q, k, v, n, t, c, w, wo, o, l, ws, nb, B, H, G, T, C, d, f(scale), None)
    assert att(d=32) == 2
    sizes = (dict(B=0), dict(H=0), dict(G=0), dict(T=0), dict(T=65, C=100), dict(T=41), dict(C=0), dict(C=1 << 30),
             dict(G=16385), dict(H=200, G=200), dict(B=1 << 20, H=1 << 12))
    for bad in sizes:
        assert att(**bad) == 1, bad
        a = dict(B=2, H=2, G=3, T=4, C=40)
        a.update(bad)
        assert sa.attn_cache_attention_workspace_size(*a.values(), 64) == 0
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(q=0), dict(k=0), dict(v=0), dict(n=0), dict(o=0),
                dict(l=0), dict(w=0), dict(wo=0), dict(o=A[0]), dict(l=A[8] + 64), dict(wo=A[6] + 4),
                dict(wo=A[2]), dict(ws=A[6]), dict(o=A[10]), dict(l=A[4]), dict(l=A[5])):
        assert att(**bad) == 1, bad
    for bad in (dict(ws=0), dict(nb=need - 1), dict(ws=A[10] + 128)):
        assert att(**bad) == 6, bad
    for bad in (dict(q=A[0] + 8), dict(v=A[2] + 2), dict(t=A[4] + 4), dict(n=A[3] + 1), dict(wo=A[7] + 2)):
        assert att(**bad) == 3, bad


def test_evict_argument_errors(lib):
    need = sa.attn_cache_evict_workspace_size(2, 3, 7000, 64, 16)
    assert need > 0 and sa.attn_cache_evict_workspace_size(2, 3, 7000, 64, 0) == 0
    assert sa.attn_cache_evict_workspace_size(2, 3, 7000, 96, 16) == 0
    assert sa.attn_cache_evict_workspace_size(2, 3, 40, 64, 16) == 0             # by single blocks, in shared memory

    def ev(k=A[0], v=A[1], w=A[2], p=A[3], n=A[4], wo=A[5], po=A[6], no=A[7], ws=A[8], nb=need, B=2, H=3, C=7000, d=64,
           keep=16, recent=4):
        return lib.attn_cache_evict(k, v, w, p, n, wo, po, no, ws, nb, B, H, C, d, keep, recent, None)
    assert ev(d=72) == 2
    for bad in (dict(B=0), dict(H=0), dict(C=0), dict(keep=0), dict(recent=-1), dict(recent=17), dict(k=0), dict(v=0),
                dict(w=0), dict(p=0), dict(n=0), dict(wo=0), dict(po=0), dict(no=0), dict(v=A[0]), dict(wo=A[2] + 4),
                dict(po=A[2]), dict(no=A[4]), dict(ws=A[3]), dict(wo=A[3]), dict(k=A[2])):
        assert ev(**bad) == 1, bad
    assert ev(nb=need - 1) == 6 and ev(ws=0) == 6 and ev(ws=A[8] + 64) == 6
    assert ev(k=A[0] + 8) == 3 and ev(no=A[7] + 2) == 3


def test_sizes_of_the_largest_workspaces():
    """No size the calls take needs a workspace that overflows."""
    for T, G in ((64, 128), (1, 16384), (64, 1)):
        assert 0 < sa.attn_cache_attention_workspace_size(1, 1, G, T, 1 << 20, 128) < 1 << 32
    assert sa.attn_cache_evict_workspace_size(4, 16, 1 << 20, 128, 1 << 19) >= 4 * 16 * (1 << 19) * 8


def test_plans_of_attention_are_all_reached(lib):
    """The GPU tests' sizes reach every kernel that the plan chooses from."""
    want = {(k, r, d) for d in (64, 128) for k, rows in ((1, (8, 16)), (2, (8, 16)), (3, (128, 256)), (4, (128, 256))) for r in rows}
    assert _cache_plans.reached() >= want, want - _cache_plans.reached()


def test_clusters_of_every_size_are_reached(lib):
    want = {(n, d) for n in range(1, 9) for d in (64, 128)}
    assert _cache_plans.clusters() >= want, want - _cache_plans.clusters()
    with pytest.raises(sa.AttnError):
        sa.attn_debug_cache_plan(1, 1, 1, 65, 100, 64)
    assert lib.attn_debug_cache_plan(1, 1, 1, 1, 100, 64, None) == 1


def test_tree_words():
    words = sa.tree_words([[-1, 0, 0, 1, 2], [-1, -1, 1, 2, 0]], device="cpu")
    assert words.tolist() == [[1, 3, 5, 11, 21], [1, 2, 6, 14, 17]]
    chain = sa.tree_words([list(range(-1, 63))], device="cpu")
    assert [w % 2 ** 64 for w in chain[0].tolist()] == [(2 << t) - 1 for t in range(64)]
    assert torch.equal(sa.tree_words(torch.tensor([[-1, 0]]), device="cpu"), torch.tensor([[1, 3]]))
    for bad in ([[0]], [[-1, 1]], [[]], [[-1], [-1, 0]]):
        with pytest.raises(ValueError):
            sa.tree_words(bad, device="cpu")


def test_turns_stand_for_the_frequencies():
    import math
    for rotated in (16, 64, 128):
        t = sa.rotary_turns(rotated, device="cpu")
        for got, want in zip(t.tolist(), ref.frequencies(rotated).tolist()):
            assert abs(got / 2 ** 64 * 2 * math.pi - want) < 1e-15 * want + 2.0 ** -63


def test_reference_attention_agrees_with_its_definition():
    """The tests' own 64-bit attention against a softmax over everything with masked scores of minus infinity."""
    g = torch.Generator().manual_seed(1)
    B, H, G, T, d, C = 2, 2, 2, 5, 8, 30
    q, k, v = (torch.randn(s, generator=g) for s in ((B, H * G, T, d), (B, H, C, d), (B, H, C, d)))
    tree = sa.tree_words([[-1, 0, 0, 1, 3], [-1, -1, 0, 2, 1]], device="cpu")
    n = [7, 0]
    (o, _), (lse, _), (w, _) = ref.attention(q, k, v, n, tree, torch.zeros(B, H, C))
    for b in range(B):
        s = torch.einsum("htd,hjd->htj", q[b].double(), k[b].double().repeat_interleave(G, 0)) / d ** 0.5
        j = torch.arange(C)
        sees = (j < n[b]) | ((j >= n[b]) & (j < n[b] + T) & (tree[b].view(T, 1) >> (j - n[b]).clamp(0, 63) & 1).bool())
        s = s.masked_fill(~sees, -torch.inf)
        p = s.softmax(-1)
        assert torch.allclose(o[b], p @ v[b].double().repeat_interleave(G, 0), atol=1e-12)
        assert torch.allclose(lse[b], s.logsumexp(-1), atol=1e-12)
        assert torch.allclose(w[b], p.view(H, G, T, C).sum((1, 2)), atol=1e-12)
