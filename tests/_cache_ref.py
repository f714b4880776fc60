"""Plain 64-bit implementations of rotary positions and of the cache's operators, with the error bounds the GPU
tests hold the kernels to.  Written from the formulas, row by row, on whatever device the tensors are on.

Bounds.  U8 = 2^-8 is half a bf16 step relative to the value, STEP = 2^-23 a whole fp32 one; a sum of n products
in fp32 in any order is off by at most (n + 8) STEP times the sum of the products' magnitudes.
  turned columns   the angle is off by 2^-25 pi (its fraction of a turn is kept to 24 bits of half a turn) and the
                   sine and cosine by 2 STEP each; two products and a sum add 3 STEP: 8 STEP of |a| + |b| in all.
  weights p        a score is off by ds = scale (d + 8) STEP sum |q k|; times log2 e, less the maximum, through the
                   exponential: 4 STEP of the largest |score| in the row and 2^-21 more.  Normalised, a weight is off
                   by twice that, relative to itself.  For the product with V it is held to 2^-8 of itself.
"""
import math

import torch

from _block_ref import STEP, U8


def frequencies(rotated, base=10000.0):
    return base ** (-2.0 * torch.arange(rotated // 2, dtype=torch.float64) / rotated)


def turned(x, positions, f, interleaved=False, amplitude=1.0, sign=1.0):
    """(y, tolerance): x [B,H,N,d] at positions [B,N], frequencies f in radians a position."""
    B, H, N, d = x.shape
    x = x.double()
    y, tol = x.clone(), torch.zeros_like(x)
    half = f.numel()
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        t = (positions.double() * f[j].item()).view(-1, 1, N)
        c, s = t.cos() * amplitude, t.sin() * amplitude * sign
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        e = 8 * STEP * abs(amplitude) * (x[..., a].abs() + x[..., b].abs())
        tol[..., a] = tol[..., b] = e
    return y, tol + U8 * (y.abs() + tol) * (tol > 0)


def word(tree, b, t):
    return (2 << t) - 1 if tree is None else int(tree[b, t]) & (2 ** 64 - 1)


def attention(q, k, v, lengths, tree=None, weights=None, counted=None, scale=None):
    """o, lse, weights (or None), each with its tolerance."""
    B, Hq, T, d = q.shape
    H, C = k.shape[1:3]
    G = Hq // H
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, lse = torch.zeros(B, Hq, T, d, dtype=torch.float64), torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    w = None if weights is None else weights.double().cpu().clone()
    tw = None if w is None else STEP * w.abs()
    for b in range(B):
        n = min(max(int(lengths[b]), 0), C - T)
        for h in range(H):
            kk, vv = k[b, h, :n + T].double().cpu(), v[b, h, :n + T].double().cpu()
            for x in range(h * G, (h + 1) * G):
                for t in range(T):
                    seen = list(range(n)) + [n + u for u in range(T) if word(tree, b, t) >> u & 1]
                    if not seen:
                        continue
                    row = q[b, x, t].double().cpu()
                    ks, vs = kk[seen], vv[seen]
                    s = ks @ row * scale
                    ds = scale * (d + 8) * STEP * (ks.abs() @ row.abs()).max() + 4 * STEP * s.abs().max() + 2.0 ** -21
                    lse[b, x, t] = torch.logsumexp(s, 0)
                    p = torch.exp(s - lse[b, x, t])
                    m = len(seen)
                    o[b, x, t] = p @ vs
                    e = (2 * ds + U8 + (m + 8) * STEP) * (p @ vs.abs())
                    to[b, x, t] = e + U8 * (o[b, x, t].abs() + e)
                    tl[b, x, t] = ds + (m + 8) * STEP + 4 * STEP * lse[b, x, t].abs()
                    if w is not None and (counted is None or int(counted[b]) >> t & 1):
                        w[b, h, seen] += p
                        tw[b, h, seen] += p * (2 * ds + (m + 8) * STEP + (G * T + 8) * STEP) + STEP * w[b, h, seen]
    return (o, to), (lse, tl), (w, tw)


def attention_many(q, k, v, lengths, tree=None):
    """(o, tolerance), (lse, tolerance) as attention() has them, for many finite rows at once, on q's device."""
    B, Hq, T, d = q.shape
    H, C = k.shape[1:3]
    G = Hq // H
    o, lse = torch.zeros(B, Hq, T, d, dtype=torch.float64), torch.zeros(B, Hq, T, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    u = torch.arange(T, device=q.device)
    for b in range(B):
        n = int(lengths[b])
        own = u.view(1, T) <= u.view(T, 1) if tree is None else (tree[b].view(T, 1) >> u & 1).bool()
        sees = torch.cat((torch.ones(T, n, dtype=torch.bool, device=q.device), own), 1)
        m = sees.sum(1).cpu()
        for h in range(H):
            rows = q[b, h * G:(h + 1) * G].double()
            kk, vv = k[b, h, :n + T].double(), v[b, h, :n + T].double()
            s = (rows @ kk.T / math.sqrt(d)).masked_fill(~sees, -math.inf)
            a = (rows.abs() @ kk.abs().T).masked_fill(~sees, 0.0).amax(-1)
            ds = (d + 8) * STEP / math.sqrt(d) * a + 4 * STEP * s.masked_fill(~sees, 0.0).abs().amax(-1) + 2.0 ** -21
            x = torch.logsumexp(s, -1)
            p = torch.exp(s - x.unsqueeze(-1))
            e = (2 * ds + U8 + (m + 8).to(q.device) * STEP).unsqueeze(-1) * (p @ vv.abs())
            y = p @ vv
            at = slice(h * G, (h + 1) * G)
            o[b, at], lse[b, at] = y.cpu(), x.cpu()
            to[b, at], tl[b, at] = (e + U8 * (y.abs() + e)).cpu(), (ds + 4 * STEP * x.abs()).cpu() + (m + 8) * STEP
    return (o, to), (lse, tl)


def evict(k, v, weights, positions, lengths, keep, recent):
    """k, v, weights, positions, lengths after the eviction (copies, on the host)."""
    k, v, w, pos = (t.cpu().clone() for t in (k, v, weights, positions))
    B, H, C = w.shape
    left = []
    for b in range(B):
        L = min(max(int(lengths[b]), 0), C)
        n = min(L, keep)
        left.append(n)
        for h in range(H):
            newest = max(pos[b, h, :L].tolist(), default=0)

            wt, at = w[b, h].tolist(), pos[b, h].tolist()

            def rank(j):
                old = at[j] <= newest - recent
                return old, -(wt[j] if wt[j] > 0 else 0.0) if old else 0.0, j
            stay = sorted(range(L), key=rank)[:n]
            gone = set(range(n)) - set(stay)
            to = sorted(gone)
            of = sorted(j for j in stay if j >= n)
            for t in (k, v, w, pos):
                t[b, h, to] = t[b, h, of].clone()
            w[b, h, n:], pos[b, h, n:] = 0.0, -1
    return k, v, w, pos, torch.tensor(left, dtype=torch.int32)


def check(name, got, want, tol):
    """got within tol of want; infinities, and NaN, in the same places."""
    got = got.double().cpu()
    want, tol = want.cpu(), tol.cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fine = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan()), name
    assert torch.equal(got.isinf(), want.isinf()) and bool((got[want.isinf()] == want[want.isinf()]).all()), name
    err = (got - want).abs()[fine]
    over = err > tol[fine]
    assert not bool(over.any()), (name, err[over].max().item(), tol[fine][over].min().item(), int(over.sum()))
