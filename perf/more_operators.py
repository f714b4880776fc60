"""The operators of serving over a cache, and the positions that training needs too, as they are measured.

    rotary           positions turned into angles between the two columns of a pair, forward and backward
    cache_append     new tokens' keys (turned) and values into the cache, their queries turned beside them
    cache_attention  one token, a chain or a tree of drafted tokens over the cache, with the accumulated
                     attention weight of every slot where it is asked for
    cache_evict      the slots with the least accumulated weight leave the cache, in place

`run` computes them with elementary torch operations in 32 bits (angles in 64), rounded once at the end;
with `own` set it calls self_attention_gb300 instead.  Tensors are bf16 [B, H, N, d_k], weights and lse
fp32, lengths and positions int32.
"""
import math

import torch

own = False

BASE = 10000.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # queries of the high-resolution ViT-L batch (8 x 4096 tokens, 16 heads of 64)
        {"name": "rotary vit-l", "op": "rotary", "B": 8, "H": 16, "N": 4096, "d": 64, "rotated": 64,
         "interleaved": False, "method": "none", "factor": 1.0, "far": 0},
        # long text (2 x 16384 tokens, 16 heads of 128), trained on shorter text: half of the head turned,
        # frequencies scaled by parts; the gradient
        {"name": "rotary bwd long text", "op": "rotary_bwd", "B": 2, "H": 16, "N": 16384, "d": 128, "rotated": 64,
         "interleaved": True, "method": "parts", "factor": 4.0, "far": 0},
        # one token far into a text: latency
        {"name": "rotary one token", "op": "rotary", "B": 1, "H": 16, "N": 1, "d": 128, "rotated": 128,
         "interleaved": False, "method": "positions", "factor": 8.0, "far": 1000003},
        # a batch of sequences takes its next tokens into the cache, grouped heads; queries turned beside them
        {"name": "append next tokens", "op": "append", "B": 32, "H": 4, "G": 4, "T": 1, "d": 128, "len": 2000,
         "ragged": 1500, "rotated": 128, "interleaved": False, "path": 0, "q": True},
        # the long-text prompt goes into an empty cache
        {"name": "append prompt", "op": "append", "B": 2, "H": 16, "G": 1, "T": 16384, "d": 128, "len": 0,
         "ragged": 0, "rotated": 128, "interleaved": False, "path": 0, "q": False},
        # one token of one sequence, 16 heads of 128: latency
        {"name": "attention one token", "op": "attention", "B": 1, "H": 16, "G": 1, "T": 1, "d": 128, "len": 1000,
         "ragged": 0, "tree": False, "weights": False, "counted": "all"},
        # the next tokens of a batch of long texts of many lengths, grouped heads: cache streaming
        {"name": "attention long batch", "op": "attention", "B": 32, "H": 4, "G": 4, "T": 1, "d": 128, "len": 16384,
         "ragged": 9001, "tree": False, "weights": False, "counted": "all"},
        # a tree of 64 drafted tokens over long texts, grouped heads: 256 query rows a cached head
        {"name": "attention tree of 64", "op": "attention", "B": 4, "H": 4, "G": 4, "T": 64, "d": 128, "len": 16384,
         "ragged": 3001, "tree": True, "weights": False, "counted": "all"},
        # a small tree over short ragged sequences, 12 heads of 64
        {"name": "attention small tree", "op": "attention", "B": 7, "H": 12, "G": 1, "T": 13, "d": 64, "len": 1111,
         "ragged": 1000, "tree": True, "weights": False, "counted": "all"},
        # next tokens with the accumulated weights that eviction goes by
        {"name": "attention with weights", "op": "attention", "B": 16, "H": 8, "G": 4, "T": 1, "d": 128, "len": 8192,
         "ragged": 801, "tree": False, "weights": True, "counted": "all"},
        # a long prompt's cache shrunk to an eighth
        {"name": "evict prompt", "op": "evict", "B": 2, "H": 16, "d": 128, "len": 16384, "ragged": 0, "keep": 2048,
         "recent": 256, "moved": False},
        # one slot too many after each step of a batch
        {"name": "evict step", "op": "evict", "B": 32, "H": 4, "d": 128, "len": 2049, "ragged": 300, "keep": 2048,
         "recent": 128, "moved": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "rotary_bwd", "append", "attention", "attention", "attention", "evict"))
    flag = lambda: rng.random() < 0.5  # noqa: E731
    d = rng.choice((64, 128))
    if op.startswith("rotary"):
        B, H = _log_int(rng, 1, 16), rng.randint(1, 24)
        N = _log_int(rng, 1, max(1, min(32768, 500000 // (B * H))))
        return {"op": op, "B": B, "H": H, "N": N, "d": d, "rotated": 16 * rng.randint(1, d // 16), "interleaved": flag(),
                "method": rng.choice(("none", "positions", "base", "parts")), "factor": rng.choice((2.0, 4.0, 8.0)),
                "far": _log_int(rng, 1, 10 ** 6)}
    if op == "append":
        B, H = _log_int(rng, 1, 32), rng.randint(1, 16)
        T = _log_int(rng, 1, max(1, min(8192, 300000 // (B * H))))
        length = _log_int(rng, 1, 4096)
        path = rng.randint(1, T) if T <= 64 and flag() else 0
        return {"op": op, "B": B, "H": H, "G": rng.choice((1, 2, 4)), "T": T, "d": d, "len": length,
                "ragged": rng.randint(0, length), "rotated": 16 * rng.randint(1, d // 16), "interleaved": flag(),
                "path": path, "q": not path and flag()}
    B, H = _log_int(rng, 1, 32), rng.randint(1, 16)
    if op == "evict":
        length = _log_int(rng, 2, max(2, min(32768, 500000 // (B * H))))
        keep = rng.randint(1, length)
        return {"op": op, "B": B, "H": H, "d": d, "len": length, "ragged": rng.randint(0, length), "keep": keep,
                "recent": rng.randint(0, keep), "moved": flag()}
    T = 1 if flag() else _log_int(rng, 1, 64)
    G = rng.randint(1, 8)
    # slots by the bytes of the cache and by the products, within the largest listed ones
    most = min(1500000 * 128 // (B * H * d), 64 * 10 ** 9 // (4 * B * H * G * T * d), 65536)
    length = _log_int(rng, 1, max(1, most))
    weights = flag() and (T == 1 or flag())
    return {"op": op, "B": B, "H": H, "G": G, "T": T, "d": d, "len": length, "ragged": rng.randint(0, length),
            "tree": T > 1 and flag(), "weights": weights, "counted": rng.choice(("all", "first"))}


def _lens(c):
    """Slots in use ahead of the call, sequence by sequence: the first has the most."""
    return [c["len"] - (b * 7919) % (c["ragged"] + 1) if c["ragged"] else c["len"] for b in range(c["B"])]


def _capacity(c):
    return (c["len"] + c.get("T", 0) + 63) // 64 * 64 + 64


# ------------------------------------------------------------------ inputs
def _frequencies(rotated, method, factor, trained=4096, low=1.0, high=32.0):
    """Radians a position, of each pair of columns."""
    i = torch.arange(rotated // 2, dtype=torch.float64)
    base = BASE * factor ** (rotated / (rotated - 2)) if method == "base" else BASE
    f = base ** (-2.0 * i / rotated)
    if method == "positions":
        f = f / factor
    elif method == "parts":
        whole = trained * f / (2.0 * math.pi)              # turns over the trained length
        g = ((whole - low) / (high - low)).clamp(0.0, 1.0)
        f = f * ((1.0 - g) / factor + g)
    return f


def _turns(c):
    import self_attention_gb300 as sa
    return sa.rotary_turns(c["rotated"], base=BASE, method=c.get("method", "none"), factor=c.get("factor", 1.0),
                           trained=4096, device="cuda")


def _tree(rng, B, T):
    """Parents drawn at random: the mask word of each token (bit u: it sees token u) and its depth."""
    words, depth = torch.zeros(B, T, dtype=torch.int64), torch.zeros(B, T, dtype=torch.int32)
    parents = (torch.rand(B, T, generator=rng) * torch.arange(T)).long()
    for b in range(B):
        w, dep = [0] * T, [0] * T
        for t in range(T):
            p = int(parents[b, t])
            w[t] = (w[p] if t else 0) | (1 << t)
            dep[t] = dep[p] + 1 if t else 0
        words[b] = torch.tensor([x - (1 << 64) if x >> 63 else x for x in w], dtype=torch.int64)
        depth[b] = torch.tensor(dep, dtype=torch.int32)
    return words, depth


def prepare(case, seed):
    c = dict(case)
    op = c["op"]
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))

    def randn(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(torch.bfloat16)

    s = {"case": c}
    B, H, d = c["B"], c["H"], c["d"]
    if op.startswith("rotary"):
        N = c["N"]
        s["x"] = randn(B, H, N, d)
        start = torch.randint(0, c["far"] + 1, (B, 1), generator=host) if c["far"] else torch.zeros(B, 1)
        s["positions"] = (start + torch.arange(N)).to(torch.int32).cuda()
        s["f"] = _frequencies(c["rotated"], c["method"], c["factor"]).cuda()
        s["turns"] = _turns(c) if own else None
        return s
    lens = _lens(c)
    s["lens"] = lens
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    C = _capacity(c)
    s["k"], s["v"] = randn(B, H, C, d), randn(B, H, C, d)
    if op == "append":
        T, G = c["T"], c["G"]
        s["nk"], s["nv"] = randn(B, H, T, d), randn(B, H, T, d)
        s["q"] = randn(B, H * G, T, d) if c["q"] else None
        s["positions"] = (torch.tensor(lens).view(B, 1) + torch.arange(T)).to(torch.int32).cuda()
        s["rows"] = None
        if c["path"]:   # an accepted path through the drafted tokens
            s["rows"] = torch.stack([torch.randperm(T, generator=host)[:c["path"]].sort().values for _ in range(B)]
                                    ).to(torch.int32).cuda()
        s["f"] = _frequencies(c["rotated"], "none", 1.0).cuda()
        s["turns"] = _turns(c) if own else None
        s["weights"] = torch.rand(B, H, C, generator=g, device="cuda")
        s["slots"] = torch.arange(C, dtype=torch.int32, device="cuda").repeat(B, H, 1)
    elif op == "attention":
        T, G = c["T"], c["G"]
        s["q"] = randn(B, H * G, T, d, std=2.0)
        s["tree"] = _tree(host, B, T)[0].cuda() if c["tree"] else None
        s["weights"] = torch.rand(B, H, C, generator=g, device="cuda") if c["weights"] else None
        s["counted"] = torch.ones(B, dtype=torch.int64, device="cuda") if c["counted"] == "first" else None
    else:
        s["weights"] = torch.rand(B, H, C, generator=g, device="cuda") ** 8 * 50.0
        s["slots"] = torch.arange(C, dtype=torch.int32, device="cuda").repeat(B, H, 1)
        if c["moved"]:   # earlier evictions left the slots out of order
            s["slots"] = torch.rand(B, H, C, generator=g, device="cuda").argsort(-1).to(torch.int32)
    return s


# ------------------------------------------------------------------ the plain forms
def _turned(x, positions, f, interleaved, sign):
    """x [B, H, N, d] fp32 with the pairs of its first 2 len(f) columns turned; positions [B, N]."""
    r = 2 * f.numel()
    angle = positions.double().unsqueeze(-1) * f
    cos, sin = angle.cos().float().unsqueeze(1), (sign * angle.sin()).float().unsqueeze(1)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_append(s):
    c = s["case"]
    T, pos = c["T"], s["positions"]
    k = _turned(s["nk"].float(), pos, s["f"], c["interleaved"], 1.0).to(torch.bfloat16)
    for b, n in enumerate(s["lens"]):
        rows = torch.arange(T, device="cuda") if s["rows"] is None else s["rows"][b].long()
        m = rows.numel()
        s["k"][b, :, n:n + m] = k[b, :, rows]
        s["v"][b, :, n:n + m] = s["nv"][b, :, rows]
        s["weights"][b, :, n:n + m] = 0.0
        s["slots"][b, :, n:n + m] = pos[b, rows]
    out = (s["k"], s["v"], s["weights"], s["slots"])
    if s["q"] is not None:
        out += (_turned(s["q"].float(), pos, s["f"], c["interleaved"], 1.0).to(torch.bfloat16),)
    return out


def _visible(words, T):
    """[B, T, T] truth values from the mask words, a chain without them."""
    u = torch.arange(T, device="cuda")
    if words is None:
        return (u.view(1, T) <= u.view(T, 1)).unsqueeze(0)
    return (words.unsqueeze(-1) >> u & 1).bool()


def _plain_attention(s):
    c = s["case"]
    B, H, G, T, d = (c[x] for x in ("B", "H", "G", "T", "d"))
    sees = _visible(s["tree"], T).expand(B, T, T)
    o = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:3], device="cuda")
    weights = None if s["weights"] is None else s["weights"].clone()
    for b, n in enumerate(s["lens"]):
        q = s["q"][b].float().view(H, G * T, d)
        k, v = s["k"][b, :, :n + T].float(), s["v"][b, :, :n + T].float()
        z = (q @ k.transpose(1, 2)).mul_(d ** -0.5).view(H, G, T, n + T)
        z[..., n:] = z[..., n:].masked_fill(~sees[b], -math.inf)
        m = z.amax(-1, keepdim=True)
        p = torch.exp(z - m)
        total = p.sum(-1, keepdim=True)
        p = p / total
        o[b] = (p.view(H, G * T, n + T) @ v).view(H * G, T, d).to(torch.bfloat16)
        lse[b] = (m + torch.log(total)).view(H * G, T)
        if weights is not None:
            w = p if s["counted"] is None else p[:, :, :1]
            weights[b, :, :n + T] += w.sum((1, 2))
    return (o, lse) if weights is None else (o, lse, weights)


def _plain_evict(s):
    c = s["case"]
    B, H, keep = c["B"], c["H"], c["keep"]
    w, slots = s["weights"], s["slots"]
    C = w.shape[-1]
    j = torch.arange(C, device="cuda")
    length = s["lengths"].view(B, 1, 1)
    n = length.clamp_max(keep)
    used = j < length
    newest = torch.where(used, slots, torch.full_like(slots, -2 ** 31)).amax(-1, keepdim=True)
    rank = torch.where(slots > newest - c["recent"], math.inf, w)
    order = torch.where(used, rank, torch.full_like(rank, -1.0)).sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(used.expand(B, H, C)).scatter_(-1, order, (j < n).expand(B, H, C))
    dst, src = (~kept & (j < n)).nonzero(as_tuple=True), (kept & (j >= n)).nonzero(as_tuple=True)
    w, slots = w.clone(), slots.clone()
    for t in (s["k"], s["v"], w, slots):
        t[dst] = t[src]
    w = torch.where(j < n, w, torch.zeros_like(w))
    slots = torch.where(j < n, slots, torch.full_like(slots, -1))
    return s["k"], s["v"], w, slots, n.view(B).to(torch.int32)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op.startswith("rotary"):
        sign = -1.0 if op == "rotary_bwd" else 1.0
        return (_turned(s["x"].float(), s["positions"], s["f"], c["interleaved"], sign).to(torch.bfloat16),)
    return {"append": _plain_append, "attention": _plain_attention, "evict": _plain_evict}[op](s)


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    import self_attention_gb300 as sa
    c = s["case"]
    op = c["op"]
    if op == "rotary":
        return (sa.rotary_forward(s["x"], s["turns"], s["positions"], c["interleaved"]),)
    if op == "rotary_bwd":
        return (sa.rotary_backward(s["x"], s["turns"], s["positions"], c["interleaved"]),)
    if op == "append":
        q = sa.cache_append(s["nk"], s["nv"], s["k"], s["v"], s["lengths"], s["turns"], s["positions"],
                            c["interleaved"], rows=s["rows"], q=s["q"], weights=s["weights"], slot_positions=s["slots"])
        out = (s["k"], s["v"], s["weights"], s["slots"])
        return out if q is None else out + (q,)
    if op == "attention":
        return sa.cache_attention(s["q"], s["k"], s["v"], s["lengths"], s["tree"], weights=s["weights"],
                                  counted=s["counted"])
    w, slots, lengths = sa.cache_evict(s["k"], s["v"], s["weights"], s["slots"], s["lengths"], c["keep"], c["recent"])
    return s["k"], s["v"], w, slots, lengths


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ work
def work(case):
    c = dict(case)
    op, B, H, d = c["op"], c["B"], c["H"], c["d"]
    if op.startswith("rotary"):
        return {"bytes": B * c["N"] * (4 * H * d + 4), "flops": 3 * B * H * c["N"] * c["rotated"]}
    lens = _lens(c)
    if op == "append":
        n = c["path"] or c["T"]
        heads = H * (2 + (c["G"] if c["q"] else 0))
        turned = H * (1 + (c["G"] if c["q"] else 0))
        return {"bytes": B * n * (4 * heads * d + 8 * H + 4), "flops": 3 * B * turned * n * c["rotated"]}
    C = _capacity(c)
    if op == "attention":
        T, rows = c["T"], B * H * c["G"] * c["T"]
        slots = sum(n + T for n in lens) * H
        return {"bytes": 4 * d * slots + rows * (4 * d + 4) + (8 * B * H * C if c["weights"] else 0),
                "flops": 4 * slots * c["G"] * T * d}
    b = 0.0
    for n in lens:
        kept = min(n, c["keep"])
        recent = min(kept, c["recent"])
        # kept slots that lie behind the first `kept`: all of the recent ones where the slots are in order
        # (as they stand in most prompts), the others by their share
        behind = (kept - recent) * (n - kept) / max(1, n)
        behind += recent * (n - kept) / max(1, n) if c["moved"] else min(recent, n - kept)
        b += H * (8 * n + 8 * C + 8 * d * behind)
    return {"bytes": b, "flops": 2 * H * sum(lens)}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_turned(x, positions, f, interleaved, sign):
    """As complex numbers: each pair times exp(i angle)."""
    x = x.double()
    h = f.numel()
    pair = x[..., :2 * h].unflatten(-1, (h, 2) if interleaved else (2, h))
    pair = pair if interleaved else pair.transpose(-1, -2)
    angle = torch.einsum("bn,j->bnj", positions.double(), f)[:, None]
    z = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(angle), sign * angle)
    y = torch.view_as_real(z)
    y = (y if interleaved else y.transpose(-1, -2)).flatten(-2)
    return torch.cat((y, x[..., 2 * h:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op.startswith("rotary"):
        return [_exact_turned(s["x"], s["positions"], s["f"], c["interleaved"], -1.0 if op == "rotary_bwd" else 1.0)]
    if op == "append":
        turned = _exact_turned(s["nk"], s["positions"], s["f"], c["interleaved"], 1.0)
        k, v, w, slots = s["k"].double(), s["v"].double(), s["weights"].double(), s["slots"].clone()
        for b in range(c["B"]):
            rows = list(range(c["T"])) if s["rows"] is None else s["rows"][b].tolist()
            at = slice(s["lens"][b], s["lens"][b] + len(rows))
            k[b, :, at], v[b, :, at] = turned[b][:, rows], s["nv"][b][:, rows].double()
            w[b, :, at], slots[b, :, at] = 0.0, s["positions"][b][rows]
        out = [k, v, w, slots]
        if s["q"] is not None:
            out.append(_exact_turned(s["q"], s["positions"], s["f"], c["interleaved"], 1.0))
        return out
    if op == "attention":
        B, H, G, T, d = (c[x] for x in ("B", "H", "G", "T", "d"))
        o = torch.zeros(B, H * G, T, d, dtype=torch.float64, device="cuda")
        lse = torch.zeros(B, H * G, T, dtype=torch.float64, device="cuda")
        w = None if s["weights"] is None else s["weights"].double()
        words = None if s["tree"] is None else s["tree"].tolist()
        for b in range(B):
            n = s["lens"][b]
            hide = torch.zeros(T, n + T, dtype=torch.bool, device="cuda")
            for t in range(T):
                word = (2 << t) - 1 if words is None else words[b][t] & (2 ** 64 - 1)
                hide[t, n:] = torch.tensor([not word >> u & 1 for u in range(T)], device="cuda")
            for h in range(H):
                k, v = s["k"][b, h, :n + T].double(), s["v"][b, h, :n + T].double()
                for x in range(h * G, (h + 1) * G):
                    z = torch.einsum("td,nd->tn", s["q"][b, x].double(), k) / math.sqrt(d)
                    z = z.masked_fill(hide, -math.inf)
                    lse[b, x] = torch.logsumexp(z, -1)
                    p = torch.exp(z - lse[b, x][:, None])
                    o[b, x] = torch.einsum("tn,nd->td", p, v)
                    if w is not None:
                        w[b, h, :n + T] += p.sum(0) if s["counted"] is None else p[0]
        return [o, lse] if w is None else [o, lse, w]
    # evict: slot by slot on the host
    k, v, w, slots = (s[x].cpu() for x in ("k", "v", "weights", "slots"))
    left = []
    for b, n in enumerate(s["lens"]):
        m = min(n, c["keep"])
        left.append(m)
        for h in range(c["H"]):
            pos, wt = slots[b, h].tolist(), w[b, h].tolist()
            newest = max(pos[:n], default=0)
            ranked = sorted(range(n), key=lambda i: (0 if pos[i] > newest - c["recent"] else 1,
                                                     0.0 if pos[i] > newest - c["recent"] else -wt[i], i))[:m]
            stay = set(ranked)
            to = [i for i in range(m) if i not in stay]
            of = sorted(i for i in ranked if i >= m)
            for t in (k, v, w, slots):
                t[b, h, to] = t[b, h, of]
            w[b, h, m:], slots[b, h, m:] = 0.0, -1
    return [k.cuda().double(), v.cuda().double(), w.cuda().double(), slots.cuda(),
            torch.tensor(left, dtype=torch.int32, device="cuda")]
