"""Operators on a key's way into attention and its cache, and out of it again, as one
measured program: the cases, their inputs, one pass through each operator, and what
that pass cannot do without.

  rope     queries and keys normalised for each head (or not) and rotated by their
           positions, which may have several axes (time, height, width)
  rope_bwd its gradients: of queries, keys and both norms' weights
  append   the same for new tokens of a serving loop, keys and values going straight
           into the pages of the cache
  weights  attention weight that the cached places got from the new tokens, summed over
           the tokens and over the query heads of a kv head, added to running sums
  evict    of each (layer, sequence, kv head), the places with the largest sums and the
           most recent ones kept, moved together in the pages

With ``own`` false a pass runs in elementary torch operations in 32 bits (64 for the
angles); with ``own`` true it makes the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # two short texts in one batch, latency only: narrow heads, a rotation without norms
        dict(name="rope-short", op="rope", B=2, N=150, H=8, Hkv=2, d=64, rot=64, norm="", axes=1, pairs=False, fused=False,
             far=0),
        # the training step's shape: norms of queries and keys, whole heads rotated
        dict(name="rope-train", op="rope", B=4, N=8192, H=16, Hkv=16, d=128, rot=128, norm="float32", axes=1, pairs=False,
             fused=False, far=0),
        # video tokens: three axes, neighbouring channels as pairs, views into one projection's output, odd length
        dict(name="rope-video", op="rope", B=1, N=20011, H=32, Hkv=8, d=128, rot=128, norm="bfloat16", axes=3, pairs=True,
             fused=True, far=0),
        # the training step's backward pass
        dict(name="rope-bwd-train", op="rope_bwd", B=4, N=8192, H=16, Hkv=16, d=128, rot=128, norm="float32", axes=1,
             pairs=False, fused=False, far=0),
        # wide heads of which a quarter is rotated, shared keys, odd length, far positions
        dict(name="rope-bwd-d256", op="rope_bwd", B=3, N=2003, H=16, Hkv=4, d=256, rot=64, norm="bfloat16", axes=1,
             pairs=False, fused=True, far=500000),
        # one decoding step of 64 users
        dict(name="append-step", op="append", B=64, H=32, Hkv=8, d=128, rot=128, norm="bfloat16", axes=1, pairs=False,
             fused=True, far=0, page=64, lo=1, hi=8192, n=1, ragged=False),
        # packed prompts of 65536 tokens in all, from short ones to long ones
        dict(name="append-prompts", op="append", B=14, H=16, Hkv=16, d=128, rot=128, norm="float32", axes=1, pairs=False,
             fused=False, far=0, page=64, lo=0, hi=0, n=4681, ragged=True),
        # the decode step of a busy server adds its weights to the running sums
        dict(name="weights-step", op="weights", B=64, H=32, Hkv=8, d=128, page=64, lo=1, hi=8192, n=1, ragged=False,
             tree=False, decay=1.0),
        # a long prompt scored by its last 64 tokens
        dict(name="weights-window", op="weights", B=1, H=32, Hkv=8, d=128, page=128, lo=32704, hi=32704, n=64, ragged=False,
             tree=False, decay=0.0),
        # drafted trees, one head of keys for each query head, many middling sequences, older sums fading
        dict(name="weights-tree-d64", op="weights", B=32, H=16, Hkv=16, d=64, page=16, lo=3, hi=2500, n=7, ragged=True,
             tree=True, decay=0.98),
        # one layer of a long prompt cut down to its budget
        dict(name="evict-prompt", op="evict", B=1, L=1, Hkv=8, d=128, page=128, lo=32768, hi=32768, keep=2048, recent=64),
        # sequences a little past their budget, in every layer
        dict(name="evict-batch", op="evict", B=16, L=16, Hkv=8, d=128, page=16, lo=1000, hi=1100, keep=1024, recent=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "rope_bwd", "rope_bwd", "append", "weights", "weights", "weights", "evict", "evict"])
    d = rng.choice([64, 128, 256])
    Hkv, G = rng.choice([(1, 8), (2, 16), (2, 7), (4, 1), (8, 4), (4, 8), (16, 1), (8, 2), (3, 5), (1, 71)])
    H, page = Hkv * G, rng.choice([16, 32, 64, 128, 256])
    how = dict(H=H, Hkv=Hkv, d=d, rot=16 * rng.randint(1, d // 16) if rng.random() < 0.5 else d,
               norm=rng.choice(["", "float32", "bfloat16"]), axes=rng.choice([1, 1, 2, 3, 4]), pairs=rng.random() < 0.5,
               fused=rng.random() < 0.5, far=rng.choice([0, 0, 3000, 2000000]))
    if op in ("rope", "rope_bwd"):
        B = _log(rng, 1, 16)
        return dict(op=op, B=B, N=max(1, min(_log(rng, 1, 32768), int(1.2e8 / (B * (H + Hkv) * d)))), **how)
    B = _log(rng, 1, 96)
    if op == "append":
        n = _log(rng, 1, 4096) if rng.random() < 0.7 else 1
        n = max(1, min(n, int(1.0e8 / (B * (H + 2 * Hkv) * d))))
        return dict(op=op, B=B, page=page, lo=0, hi=_log(rng, 1, 2000), n=n, ragged=rng.random() < 0.7, **how)
    if op == "weights":
        n = _log(rng, 1, 160) if rng.random() < 0.7 else 1
        hi = min(_log(rng, 16, 32768), int(2.5e8 / (B * Hkv * d)), int(4e9 / (B * H * n * d)))
        hi = max(hi, 2)
        return dict(op=op, B=B, H=H, Hkv=Hkv, d=d, page=page, lo=rng.choice([0, 1, hi // 3, hi]), hi=hi, n=n,
                    ragged=rng.random() < 0.7, tree=rng.random() < 0.5, decay=rng.choice([0.0, 1.0, 1.0, 0.9]))
    B, L = _log(rng, 1, 24), rng.randint(1, 8)
    hi = max(4, min(_log(rng, 16, 32768), int(1.0e8 / (B * L * Hkv * d))))
    keep = rng.randint(0, hi) if rng.random() < 0.9 else hi + 5
    return dict(op=op, B=B, L=L, Hkv=Hkv, d=d, page=page, lo=rng.choice([0, 1, hi // 3, hi]), hi=hi, keep=keep,
                recent=rng.choice([0, min(1, keep), keep // 4, keep]))


def _lengths(case):
    """Cached and new tokens of each sequence: fixed by the case, so that its work is."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    n = case.get("n", 0)
    new = [r.randint(0, n) if case.get("ragged") else n for _ in range(case["B"])]
    if case["op"] == "append" and case["ragged"]:  # mostly short prompts, a few long ones, n a sequence on average
        w = [math.exp(r.uniform(0.0, 4.85)) for _ in range(case["B"])]
        new = [int(n * case["B"] * x / sum(w)) for x in w]
    if sum(new) == 0 and n:
        new[-1] = n
    return lens, new


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    op, Hkv, d = case["op"], case["Hkv"], case["d"]
    if op in ("rope", "rope_bwd"):
        tokens, heads = case["B"] * case["N"], case["H"] + Hkv
        passes = 2 if op == "rope" else 3 if case["norm"] else 2  # the norm's gradient takes the inputs too
        each = (4 if case["norm"] else 0) + 3 * case["rot"] / d + (8 if case["norm"] and op == "rope_bwd" else 0)
        return {"bytes": passes * tokens * heads * d * 2 + tokens * case["axes"] * 4, "flops": tokens * heads * d * each}
    lens, new = _lengths(case)
    if op == "append":
        tokens, H = sum(new), case["H"]
        each = (4 if case["norm"] else 0) + 3 * case["rot"] / d
        return {"bytes": 2 * 2 * tokens * (H + 2 * Hkv) * d + 4 * sum(_pages(b, case["page"]) for b in new),
                "flops": tokens * (H + Hkv) * d * each}
    if op == "weights":
        H, live = case["H"], [(a, b) for a, b in zip(lens, new) if b]
        places = sum(a + b for a, b in live)
        mask = sum(new) * 8 * _pages(case["n"], 64) if case["tree"] else 0
        return {"bytes": places * Hkv * (d * 2 + (8 if case["decay"] else 4)) + sum(new) * H * (d * 2 + 4) + mask
                + 4 * sum(_pages(a + b, case["page"]) for a, b in live),
                "flops": sum(2 * b * H * d * (a + (b if case["tree"] else (b + 1) / 2)) for a, b in live)}
    heads, keep, recent, moved, sums = case["L"] * Hkv, case["keep"], case["recent"], 0, 0
    for a in lens:
        if a > keep:  # all rows behind the first place that goes; of m places that go it is about the m-th part
            moved += max(0, keep - (a - recent) // (a - keep + 1))
            sums += a
    return {"bytes": heads * (moved * d * 2 * 2 * 2 + sums * 4 * 2 + 4 * sum(min(a, keep) for a in lens)), "flops": 0}


# ------------------------------------------------------------------ inputs
def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _rope_state(s, case, g, lead):
    """q, k (and v) of shape lead + (heads, d), each head with a scale of its own; weights, angles' tables."""
    H, Hkv, d, rot = case["H"], case["Hkv"], case["d"], case["rot"]
    heads = [H, Hkv, Hkv]
    size = torch.exp(0.5 * torch.randn((sum(heads), 1), generator=g, device=DEV)).to(torch.bfloat16)
    x = _normal(lead + (sum(heads), d), g).mul_(size)
    parts = torch.split(x, heads, dim=-2)
    s["q"], s["k"], s["v"] = parts if case["fused"] else [p.contiguous() for p in parts]
    s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).to(torch.float32).to(DEV)
    s["qw"] = s["kw"] = None
    if case["norm"]:
        t = getattr(torch, case["norm"])
        s["qw"], s["kw"] = [(1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(t) for _ in range(2)]
    s["axes"], s["pairs"] = None, case["pairs"]
    if case["axes"] > 1:  # a run of frequencies for each axis, the first one's the shortest
        cut = sorted(rot // 2 * (2 * a + 1) // (2 * case["axes"]) for a in range(1, case["axes"]))
        s["axes"] = tuple(sum(i >= c for c in cut) for i in range(rot // 2))
    return s


def _grid(case, count, g):
    """Positions of `count` tokens: a line, or the cells of frames of 30 x 52 on several axes."""
    i = torch.arange(count, dtype=torch.int32, device=DEV) + case["far"]
    if case["axes"] == 1:
        return i
    return torch.stack([i // 1560, i // 52 % 30, i % 52, i // 7][: case["axes"]])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = random.Random(seed)
    op, B = case["op"], case["B"]
    s = dict(op=op)
    if op in ("rope", "rope_bwd"):
        N = case["N"]
        _rope_state(s, case, g, (B, N))
        at = _grid(case, N, g)
        s["positions"] = at.unsqueeze(-2).expand(at.shape[:-1] + (B, N)).contiguous()
        if op == "rope_bwd":
            s["dq"], s["dk"] = _normal((B, N, case["H"], case["d"]), g), _normal((B, N, case["Hkv"], case["d"]), g)
        return s
    lens, new = _lengths(case)
    page = case["page"]
    s.update(page=page, B=B, lens=_int(lens))
    held = [_pages(a + b, page) for a, b in zip(lens, new)]
    cols = max(held) + 1
    pool = sum(held) + 8
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32, device=DEV)
    held_t = _int(held)
    at = torch.cumsum(held_t, 0) - held_t
    c = torch.arange(cols, device=DEV)
    inside = c[None] < held_t[:, None]
    table[inside] = order[(at[:, None] + c[None])[inside]]
    s["table"] = table
    shape = (pool, page, case["Hkv"], case["d"])
    if op == "evict":
        L, places = case["L"], cols * page
        s["refs"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
        s["refs"][order[: sum(held)].long()] = 1
        s["k_pages"], s["v_pages"] = _normal((L,) + shape, g), _normal((L,) + shape, g)
        # sums of attention weight: a few large ones, many small ones, equal ones among them
        w = torch.exp(2.0 * torch.randn((L, B, case["Hkv"], places), generator=g, device=DEV)).to(torch.bfloat16).float()
        w = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.02, 0.0, w)
        s["weights"] = w * (torch.arange(places, device=DEV) < s["lens"][:, None, None])
        s["keep"], s["recent"] = case["keep"], case["recent"]
        return s
    s["cu"] = _int(np.concatenate([[0], np.cumsum(new)]).tolist())
    total = sum(new)
    s["k_pages"] = _normal(shape, g)
    if op == "append":
        s["v_pages"] = _normal(shape, g)
        _rope_state(s, case, g, (total,))
        # with several axes, or cut out of a longer text, positions are not the places in the cache
        s["positions"] = _grid(case, total, g) if case["axes"] > 1 or case["far"] else None
        return s
    H, n = case["H"], case["n"]
    s["q"], s["n"], s["decay"] = _normal((total, H, case["d"]), g), n, case["decay"]
    s["mask"] = None
    if case["tree"]:  # a drafted tree: every token's parent is an earlier one, often the one before
        words = -(-n // 64)
        rows = []
        for b in new:
            seen = []
            for i in range(b):
                p = -1 if i == 0 else (i - 1 if r.random() < 0.4 else r.randrange(-1 if r.random() < 0.1 else 0, i))
                seen.append((seen[p] if p >= 0 else 0) | (1 << i))
            rows += [[(x >> (64 * w)) & (2**64 - 1) for w in range(words)] for x in seen]
        s["mask"] = torch.from_numpy(np.array(rows, dtype=np.uint64).reshape(total, words).view(np.int64)).to(DEV)
    s["lse"] = torch.empty((H, total), dtype=torch.float32, device=DEV)  # what the attention of these tokens has left
    x, _, real = _scores(s)
    s["lse"][:] = torch.logsumexp(x, -1).permute(1, 2, 0, 3).reshape(H, B, n)[:, real]
    w = torch.rand((B, case["Hkv"], cols * page), generator=g, device=DEV)
    s["weights"] = w * (torch.arange(cols * page, device=DEV) < s["lens"][:, None, None])
    return s


# ------------------------------------------------------------------ plain forms
def _turn(x, cos, sin, pairs):
    """The first 2 * cos.shape[-1] columns of x rotated."""
    half = cos.shape[-1]
    a, b = (x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]) if pairs else (x[..., :half], x[..., half : 2 * half])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([y, x[..., 2 * half :]], -1)


def _angles(s, positions):
    pos = positions.double()
    if s["axes"] is None:
        turn = pos[..., None] * s["inv_freq"].double()
    else:
        turn = pos[torch.tensor(s["axes"], device=DEV)].movedim(0, -1) * s["inv_freq"].double()
    return torch.cos(turn).float()[..., None, :], torch.sin(turn).float()[..., None, :]


def _rope(s, positions):
    cos, sin = _angles(s, positions)
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        out.append(_turn(x, cos, sin, s["pairs"]).to(torch.bfloat16))
    return out


def _rope_bwd(s):
    cos, sin = _angles(s, s["positions"])
    out, sums = [], []
    for dy, x, w in ((s["dq"], s["q"], s["qw"]), (s["dk"], s["k"], s["kw"])):
        g = _turn(dy.float(), cos, -sin, s["pairs"])
        if w is not None:
            x, w = x.float(), w.float()
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            sums.append((g * x * r).flatten(0, -2).sum(0))
            g = r * (w * g - x * r * r * (x * w * g).mean(-1, keepdim=True))
        out.append(g.to(torch.bfloat16))
    return tuple(out + sums)


def _append(s):
    total = s["q"].shape[0]
    cu = s["cu"].long()
    t = torch.arange(total, device=DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = s["lens"].long()[b] + t - cu[b]
    page = s["table"].long()[b, pos // s["page"]]
    at = pos if s["positions"] is None else s["positions"]
    q, k = _rope(s, at)
    s["k_pages"][page, pos % s["page"]] = k
    s["v_pages"][page, pos % s["page"]] = s["v"]
    return q, s["k_pages"], s["v_pages"]


def _scores(s):
    """Scores of all new tokens and places [B, Hkv, G, n, places], -inf where a token does not see a place or
    is none; which places are the sequence's; which tokens there are."""
    q, n, B, page = s["q"], s["n"], s["B"], s["page"]
    total, H, d = q.shape
    Hkv = s["k_pages"].shape[2]
    most = s["table"].shape[1] * page
    pos = torch.arange(most, device=DEV)
    k = s["k_pages"][s["table"].long().clamp(min=0)[:, pos // page], (pos % page).expand(B, most)]
    k = k.float().permute(0, 2, 1, 3)  # [B, Hkv, most, d]
    cu = s["cu"].long()
    i = torch.arange(n, device=DEV)
    real = i[None] < (cu[1:] - cu[:-1])[:, None]  # [B, n]
    src = (cu[:-1, None] + i[None]).clamp(max=total - 1)
    rows = q[src].float().reshape(B, n, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    x = (torch.matmul(rows, k.transpose(2, 3)) * (1.0 / math.sqrt(d))).reshape(B, Hkv, H // Hkv, n, most)
    at = pos[None] - s["lens"].long()[:, None]  # place among the new tokens
    j = at.clamp(0, n - 1)
    if s["mask"] is None:
        sees = j[:, None, :] <= i[None, :, None]
    else:
        words = s["mask"][src]  # [B, n, words]
        sees = (torch.gather(words, 2, (j // 64)[:, None, :].expand(B, n, most)) >> (j % 64)[:, None, :]) & 1 == 1
    held = at < (cu[1:] - cu[:-1])[:, None]
    sees = ((at < 0)[:, None, :] | (held[:, None, :] & sees)) & real[:, :, None]
    return x.masked_fill_(~sees[:, None, None], float("-inf")), held & real[:, :1], real


def _weights(s):
    x, held, real = _scores(s)
    B, Hkv, G, n, most = x.shape
    lse = torch.zeros((Hkv, G, B, n), dtype=torch.float32, device=DEV)
    lse[:, :, real] = s["lse"].reshape(Hkv, G, -1)
    lse = torch.where(torch.isneginf(lse), 0.0, lse)  # a token that sees nothing
    p = torch.exp(x - lse.permute(2, 0, 1, 3)[..., None]).sum((2, 3))
    w = s["weights"]
    old = w * s["decay"] if s["decay"] else torch.zeros_like(w)
    w.copy_(torch.where(held[:, None], old + p, w))
    return w


def _evict(s):
    w = s["weights"].clone()  # the sums as they are before the call, for the next pass
    keep, recent, page, table = s["keep"], s["recent"], s["page"], s["table"].long()
    L, B, Hkv, places = w.shape
    lens = s["lens"].long()
    goes = lens > keep
    pos = torch.arange(places, device=DEV)
    value = torch.where(torch.isnan(w), float("-inf"), w + 0.0)
    first = torch.argsort(value, dim=-1, descending=True, stable=True)
    late = (pos >= (lens - recent)[:, None]).int() + 3 * (pos >= lens[:, None]).int()  # 0 older, 1 recent, 4 none
    rank = torch.tensor([1, 0, 0, 0, 2], device=DEV)[late][None, :, None].expand(L, B, Hkv, places)
    first = torch.gather(first, -1, torch.argsort(torch.gather(rank, -1, first), dim=-1, stable=True))
    if keep > places:
        first = torch.cat([first, first.new_zeros((L, B, Hkv, keep - places))], -1)
    i = torch.arange(keep, device=DEV)
    kept = torch.where(goes[:, None, None], first[..., :keep].sort(-1).values, i)  # [L, B, Hkv, keep]
    kept = torch.where((goes[:, None] | (i < lens[:, None]))[:, None], kept, -1)
    b = goes.nonzero()[:, 0]
    src = kept[:, b]
    ids = torch.gather(table[b][None, :, None].expand(L, -1, Hkv, -1), -1, src // page)
    layer = torch.arange(L, device=DEV)[:, None, None, None]
    head = torch.arange(Hkv, device=DEV)[:, None]
    to = table[b][:, i // page][None, :, None]
    for x in (s["k_pages"], s["v_pages"]):
        x[layer, to, i % page, head] = x[layer, ids, src % page, head]
    new = torch.zeros_like(w[:, b])
    if keep:
        new[..., : min(keep, places)] = torch.gather(w[:, b], -1, src)[..., : min(keep, places)]
    w[:, b] = torch.where(pos < lens[b, None, None], new, w[:, b])
    return s["k_pages"], s["v_pages"], w, torch.where(goes, keep, lens).to(torch.int32), kept.to(torch.int32)


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["op"]
    if not own:
        if op == "rope":
            return tuple(_rope(s, s["positions"]))
        return {"rope_bwd": _rope_bwd, "append": _append, "weights": _weights, "evict": _evict}[op](s)
    import exact_attention_blackwell_gb300 as fa

    if op == "rope":
        return fa.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                               axes=s["axes"], interleaved=s["pairs"])
    if op == "rope_bwd":
        out = fa.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["qw"],
                                  k_weight=s["kw"], eps=EPS, axes=s["axes"], interleaved=s["pairs"])
        return out if s["qw"] is not None else out[:2]
    if op == "append":
        q = fa.cache_append_rope(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"],
                                 s["inv_freq"], positions=s["positions"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                                 axes=s["axes"], interleaved=s["pairs"])
        return q, s["k_pages"], s["v_pages"]
    if op == "weights":
        return fa.attention_weights_paged(s["q"], s["k_pages"], s["table"], s["lens"], s["cu"], s["n"], s["lse"],
                                          s["weights"], tree_mask=s["mask"], decay=s["decay"])
    w = s["weights"].clone()  # the sums as they are before the call, for the next pass
    lens, kept = fa.cache_evict(s["refs"], s["k_pages"], s["v_pages"], s["table"], s["lens"], w, s["keep"], s["recent"])
    return s["k_pages"], s["v_pages"], w, lens, kept


# ------------------------------------------------------------------ 64 bits, from the definitions
def _spin(x, angle, pairs):
    """Complex numbers turned: column pairs of x as real and imaginary parts."""
    half = angle.shape[-1]
    y = x.clone()
    re, im = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    z = torch.complex(x[..., re], x[..., im]) * torch.polar(torch.ones_like(angle), angle).unsqueeze(-2)
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_rope(s, positions):
    f = s["inv_freq"].double()
    lead = s["q"].shape[:-2]
    rows = positions.double().reshape((-1,) + tuple(lead))
    angle = torch.empty(lead + (f.numel(),), dtype=torch.float64, device=DEV)
    for i in range(f.numel()):
        angle[..., i] = rows[0 if s["axes"] is None else s["axes"][i]] * f[i]
    ins, outs = [], []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.double().requires_grad_(s["op"] == "rope_bwd")
        y = x
        ins.append(x)
        if w is not None:
            w = w.double().requires_grad_(s["op"] == "rope_bwd")
            ins.append(w)
            y = w * x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)
        outs.append(_spin(y, angle, s["pairs"]))
    return ins, outs


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "rope":
        return tuple(_exact_rope(s, s["positions"])[1])
    if op == "rope_bwd":
        ins, outs = _exact_rope(s, s["positions"])
        got = torch.autograd.grad(outs, ins, [s["dq"].double(), s["dk"].double()])
        return (got[0], got[2], got[1], got[3]) if len(ins) == 4 else tuple(got)
    page, lens, table = s["page"], s["lens"].tolist(), s["table"].tolist()
    if op == "append":
        cu = s["cu"].tolist()
        if s["positions"] is None:
            places = [lens[b] + i for b in range(case["B"]) for i in range(cu[b + 1] - cu[b])]
            positions = torch.tensor(places, device=DEV)
            if s["axes"] is not None:
                positions = positions.expand(case["axes"], -1)
        else:
            positions = s["positions"]
        q, new = _exact_rope(s, positions)[1]
        k, v = s["k_pages"].double(), s["v_pages"].double()
        for b in range(case["B"]):
            done = 0
            while done < cu[b + 1] - cu[b]:  # page by page
                p = lens[b] + done
                m = min(page - p % page, cu[b + 1] - cu[b] - done)
                a = cu[b] + done
                k[table[b][p // page], p % page : p % page + m] = new[a : a + m]
                v[table[b][p // page], p % page : p % page + m] = s["v"][a : a + m].double()
                done += m
        return q, k, v
    Hkv, d = case["Hkv"], case["d"]
    if op == "weights":
        q, cu, G = s["q"], s["cu"].tolist(), case["H"] // Hkv
        out = s["weights"].double()
        bits = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint64)
        for b in range(case["B"]):
            n = cu[b + 1] - cu[b]
            keys = lens[b] + n
            if n == 0:
                continue
            ids = torch.tensor(table[b][: _pages(keys, page)], device=DEV)
            see = np.ones((n, keys), dtype=bool)
            for i in range(n):
                for j in range(n):
                    see[i, lens[b] + j] = j <= i if bits is None else bool((int(bits[cu[b] + i, j // 64]) >> (j % 64)) & 1)
            see = torch.from_numpy(see).to(DEV)
            for h in range(Hkv):
                kk = s["k_pages"][ids, :, h].reshape(-1, d)[:keys].double()
                z = torch.einsum("ngd,kd->gnk", q[cu[b] : cu[b + 1], h * G : (h + 1) * G].double(), kk) / math.sqrt(d)
                z = torch.exp(z - s["lse"][h * G : (h + 1) * G, cu[b] : cu[b + 1], None].double())
                out[b, h, :keys] = out[b, h, :keys] * s["decay"] + torch.where(see, z, 0.0).sum((0, 1))
        return out
    k, v, w = s["k_pages"].double(), s["v_pages"].double(), s["weights"].double()
    keep, recent = s["keep"], s["recent"]
    for b in range(case["B"]):
        a = lens[b]
        if a <= keep:
            continue
        ids = torch.tensor(table[b][: _pages(a, page)], device=DEV)
        older = w[:, b, :, : a - recent]
        rank = older.cpu().numpy()
        stay = np.argsort(-rank, axis=-1, kind="stable")[..., : keep - recent]
        stay.sort(axis=-1)
        stay = np.concatenate([stay, np.broadcast_to(np.arange(a - recent, a), stay.shape[:-1] + (recent,))], -1)
        stay = torch.from_numpy(stay).to(DEV)  # [L, Hkv, keep]
        for x in (k, v):
            rows = x[:, ids].flatten(1, 2)  # [L, places, Hkv, d]
            moved = torch.gather(rows, 1, stay.transpose(1, 2)[..., None].expand(-1, -1, -1, d))
            rows[:, :keep] = moved
            x[:, ids] = rows.unflatten(1, (-1, page))
        sums = torch.gather(w[:, b], -1, stay)
        w[:, b, :, :a] = 0.0
        w[:, b, :, :keep] = sums
    return k, v, w, None, None
