"""The paged-cache operators as one measured program: the cases, their inputs,
one pass through each operator, and what that pass cannot do without.

A serving loop keeps the keys and values of its sequences in pages of a shared
pool.  The operators around such a cache are

  attend   attention of a few new tokens (one, a chain, or a tree of drafted
           tokens) over the cached prefix and over one another
  append   new keys and values written into the pages
  compact  the accepted path of a drafted tree moved together, in every layer
  fork     rows of the page table copied from parent rows, shared by counting
  resize   pages taken for growing rows (a shared last page is copied first)
           and given back by shrinking ones
  beam     fork, then resize up and back: what one step of a beam search does

With ``own`` false a pass runs in elementary torch operations in 32 bits; with
``own`` true it makes the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest call of a chat with one user: one token over a short prefix, latency only
        dict(name="attend-one-short", op="attend", B=1, H=32, Hkv=8, d=128, page=16, lo=777, hi=777, n=1, ragged=False,
             tree=False),
        # the ordinary decode step of a busy server: 64 users, lengths of every size
        dict(name="attend-one-batch", op="attend", B=64, H=32, Hkv=8, d=128, page=64, lo=1, hi=8192, n=1, ragged=False,
             tree=False),
        # a chain of drafted tokens, one head of keys for each query head, many middling sequences
        dict(name="attend-chain-d64", op="attend", B=32, H=16, Hkv=16, d=64, page=16, lo=3, hi=2500, n=7, ragged=True,
             tree=False),
        # verifying drafted trees of up to 33 tokens in a batch, the widest heads
        dict(name="attend-tree-d256", op="attend", B=16, H=16, Hkv=4, d=256, page=32, lo=100, hi=7000, n=33,
             ragged=True, tree=True),
        # one long document: a tree of 64 tokens over 32768 cached ones
        dict(name="attend-tree-long", op="attend", B=1, H=32, Hkv=8, d=128, page=128, lo=32768, hi=32768, n=64,
             ragged=False, tree=True),
        # the keys and values of one decode step
        dict(name="append-step", op="append", B=64, Hkv=8, d=128, page=16, lo=1, hi=4000, n=1, ragged=False),
        # packed prompts of 65536 tokens in all, from short ones to long ones
        dict(name="append-prompts", op="append", B=14, Hkv=16, d=128, page=64, lo=0, hi=0, n=9362, ragged=True),
        # a single user's accepted path, in every layer
        dict(name="compact-one", op="compact", B=1, L=16, Hkv=8, d=128, page=16, lo=333, hi=333, n=24, keep=5),
        # the accepted paths of a batch, in every layer
        dict(name="compact-batch", op="compact", B=32, L=32, Hkv=8, d=128, page=32, lo=20, hi=400, n=64, keep=17),
        # the table of a beam search reordered: wide rows, a tenth of them freed
        dict(name="fork-tables", op="fork", B=128, page=16, lo=1, hi=30000, cols=2048),
        # pages taken for a drafted tree and given back
        dict(name="resize-draft", op="resize", B=48, L=2, Hkv=8, d=64, page=16, lo=1, hi=900, n=40, cols=64),
        # one step of a beam search: rows share last pages, which are copied in every layer
        dict(name="beam-step", op="beam", B=64, L=24, Hkv=8, d=128, page=64, lo=30, hi=1000, n=1, cols=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "compact", "fork", "resize", "beam"])
    page = rng.choice([16, 32, 64, 128])
    d = rng.choice([64, 128, 256])
    if op == "attend":
        Hkv, G = rng.choice([(1, 8), (2, 16), (2, 7), (4, 1), (8, 4), (4, 8), (16, 1), (8, 2), (3, 5), (1, 71)])
        B = _log(rng, 1, 96)
        n = _log(rng, 1, 160) if rng.random() < 0.7 else 1
        # bounds that keep every draw below the largest listed case
        hi = min(_log(rng, 16, 32768), int(2.5e8 / (B * Hkv * d)), int(4e9 / (B * Hkv * G * n * d)))
        hi = max(hi, 2)
        lo = rng.choice([0, 1, hi // 3, hi])
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, d=d, page=page, lo=lo, hi=hi, n=n, ragged=rng.random() < 0.7,
                    tree=rng.random() < 0.7)
    if op == "append":
        Hkv = rng.choice([1, 2, 3, 8, 16])
        B = _log(rng, 1, 128)
        n = min(_log(rng, 1, 8192), int(1.2e8 / (B * Hkv * d)))
        return dict(op=op, B=B, Hkv=Hkv, d=d, page=page, lo=0, hi=_log(rng, 1, 2000), n=max(n, 1), ragged=True)
    if op == "compact":
        n = _log(rng, 2, 64)
        return dict(op=op, B=_log(rng, 1, 32), L=rng.randint(1, 24), Hkv=rng.choice([1, 2, 5, 8]), d=min(d, 128), page=page,
                    lo=0, hi=_log(rng, 1, 400), n=n, keep=rng.randint(1, min(n, 20)))
    cols = _log(rng, 8, 1500)
    if op == "fork":
        return dict(op=op, B=_log(rng, 1, 160), page=page, lo=0, hi=cols * page - rng.randint(0, page), cols=cols)
    cols = min(cols, 24)
    n = 1 if op == "beam" else _log(rng, 1, 64)
    return dict(op=op, B=_log(rng, 1, 56), L=rng.randint(1, 16), Hkv=rng.choice([1, 2, 5, 8]), d=min(d, 128), page=page, lo=0,
                hi=max(1, cols * page - n - 1), n=n, cols=cols)


def _lengths(case):
    """Cached and new tokens of each sequence: fixed by the case, so that its work is."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    n = case.get("n", 0)
    new = [r.randint(0, n) if case.get("ragged") else n for _ in range(case["B"])]
    if case["op"] == "append" and case.get("ragged"):  # mostly short prompts, a few long ones, n a sequence on average
        w = [math.exp(r.uniform(0.0, 4.85)) for _ in range(case["B"])]
        new = [int(n * case["B"] * x / sum(w)) for x in w]
    if sum(new) == 0 and n:
        new[-1] = n
    keep = [r.randint(0, case.get("keep", 0)) for _ in range(case["B"])]
    if case["op"] == "compact":
        keep[0] = case["keep"]
    return lens, new, keep


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    lens, new, keep = _lengths(case)
    op, page = case["op"], case["page"]
    if op == "attend":
        Hkv, H, d = case["Hkv"], case["H"], case["d"]
        kv = sum(a + b for a, b in zip(lens, new) if b) * Hkv * d * 2 * 2
        q = sum(new) * H * d * 2 * 2 + sum(new) * (H * 4 + (8 * -(-case["n"] // 64) if case["tree"] else 0))
        table = sum(_pages(a + b, page) for a, b in zip(lens, new)) * 4
        return {"bytes": kv + q + table, "flops": sum(4 * b * H * d * (a + (b if case["tree"] else (b + 1) / 2)) for a, b in zip(lens, new))}
    if op == "append":
        return {"bytes": 2 * 2 * sum(new) * case["Hkv"] * case["d"] * 2 + 4 * sum(_pages(b, page) for b in new), "flops": 0}
    if op == "compact":
        return {"bytes": 2 * 2 * case["L"] * sum(keep) * case["Hkv"] * case["d"] * 2 + 4 * sum(keep), "flops": 0}
    pages = sum(_pages(a, page) for a in lens)
    if op == "fork":  # each row read and written, each page counted twice
        return {"bytes": pages * 4 * 6, "flops": 0}
    if op == "resize":
        grown = sum(_pages(a + b, page) - _pages(a, page) for a, b in zip(lens, new))
        return {"bytes": grown * 4 * 8 + case["B"] * 4 * 6, "flops": 0}
    # beam: the table as for fork; three of four rows share a last page with another row
    share = 2 * 2 * case["L"] * case["Hkv"] * case["d"] * 2 * sum(a % page for a in lens) // 2
    return {"bytes": pages * 4 * 6 + share, "flops": 0}


# ------------------------------------------------------------------ inputs
def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = random.Random(seed)
    lens, new, keep = _lengths(case)
    op, page, B = case["op"], case["page"], case["B"]
    s = dict(op=op, page=page, B=B, lens=_int(lens))
    held = [_pages(a + (b if op in ("attend", "append", "compact") else 0), page) for a, b in zip(lens, new)]
    if op == "compact":
        held = [_pages(a + case["n"], page) for a in lens]
    cols = case.get("cols", max(held) + 1)
    spare = 8 if op in ("attend", "append", "compact") else 8 + B * (2 + _pages(case.get("n", 0), page))
    pool = sum(held) + spare
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32, device=DEV)
    held_t = _int(held)
    at = torch.cumsum(held_t, 0) - held_t
    c = torch.arange(cols, device=DEV)
    inside = c[None] < held_t[:, None]
    table[inside] = order[(at[:, None] + c[None])[inside]]
    s["table"] = table
    refs = torch.zeros(pool, dtype=torch.int32, device=DEV)
    refs[order[: sum(held)].long()] = 1
    s["refs"] = refs
    if op in ("attend", "append", "compact", "resize", "beam"):
        shape = (pool, page, case["Hkv"], case["d"])
        if "L" in case:
            shape = (case["L"],) + shape
        s["k_pages"], s["v_pages"] = _normal(shape, g), _normal(shape, g)
    if op in ("attend", "append"):
        total = sum(new)
        s["cu"] = _int(np.concatenate([[0], np.cumsum(new)]).tolist())
        if op == "append":
            s["k"] = _normal((total, case["Hkv"], case["d"]), g)
            s["v"] = _normal((total, case["Hkv"], case["d"]), g)
            return s
        s["q"] = _normal((total, case["H"], case["d"]), g)
        s["n"] = case["n"]
        s["mask"] = None
        if case["tree"]:  # a drafted tree: every token's parent is an earlier one, often the one before
            words = -(-case["n"] // 64)
            rows = []
            for b in new:
                seen = []
                for i in range(b):
                    p = -1 if i == 0 else (i - 1 if r.random() < 0.4 else r.randrange(-1 if r.random() < 0.1 else 0, i))
                    seen.append((seen[p] if p >= 0 else 0) | (1 << i))
                rows += [[(x >> (64 * w)) & (2**64 - 1) for w in range(words)] for x in seen]
            s["mask"] = torch.from_numpy(np.array(rows, dtype=np.uint64).reshape(total, words).view(np.int64)).to(DEV)
        return s
    if op == "compact":
        path = [sorted(r.sample(range(case["n"]), m)) + [0] * (case["keep"] - m) for m in keep]
        s["path"], s["kept"] = _int(path), _int(keep)
        return s
    if op in ("fork", "beam"):
        parents = [r.randrange(B) if r.random() < 0.75 else b for b in range(B)]
        if op == "fork":
            parents = [-1 if r.random() < 0.1 else p for p in parents]
        s["parents"] = _int(parents)
    s["grow"] = case.get("n", 0)
    s["new"] = _int(new)
    return s


# ------------------------------------------------------------------ plain forms
def _positions(s, count):
    """Page and row of the first `count` places of every sequence: [B, count] each."""
    pos = torch.arange(count, device=DEV)
    page = s["table"].long()[:, (pos // s["page"]).clamp(max=s["table"].shape[1] - 1)]
    return page.clamp(min=0), (pos % s["page"]).expand_as(page)


def _attend(s):
    q, n, B = s["q"], s["n"], s["B"]
    total, H, d = q.shape
    Hkv = s["k_pages"].shape[2]
    most = s["table"].shape[1] * s["page"]
    page, row = _positions(s, most)
    k = s["k_pages"][page, row].float().permute(0, 2, 1, 3)  # [B, Hkv, most, d]
    v = s["v_pages"][page, row].float().permute(0, 2, 1, 3)
    cu = s["cu"].long()
    i = torch.arange(n, device=DEV)
    real = i[None] < (cu[1:] - cu[:-1])[:, None]  # [B, n]
    src = (cu[:-1, None] + i[None]).clamp(max=total - 1)
    rows = q[src].float().reshape(B, n, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    x = torch.matmul(rows, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    x = x.reshape(B, Hkv, H // Hkv, n, most)
    at = torch.arange(most, device=DEV)[None] - s["lens"].long()[:, None]  # place among the new tokens
    j = at.clamp(0, n - 1)
    if s["mask"] is None:
        sees = j[:, None, :] <= i[None, :, None]
    else:
        words = s["mask"][src]  # [B, n, words]
        sees = (torch.gather(words, 2, (j // 64)[:, None, :].expand(B, n, most)) >> (j % 64)[:, None, :]) & 1 == 1
    inside = (at >= 0) & (at < (cu[1:] - cu[:-1])[:, None])
    sees = (at < 0)[:, None, :] | (inside[:, None, :] & sees)
    x = torch.where(sees[:, None, None], x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    x = torch.exp(x - top)
    total_p = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(B, Hkv, -1, most), v).reshape(B, Hkv, H // Hkv, n, d)
    o = o / torch.where(total_p > 0, total_p, 1.0)
    lse = (top + torch.log(total_p))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, H, d)[real].to(torch.bfloat16)
    lse = lse.permute(1, 2, 0, 3).reshape(H, B, n)[:, real]
    return o, lse


def _append(s):
    total = s["k"].shape[0]
    cu = s["cu"].long()
    t = torch.arange(total, device=DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = s["lens"].long()[b] + t - cu[b]
    page = s["table"].long()[b, pos // s["page"]]
    s["k_pages"][page, pos % s["page"]] = s["k"]
    s["v_pages"][page, pos % s["page"]] = s["v"]
    return s["k_pages"], s["v_pages"]


def _compact(s):
    b, i = torch.nonzero(torch.arange(s["path"].shape[1], device=DEV)[None] < s["kept"][:, None], as_tuple=True)
    table, lens, page = s["table"].long(), s["lens"].long(), s["page"]
    src = lens[b] + s["path"].long()[b, i]
    dst = lens[b] + i
    for x in (s["k_pages"], s["v_pages"]):
        x[:, table[b, dst // page], dst % page] = x[:, table[b, src // page], src % page]
    return s["k_pages"], s["v_pages"], s["lens"] + s["kept"]


def _count(refs, pages, here, by):
    refs.index_add_(0, torch.where(here, pages, 0).reshape(-1).long(), here.reshape(-1).to(torch.int32) * by)


def _fork(s, lens):
    table, refs, parents = s["table"], s["refs"], s["parents"].long()
    held = (lens + s["page"] - 1) // s["page"]
    changed = parents != torch.arange(s["B"], device=DEV)
    c = torch.arange(table.shape[1], device=DEV)
    source = parents.clamp(min=0)
    takes = (parents >= 0)[:, None] & (c[None] < held[source][:, None])
    fresh = torch.where(takes, table[source], -1)
    _count(refs, fresh, takes & changed[:, None], 1)
    _count(refs, table, (c[None] < held[:, None]) & changed[:, None], -1)
    table.copy_(torch.where(changed[:, None], fresh, table))
    return torch.where(parents >= 0, lens[source], 0).to(torch.int32)


def _resize(s, lens, new):
    table, refs, page, B = s["table"], s["refs"], s["page"], s["B"]
    had, has = (lens + page - 1) // page, (new + page - 1) // page
    c = torch.arange(table.shape[1], device=DEV)[None]
    gone = (c >= has[:, None]) & (c < had[:, None])
    _count(refs, table, gone, -1)
    table.masked_fill_(gone, -1)
    grows = new > lens
    last = torch.gather(table, 1, (lens // page).clamp(max=table.shape[1] - 1)[:, None].long())[:, 0]
    partial = grows & (lens % page != 0)
    before = torch.tril(torch.ones(B, B, dtype=torch.bool, device=DEV), -1)
    rank = ((last[:, None] == last[None]) & partial[:, None] & partial[None] & before).sum(1)
    copies = partial & (refs[last.clamp(min=0).long()] - rank > 1)
    need = torch.where(grows, has - had, 0) + copies
    free = torch.argsort((refs != 0).int(), stable=True)
    lack = (need.sum() - (refs == 0).sum()).clamp(min=0)
    can = lack == 0
    grows, copies = grows & can, copies & can
    first = torch.cumsum(need, 0) - need
    k = (first + copies)[:, None] + c - had[:, None]
    taken = grows[:, None] & (c >= had[:, None]) & (c < has[:, None])
    own_page = copies[:, None] & (c == (lens // page)[:, None])
    k = torch.where(own_page, first[:, None], k).clamp(0, free.shape[0] - 1)
    _count(refs, last.clamp(min=0), copies, -1)
    _count(refs, free[k], taken | own_page, 1)
    table.copy_(torch.where(taken | own_page, free[k].to(torch.int32), table))
    moved = copies[:, None] & (torch.arange(page, device=DEV)[None] < (lens % page)[:, None])
    b, row = torch.nonzero(moved, as_tuple=True)
    to = free[first.clamp(0, free.shape[0] - 1)]
    for x in (s["k_pages"], s["v_pages"]):
        x[:, to[b], row] = x[:, last.long()[b], row]
    return torch.where((new > lens) & ~can, lens, new).to(torch.int32), torch.stack([lack, torch.zeros_like(lack)]).to(torch.int32)


def _plain(s):
    op = s["op"]
    if op == "attend":
        return _attend(s)
    if op == "append":
        return _append(s)
    if op == "compact":
        return _compact(s)
    if op == "fork":
        s["lens"] = _fork(s, s["lens"])
        return s["table"], s["refs"], s["lens"]
    if op == "resize":
        up, said = _resize(s, s["lens"], s["lens"] + s["new"])
        grown = s["table"].clone()
        down, _ = _resize(s, up, s["lens"])
        return grown, s["table"], s["refs"], up, down, said
    lens = _fork(s, s["lens"])
    up, said = _resize(s, lens, lens + s["grow"])
    s["lens"], _ = _resize(s, up, lens)
    return s["table"], s["refs"], s["lens"], up, said, s["k_pages"], s["v_pages"]


# ------------------------------------------------------------------ one pass
def run(s):
    if not own:
        return _plain(s)
    import exact_attention_blackwell_gb300 as fa

    op = s["op"]
    if op == "attend":
        return fa.attention_fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], s["n"],
                                      tree_mask=s["mask"])
    if op == "append":
        fa.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"])
        return s["k_pages"], s["v_pages"]
    if op == "compact":
        lens = fa.cache_compact(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["path"], s["kept"])
        return s["k_pages"], s["v_pages"], lens
    if op == "fork":
        s["lens"] = fa.cache_fork(s["refs"], s["table"], s["lens"], s["parents"], s["page"])
        return s["table"], s["refs"], s["lens"]
    if op == "resize":
        up, said = fa.cache_resize(s["refs"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["lens"] + s["new"])
        grown = s["table"].clone()
        down, _ = fa.cache_resize(s["refs"], s["k_pages"], s["v_pages"], s["table"], up, s["lens"])
        return grown, s["table"], s["refs"], up, down, said
    lens = fa.cache_fork(s["refs"], s["table"], s["lens"], s["parents"], s["page"])
    up, said = fa.cache_resize(s["refs"], s["k_pages"], s["v_pages"], s["table"], lens, lens + s["grow"])
    s["lens"], _ = fa.cache_resize(s["refs"], s["k_pages"], s["v_pages"], s["table"], up, lens)
    return s["table"], s["refs"], s["lens"], up, said, s["k_pages"], s["v_pages"]


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    op, page = s["op"], s["page"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    if op == "attend":
        q, cu = s["q"], s["cu"].tolist()
        total, H, d = q.shape
        Hkv = case["Hkv"]
        out = torch.zeros((total, H, d), dtype=torch.float64, device=DEV)
        lse = torch.full((H, total), float("-inf"), dtype=torch.float64, device=DEV)
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
            for h in range(H):
                kk = s["k_pages"][ids, :, h // (H // Hkv)].reshape(-1, d)[:keys].double()
                vv = s["v_pages"][ids, :, h // (H // Hkv)].reshape(-1, d)[:keys].double()
                z = (q[cu[b] : cu[b + 1], h].double() @ kk.T) / math.sqrt(d)
                z = z.masked_fill(~see, float("-inf"))
                norm = torch.logsumexp(z, dim=1)
                out[cu[b] : cu[b + 1], h] = torch.exp(z - norm[:, None]) @ vv
                lse[h, cu[b] : cu[b + 1]] = norm
        return out, lse
    if op == "append":
        cu = s["cu"].tolist()
        k, v = s["k_pages"].double(), s["v_pages"].double()
        for b in range(case["B"]):
            done = 0
            while done < cu[b + 1] - cu[b]:  # page by page
                p = lens[b] + done
                m = min(page - p % page, cu[b + 1] - cu[b] - done)
                a = cu[b] + done
                k[table[b][p // page], p % page : p % page + m] = s["k"][a : a + m].double()
                v[table[b][p // page], p % page : p % page + m] = s["v"][a : a + m].double()
                done += m
        return k, v
    if op == "compact":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        path, kept = s["path"].tolist(), s["kept"].tolist()
        for b in range(case["B"]):
            for i in range(kept[b]):  # paths ascend, so that a row is read before it is overwritten
                f, t = lens[b] + path[b][i], lens[b] + i
                for x in (k, v):
                    x[:, table[b][t // page], t % page] = x[:, table[b][f // page], f % page]
        return k, v, None
    if op != "beam":
        return None  # whole numbers
    k, v, refs = s["k_pages"].double(), s["v_pages"].double(), s["refs"].tolist()
    parents = s["parents"].tolist()
    old = [row[: _pages(a, page)] for row, a in zip(table, lens)]
    rows = [list(old[p]) for p in parents]
    lens = [lens[p] for p in parents]
    refs = [0] * len(refs)
    for row in rows:
        for p in row:
            refs[p] += 1
    plan = []
    for b, row in enumerate(rows):  # one row after another, the lowest free page first
        a = lens[b]
        if a % page and refs[row[a // page]] > 1:
            plan.append((b, a // page))
            refs[row[a // page]] -= 1
    free = [p for p, r in enumerate(refs) if r == 0]
    taken = 0
    copied = dict(plan)
    for b, row in enumerate(rows):
        a = lens[b]
        if b in copied:
            to, taken = free[taken], taken + 1
            for x in (k, v):
                x[:, to, : a % page] = x[:, row[a // page], : a % page]
            row[a // page] = to
        taken += _pages(a + s["grow"], page) - _pages(a, page)
    return None, None, None, None, None, k, v
