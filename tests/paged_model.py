"""A plain model of the paged cache for the tests: Python lists and 64-bit torch
arithmetic, written from the operators' definitions."""
from __future__ import annotations

import math

import numpy as np
import torch


def pages_of(n, page):
    return -(-n // page)


class Setup:
    """A random cache: pages scattered over the pool, every row that holds no place filled with `fill`
    (NaN by default), unused table entries naming no page."""

    def __init__(self, lens, new, page, Hkv, d, seed, H=None, layers=None, device="cuda", fill=float("nan"),
                 extra_cols=1, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.page, self.Hkv, self.d, self.B = list(lens), list(new), page, Hkv, d, len(lens)
        held = [pages_of(a + n, page) for a, n in zip(lens, new)]
        self.cols = max(max(held), 1) + extra_cols
        self.num_pages = sum(held) + spare
        order = torch.randperm(self.num_pages, generator=g).tolist()
        junk = [-1, -7, self.num_pages, self.num_pages + 100, 2**31 - 1, -(2**31)]
        self.table, at = [], 0
        for b, h in enumerate(held):
            self.table.append(order[at : at + h] + [junk[(b + c) % len(junk)] for c in range(self.cols - h)])
            at += h
        self.refs = [0] * self.num_pages
        for p in order[:at]:
            self.refs[p] = 1
        shape = (layers or 1, self.num_pages, page, Hkv, d)
        k = torch.full(shape, fill, dtype=torch.bfloat16)
        v = torch.full(shape, fill, dtype=torch.bfloat16)
        for b in range(self.B):
            for pos in range(lens[b] + new[b]):
                p, r = self.place(b, pos)
                k[:, p, r] = torch.randn((shape[0], Hkv, d), generator=g).to(torch.bfloat16)
                v[:, p, r] = torch.randn((shape[0], Hkv, d), generator=g).to(torch.bfloat16)
        if layers is None:
            k, v = k[0], v[0]
        self.k_pages, self.v_pages = k.to(device), v.to(device)
        self.total = sum(new)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)
        self.t_table, self.t_lens, self.t_cu, self.t_refs = i32(self.table), i32(self.lens), i32(self.cu), i32(self.refs)
        if H is not None:
            self.q = torch.randn((self.total, H, d), generator=g).to(torch.bfloat16).to(device)

    def place(self, b, pos):
        return self.table[b][pos // self.page], pos % self.page


def tree_masks(new, words, seed):
    """Random drafted trees -> (int64 [total, words], for each token the set of drafted tokens it sees)."""
    r = np.random.default_rng(seed)
    seen = []
    for n in new:
        mine = []
        for i in range(n):
            p = int(r.integers(-1, i)) if r.random() < 0.6 else i - 1
            mine.append((mine[p] if p >= 0 else set()) | {i})
        seen += mine
    return pack_masks(seen, words), seen


def pack_masks(seen, words):
    m = np.zeros((max(len(seen), 1), words), dtype=np.uint64)
    for t, s in enumerate(seen):
        for j in s:
            m[t, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return torch.from_numpy(m[: len(seen)].view(np.int64))


def attention(s: Setup, q, seen=None, scale=None, k_pages=None, v_pages=None):
    """64-bit attention from the definition -> (o, lse, attention of |v|, largest sum of |q_e k_e| * scale
    over the places each row sees), all on the CPU."""
    k_pages = s.k_pages if k_pages is None else k_pages
    v_pages = s.v_pages if v_pages is None else v_pages
    q, k_pages, v_pages = q.cpu().double(), k_pages.cpu().double(), v_pages.cpu().double()
    total, H, d = q.shape
    G = H // s.Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.zeros((total, H, d), dtype=torch.float64)
    mag, big = torch.zeros_like(o), torch.zeros((H, total), dtype=torch.float64)
    lse = torch.full((H, total), float("-inf"), dtype=torch.float64)
    for b in range(s.B):
        for i in range(s.new[b]):
            t = s.cu[b] + i
            vis = []
            for pos in range(s.lens[b] + s.new[b]):
                j = pos - s.lens[b]
                if j >= 0 and not (j <= i if seen is None else j in seen[t]):
                    continue
                p, r = s.place(b, pos)
                if 0 <= p < k_pages.shape[0]:
                    vis.append(p * s.page + r)
            if not vis:
                continue
            kk = k_pages.reshape(-1, s.Hkv, d)[vis].repeat_interleave(G, dim=1)  # [keys, H, d]
            vv = v_pages.reshape(-1, s.Hkv, d)[vis].repeat_interleave(G, dim=1)
            z = torch.einsum("hd,khd->hk", q[t], kk) * scale
            lse[:, t] = torch.logsumexp(z, dim=1)
            w = torch.exp(z - lse[:, t : t + 1])
            o[t] = torch.einsum("hk,khd->hd", w, vv)
            mag[t] = torch.einsum("hk,khd->hd", w, vv.abs())
            big[:, t] = (torch.einsum("hd,khd->hk", q[t].abs(), kk.abs()) * scale).amax(1)
    return o, lse, mag, big


def check_attention(s, o, lse, ref, what=""):
    """The bounds, from the roundings that the operator may make:
      scores: d products summed in fp32, then scaled: relative 2^-24 a step of the sum of magnitudes;
        2^x itself within 2^-21 with its argument's rounding (|argument| * 2^-23, below that sum);
      O: a score error e changes every weight by at most e^(2e) - 1 <= 2.1 e; the weights are rounded to bf16
        (2^-8 each), both times the attention of |v|; fp32 sums over n places, n * 2^-23; the result's own
        rounding to bf16, 2^-8 of it;
      LSE: the score error, the sum's n * 2^-23, and the logarithm's and its own rounding, 2^-22 of it."""
    o64, lse64, mag, big = ref
    o, lse = o.cpu().double(), lse.cpu().double()
    n = max([a + b for a, b in zip(s.lens, s.new)] + [1])
    e = (s.d + 8) * 2.0**-24 * big + 2.0**-21
    assert torch.equal(torch.isneginf(lse64), torch.isneginf(lse)), f"{what}: rows that see nothing"
    seen = ~torch.isneginf(lse64)
    assert torch.isfinite(o).all(), f"{what}: non-finite O"
    bound = 2.0**-8 * o64.abs() + (2.0**-8 * (1 + 2.0**-8) + 2.1 * e.T[..., None] + n * 2.0**-23) * mag
    bad = (o - o64).abs() > bound
    assert not bad.any(), (f"{what}: O off by {float((o - o64).abs()[bad].max()):.3e}, bound "
                           f"{float(bound[bad].min()):.3e}, {int(bad.sum())} values, first {bad.nonzero()[0].tolist()}")
    bound = e + n * 2.0**-23 + 2.0**-22 * lse64.abs() + 2.0**-22
    bad = ((lse - lse64).abs() > bound) & seen
    assert not bad.any(), (f"{what}: LSE off by {float((lse - lse64).abs()[bad].max()):.3e}, first "
                           f"{bad.nonzero()[0].tolist()}")


# ------------------------------------------------------------------ the books of the page table
def fork(table, lens, refs, parents, page):
    old = [row[: pages_of(n, page)] for row, n in zip(table, lens)]
    out = []
    for b, row in enumerate(table):
        p = parents[b]
        if p == b or not -1 <= p < len(table):
            out.append(list(row))
            continue
        for x in old[b]:
            refs[x] -= 1
        mine = old[p] if p >= 0 else []
        for x in mine:
            refs[x] += 1
        out.append(mine + [-1] * (len(row) - len(mine)))
    new_lens = [n if p == b or not -1 <= p < len(table) else (lens[p] if p >= 0 else 0)
                for b, (n, p) in enumerate(zip(lens, parents))]
    return out, new_lens


def resize(table, lens, refs, new_lens, page):
    """In place -> (lengths, [missing, refused], copies [(from, to, rows)])."""
    cap = len(table[0]) * page
    ok = [0 <= a <= cap and 0 <= n <= cap for a, n in zip(lens, new_lens)]
    for b, (a, n) in enumerate(zip(lens, new_lens)):
        if ok[b] and n < a:
            for c in range(pages_of(n, page), pages_of(a, page)):
                refs[table[b][c]] -= 1
                table[b][c] = -1
    free = sum(r == 0 for r in refs)
    trial, plan, need = list(refs), [], 0
    for b, (a, n) in enumerate(zip(lens, new_lens)):
        if not ok[b] or n <= a:
            continue
        copy = a % page != 0 and trial[table[b][a // page]] > 1
        if copy:
            trial[table[b][a // page]] -= 1
        plan.append((b, a, n, copy))
        need += copy + pages_of(n, page) - pages_of(a, page)
    out = [n if k and n <= a else a for a, n, k in zip(lens, new_lens, ok)]
    if need > free:
        return out, [need - free, ok.count(False)], []
    order = iter([p for p, r in enumerate(refs) if r == 0])
    copies = []
    for b, a, n, copy in plan:
        out[b] = n
        if copy:
            to, frm = next(order), table[b][a // page]
            copies.append((frm, to, a % page))
            refs[frm] -= 1
            refs[to] = 1
            table[b][a // page] = to
        for c in range(pages_of(a, page), pages_of(n, page)):
            table[b][c] = next(order)
            refs[table[b][c]] = 1
    return out, [0, ok.count(False)], copies
