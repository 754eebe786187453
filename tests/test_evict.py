"""A paged cache cut down to a budget, against a plain model: ties, values that are not
finite, every budget from none to all, rows that are left alone, pages that end inside what
moves, long rows, layers, and what follows the call."""
import math

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm

A = 0x10000
INV, UNS, ALI = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_ALIGNMENT


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(x):
    return x.view(torch.int16)


def order(w, older, stay):
    """The places that stay of the first `older`, by definition."""
    value = [(-math.inf if math.isnan(x) else x, not math.isnan(x)) for x in w[:older].tolist()]
    best = sorted(range(older), key=lambda p: (-value[p][0], not value[p][1], p))
    return sorted(best[:stay])


def model(s, weights, keep, recent, alone=()):
    """-> k, v, weights, lens, kept, all on the CPU."""
    layered = s.k_pages.dim() == 5
    k, v, w = s.k_pages.cpu().clone(), s.v_pages.cpu().clone(), weights.cpu().clone()
    if not layered:
        k, v, w = k[None], v[None], w[None]
    L = k.shape[0]
    kept = torch.full((L, s.B, s.Hkv, keep), -1, dtype=torch.int32)
    lens = list(s.lens)
    for b in range(s.B):
        a = s.lens[b]
        if a <= keep or a > w.shape[-1] or b in alone:
            n = max(min(a, keep), 0)
            kept[:, b, :, :n] = torch.arange(n, dtype=torch.int32)
            continue
        lens[b] = keep
        at = torch.tensor([s.place(b, p)[0] * s.page + s.place(b, p)[1] for p in range(a)], dtype=torch.long)
        for l in range(L):
            for h in range(s.Hkv):
                stay = order(w[l, b, h], a - recent, keep - recent) + list(range(a - recent, a))
                kept[l, b, h] = torch.tensor(stay, dtype=torch.int32)
                for x in (k, v):
                    flat = x[l].view(-1, s.Hkv, s.d)
                    flat[at[:keep], h] = flat[at[stay], h].clone()
                new = w[l, b, h].clone()
                new[:a] = 0
                new[:keep] = w[l, b, h, stay]
                w[l, b, h] = new
    return (k, v, w, lens, kept) if layered else (k[0], v[0], w[0], lens, kept[0])


def sums(s, places, seed=0, layers=None, kind="many"):
    g = torch.Generator().manual_seed(seed)
    shape = (layers,) * (layers is not None) + (s.B, s.Hkv, places)
    if kind == "same":
        return torch.full(shape, 0.25).cuda()
    w = torch.exp(3 * torch.randn(shape, generator=g)).to(torch.bfloat16).float()
    if kind == "few":
        w = torch.randint(0, 3, shape, generator=g).float()
    if kind == "odd":
        pick = torch.randint(0, 8, shape, generator=g)
        w = w * (torch.randint(0, 2, shape, generator=g) * 2 - 1)
        for i, x in enumerate((math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-42)):
            w[pick == i] = x
        w[..., 3] = -torch.tensor(math.nan)
    return w.cuda()


def check(s, w, keep, recent, alone=(), table=None):
    want = model(s, w, keep, recent, alone)
    got_w = w.clone()
    lens, kept = fa.cache_evict(s.t_refs, s.k_pages, s.v_pages, s.t_table if table is None else table, s.t_lens, got_w, keep, recent)
    torch.cuda.synchronize()
    assert lens.tolist() == want[3]
    assert torch.equal(kept.cpu(), want[4]), (kept.cpu() != want[4]).nonzero()[:3]
    assert torch.equal(got_w.cpu().view(torch.int32), want[2].view(torch.int32))
    assert torch.equal(bits(s.k_pages.cpu()), bits(want[0])) and torch.equal(bits(s.v_pages.cpu()), bits(want[1]))


# lens, page, Hkv, d, layers, keep, recent
CASES = [
    ([5], 16, 1, 64, None, 3, 0),
    ([5], 16, 1, 64, None, 0, 0),
    ([2, 1, 0], 16, 2, 128, None, 1, 1),
    ([100, 33, 0, 64, 65], 16, 2, 128, None, 64, 16),
    ([100, 33, 0, 64, 65], 16, 3, 64, 2, 64, 64),
    ([100, 33, 0, 64, 65], 32, 2, 256, 3, 1, 0),
    ([300, 299, 17], 64, 2, 128, 2, 299, 31),
    ([700], 256, 8, 64, None, 33, 5),
    ([1500, 1100], 16, 1, 256, None, 1024, 100),
    ([1025, 2049, 40], 128, 2, 64, 2, 1000, 0),
    ([3000], 16, 2, 64, None, 2999, 2998),
    ([40] * 30, 16, 1, 64, 2, 39, 7),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["many", "few", "odd"])
@pytest.mark.parametrize("lens,page,Hkv,d,layers,keep,recent", CASES)
def test_matches_the_model(lens, page, Hkv, d, layers, keep, recent, kind):
    s = pm.Setup(lens, [0] * len(lens), page, Hkv, d, seed=keep + d, layers=layers)
    check(s, sums(s, max(lens) + 3, keep, layers, kind), keep, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["same", "few", "many"])
@pytest.mark.parametrize("length,keep,recent", [(40000, 3000, 64), (33000, 32999, 0), (70000, 1, 0), (66000, 40000, 20000)])
def test_long_rows(length, keep, recent, kind):
    s = pm.Setup([1], [0], 256, 2, 64, seed=1)
    g = torch.Generator().manual_seed(3)
    pages = pm.pages_of(length, 256)
    s.lens, s.table = [length], [torch.randperm(pages, generator=g).tolist()]
    s.k_pages, s.v_pages = (torch.randn((pages, 256, 2, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    s.t_lens, s.t_table, s.t_refs = i32(s.lens), i32(s.table), i32([1] * pages)
    check(s, sums(s, length, 7, kind=kind), keep, recent)


@pytest.mark.gpu
def test_rows_that_are_left_alone():
    """Shorter than the budget, longer than the sums or the table, without a page, sharing a page that would be
    written; a page that is shared but only read from is no hindrance."""
    s = pm.Setup([100, 100, 100, 100, 20, 100, -3], [0] * 7, 16, 2, 64, seed=9, fill=0.25)
    s.table[1][2] = -1  # a place without a page
    s.table[2][6] = s.num_pages
    s.refs[s.table[3][1]] = 2  # shared and written
    s.refs[s.table[5][5]] = 3  # shared and only read: places 80 on
    s.t_table, s.t_refs = i32(s.table), i32(s.refs)
    w = sums(s, 100)
    check(s, w, 40, 8, alone=(1, 2, 3, 6))
    s = pm.Setup([100, 90], [0, 0], 16, 2, 64, seed=9)
    check(s, sums(s, 95), 40, 8)  # the first has more places than sums
    s = pm.Setup([100, 90], [0, 0], 16, 2, 64, seed=9)
    check(s, sums(s, 100), 40, 8, alone=(0,), table=s.t_table[:, :6].contiguous())


@pytest.mark.gpu
def test_budgets_past_every_length():
    s = pm.Setup([100, 7], [0, 0], 16, 2, 64, seed=9)
    check(s, sums(s, 100), 5000, 4000)
    s.t_lens = i32([2**31 - 1, -(2**31)])
    w = sums(s, 100)
    lens, kept = fa.cache_evict(s.t_refs, s.k_pages, s.v_pages, s.t_table, s.t_lens, w.clone(), 50, 3)
    assert lens.tolist() == [2**31 - 1, -(2**31)] and kept[0, 0].tolist() == list(range(50)) and (kept[1] == -1).all()


@pytest.mark.gpu
def test_captured_on_a_stream_and_twice():
    s = pm.Setup([900, 333], [0, 0], 32, 4, 128, seed=5, layers=2)
    w0, k0, v0 = sums(s, 900, layers=2), s.k_pages.clone(), s.v_pages.clone()
    want = model(s, w0, 300, 20)
    w = w0.clone()

    def same(lens, kept):
        torch.cuda.synchronize()
        return (lens.tolist() == want[3] and torch.equal(kept.cpu(), want[4]) and torch.equal(w.cpu(), want[2])
                and torch.equal(bits(s.k_pages.cpu()), bits(want[0])) and torch.equal(bits(s.v_pages.cpu()), bits(want[1])))

    def reset():
        w.copy_(w0), s.k_pages.copy_(k0), s.v_pages.copy_(v0)
        torch.cuda.synchronize()

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens, kept = fa.cache_evict(s.t_refs, s.k_pages, s.v_pages, s.t_table, s.t_lens, w, 300, 20)
    for _ in range(3):
        reset()
        graph.replay()
        assert same(lens, kept)
    side = torch.cuda.Stream()
    reset()
    assert same(*fa.cache_evict(s.t_refs, s.k_pages, s.v_pages, s.t_table, s.t_lens, w, 300, 20, stream=side))
    # the second call finds nothing to do
    k, v = s.k_pages.clone(), s.v_pages.clone()
    again, kept = fa.cache_evict(s.t_refs, s.k_pages, s.v_pages, s.t_table, lens, w, 300, 20)
    assert again.tolist() == lens.tolist() and torch.equal(bits(k), bits(s.k_pages)) and torch.equal(bits(v), bits(s.v_pages))
    assert (kept == torch.arange(300, dtype=torch.int32, device="cuda")).all()


# ------------------------------------------------------------------ refusals
@pytest.mark.parametrize("args,code", [
    (dict(page_refs=None), INV), (dict(k_pages=None), INV), (dict(v_pages=None), INV), (dict(page_table=None), INV),
    (dict(cache_lens=None), INV), (dict(weights=None), INV), (dict(lens_out=None), INV), (dict(kept=None), INV),
    (dict(lens_out=A), INV), (dict(places=0), INV), (dict(keep=-1), INV), (dict(recent=-1), INV), (dict(recent=4), INV),
    (dict(B=0), INV), (dict(B=65536), UNS), (dict(page_size=24), UNS), (dict(layers=0), INV), (dict(layers=65536), UNS),
    (dict(Hkv=0), INV), (dict(d=96), UNS), (dict(max_pages=1 << 27), UNS), (dict(k_pages=A + 8), ALI), (dict(v_pages=A + 4), ALI),
    (dict(v_pages=A), INV), (dict(page_refs=A + 2), ALI), (dict(weights=A + 1), ALI), (dict(lens_out=A + 66), ALI), (dict(kept=A + 2), ALI),
    (dict(B=65535, layers=65535, num_pages=1), UNS), (dict(B=65535, Hkv=1000, num_pages=1, places=2**31 - 1), UNS),
    (dict(B=65535, Hkv=1000, num_pages=1, keep=2**31 - 1), UNS)], ids=lambda x: str(x) if isinstance(x, dict) else None)
def test_refusals(args, code):
    a = dict(page_refs=A, k_pages=A, v_pages=A + 4096, page_table=A, cache_lens=A, weights=A, places=70, keep=3, recent=1, lens_out=A + 64,
             kept=A, B=2, max_pages=4, num_pages=9, page_size=16, layers=2, Hkv=2, d=128, stream=0) | args
    assert fa.fa_cache_evict(**a) == code


@pytest.mark.parametrize("layers", [None, 2])
def test_every_operand_is_checked(layers):
    lead = () if layers is None else (layers,)
    bf = lambda *x: torch.zeros(x, dtype=torch.bfloat16)
    n = lambda *x: torch.zeros(x, dtype=torch.int32)
    good = dict(page_refs=n(9), k_pages=bf(*lead, 9, 16, 2, 64), v_pages=bf(*lead, 9, 16, 2, 64), page_table=n(3, 4), cache_lens=n(3),
                weights=torch.zeros((*lead, 3, 2, 50)), keep=5, recent=2)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_evict(**good)
    for name, x in good.items():
        if name in ("keep", "recent"):
            continue
        wide = torch.zeros(x.shape[:-1] + (2 * x.shape[-1],), dtype=x.dtype)
        for bad in (x.double() if x.is_floating_point() else x.to(torch.int16), x[..., None], x[:-1], wide[..., ::2]):
            with pytest.raises(ValueError, match="^(?!.*CUDA tensor)"):
                fa.cache_evict(**(good | {name: bad}))
    for bad in (dict(keep=-1, recent=-1), dict(recent=6), dict(recent=-1), dict(keep=2**31)):
        with pytest.raises(ValueError):
            fa.cache_evict(**(good | bad))
