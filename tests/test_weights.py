"""Attention weight summed over the places of the paged cache, against a 64-bit form: single
tokens, chains and trees, ragged batches, every page size and head dim, more rows than one
tile, rows that see nothing, rubbish wherever a token must not look, and what the call must
leave alone."""
import math

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm

A = 0x10000
INV, UNS, ALI = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_ALIGNMENT


def reference(s, q, lse, weights, seen=None, decay=1.0, scale=None, k_pages=None):
    """64 bits, from the definition -> (weights, bound)."""
    k_pages = (s.k_pages if k_pages is None else k_pages).cpu().double()
    q, lse, out = q.cpu().double(), lse.cpu().double(), weights.cpu().double().clone()
    H, d = q.shape[1:]
    G = H // s.Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    bound = torch.zeros_like(out)
    for b in range(s.B):
        keys = min(s.lens[b] + s.new[b], out.shape[2])
        if s.new[b] == 0 or keys == 0:
            continue
        flat = [p * s.page + r if 0 <= p < k_pages.shape[0] else -1 for p, r in (s.place(b, pos) for pos in range(keys))]
        rows = slice(s.cu[b], s.cu[b + 1])
        see = torch.zeros((s.new[b], keys), dtype=torch.bool)
        for i in range(s.new[b]):
            for pos in range(keys):
                j = pos - s.lens[b]
                see[i, pos] = flat[pos] >= 0 and (j < 0 or (j <= i if seen is None else j in seen[s.cu[b] + i]))
        for h in range(s.Hkv):
            kk = k_pages.reshape(-1, s.Hkv, d)[[max(f, 0) for f in flat], h]
            qq = q[rows, h * G : (h + 1) * G]
            z, size = torch.einsum("igd,kd->gik", qq, kk) * scale, torch.einsum("igd,kd->gik", qq.abs(), kk.abs()) * scale
            l = lse[h * G : (h + 1) * G, rows, None]
            use = see[None] & ~torch.isneginf(l)
            p = torch.where(use, torch.exp(z - l), 0.0)
            # d products summed in fp32; the argument and what is rounded into it, each 2^-23 of their sizes; 2^x itself
            e = (d + 8) * 2.0**-24 * size + 2.0**-22 * (z.abs() + l.abs()) + 2.0**-20
            old = out[b, h, :keys]
            got = p.sum((0, 1))
            n = G * s.new[b]
            bound[b, h, :keys] = torch.where(use, p * e, 0.0).sum((0, 1)) * 1.01 + n * 2.0**-23 * got + 2.0**-23 * (
                (decay * old).abs() if decay else 0.0)
            out[b, h, :keys] = got + (decay * old if decay else 0.0)
    return out, bound + 2.0**-126


def check(s, got, ref, before, what=""):
    want, bound = ref
    off = (got.cpu().double() - want).abs()
    assert not (off > bound).any() and torch.isfinite(got[torch.isfinite(before)]).all(), (
        f"{what}: off by {float((off / bound).max()):.2f} of its bound, {int((off > bound).sum())} values, "
        f"first {(off > bound).nonzero()[:1].tolist()}")
    for b in range(s.B):  # behind the sequence, and sequences without new tokens: left as they were
        at = s.lens[b] + s.new[b] if s.new[b] else 0
        assert torch.equal(got[b, :, max(at, 0) :], before[b, :, max(at, 0) :]), f"{what}: sequence {b} past its end"


def run(s, max_new, mask=None, lse=None, extra=5, decay=1.0, places=None, **kw):
    g = torch.Generator(device="cuda").manual_seed(1)
    places = max([a + b for a, b in zip(s.lens, s.new)] + [1]) + extra if places is None else places
    w = torch.rand((s.B, s.Hkv, places), generator=g, device="cuda")
    before = w.clone()
    mask = None if mask is None else mask.cuda()
    if lse is None:
        _, lse = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, max_new, tree_mask=mask)
    out = fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, max_new, lse, w, tree_mask=mask,
                                     decay=decay, **kw)
    torch.cuda.synchronize()
    assert out is w and fa.fa_last_device_status() == fa.FA_OK
    return w, before, lse


# lens, new, page, H, Hkv, d
CASES = [
    ([1], [1], 16, 1, 1, 64),
    ([0], [1], 16, 2, 1, 128),
    ([15, 16, 17, 0, 300], [1, 1, 1, 1, 1], 16, 8, 2, 128),
    ([127, 128, 129, 255, 1], [1, 1, 1, 1, 1], 64, 8, 8, 64),
    ([63, 500, 64], [1, 1, 1], 32, 4, 4, 256),
    ([1000], [1], 128, 32, 8, 128),
    ([200, 31, 0, 77], [5, 0, 3, 1], 32, 16, 2, 128),
    ([200, 31, 0, 77], [16, 7, 33, 0], 16, 8, 4, 64),
    ([130, 250], [33, 64], 128, 8, 1, 128),
    ([130, 0, 250], [65, 1, 128], 64, 4, 2, 128),
    ([90, 700], [31, 7], 256, 6, 2, 256),
    ([513, 40], [9, 40], 64, 21, 3, 128),
    ([300], [3], 16, 71, 1, 64),
    ([129, 2], [2, 3], 64, 128, 1, 128),
    ([129, 2], [2, 3], 64, 128, 1, 256),
    ([60, 3], [256, 200], 32, 2, 1, 64),
    ([60, 3], [256, 131], 16, 4, 2, 256),
    ([5] * 40, [1, 2] * 20, 16, 2, 2, 64),
    ([600, 33], [90, 70], 256, 4, 2, 128),
    ([700, 300], [33, 31], 128, 20, 4, 256),
    ([40, 500, 90], [4, 2, 4], 16, 12, 3, 128),
    ([2] * 700, [1] * 700, 16, 2, 1, 64),
    ([500, 20], [256, 70], 32, 4, 1, 64),
    ([300, 290, 10], [1, 40, 130], 32, 4, 2, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("lens,new,page,H,Hkv,d", CASES)
def test_matches_64_bit_form(lens, new, page, H, Hkv, d, tree):
    s = pm.Setup(lens, new, page, Hkv, d, seed=sum(lens) + d + page, H=H)
    mask = seen = None
    if tree:
        mask, seen = pm.tree_masks(new, (max(new) + 63) // 64, seed=7 + d)
    for decay in (1.0, 0.0, 0.75)[: 1 if len(lens) > 9 else 3]:
        w, before, lse = run(s, max(new), mask, decay=decay)
        check(s, w, reference(s, s.q, lse, before, seen, decay), before, f"{lens[:5]} {new[:5]} page {page} H{H}/{Hkv} d{d} {decay}")


@pytest.mark.gpu
def test_weights_of_one_call_sum_to_its_rows():
    """Every row's weights sum to 1: each kv head's to the number of its rows."""
    s = pm.Setup([5000, 70], [20, 3], 64, 2, 128, seed=2, H=8)
    w, _, _ = run(s, 20, decay=0.0, extra=0)
    for b in range(2):
        total = w[b, :, : s.lens[b] + s.new[b]].double().sum(1).cpu()
        want = s.new[b] * 4
        assert ((total - want).abs() <= 1e-5 * want).all(), total


@pytest.mark.gpu
@pytest.mark.parametrize("d,H,Hkv,new", [(128, 4, 2, [3, 5]), (64, 2, 2, [70, 90]), (256, 16, 1, [2, 40])])
def test_rows_that_see_nothing(d, H, Hkv, new):
    s = pm.Setup([0, 0], new, 16, Hkv, d, seed=3, H=H)
    seen = [set() if t % 2 else {t % new[0]} for t in range(sum(new))]
    seen = [{j for j in x if j < n} for x, n in zip(seen, [new[0]] * new[0] + [new[1]] * new[1])]
    w, before, lse = run(s, max(new), pm.pack_masks(seen, (max(new) + 63) // 64))
    check(s, w, reference(s, s.q, lse, before, seen), before, "half the rows see nothing")


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("new,H,Hkv,d", [([6], 4, 2, 128), ([40], 8, 2, 64), ([100], 4, 2, 128), ([20], 8, 1, 256)])
def test_unseen_drafted_tokens_may_hold_anything(bad, new, H, Hkv, d):
    s = pm.Setup([37], new, 16, Hkv, d, seed=11, H=H)
    n = new[0]
    hidden = {2, n - 1}
    seen = [{j for j in range(i + 1) if j not in hidden} for i in range(n)]
    for j in hidden:
        p, r = s.place(0, 37 + j)
        s.k_pages[p, r], s.v_pages[p, r] = bad, bad
    clean = torch.nan_to_num(s.k_pages, nan=0.0, posinf=0.0, neginf=0.0)
    w, before, lse = run(s, n, pm.pack_masks(seen, (n + 63) // 64))
    check(s, w, reference(s, s.q, lse, before, seen, k_pages=clean), before, f"{bad} hidden")


@pytest.mark.gpu
@pytest.mark.parametrize("new,H,Hkv,d", [([1, 1], 8, 2, 128), ([3, 40], 8, 2, 64), ([100, 9], 4, 2, 128), ([20, 70], 8, 1, 256)])
def test_other_sequences_tokens_may_hold_anything(new, H, Hkv, d):
    s = pm.Setup([37, 300], new, 16, Hkv, d, seed=13, H=H)
    _, lse = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, max(new))
    want, before, _ = run(s, max(new), lse=lse)
    for b in range(2):
        q, l, keys = s.q.clone(), lse.clone(), s.k_pages.clone()
        rows = slice(s.cu[1 - b], s.cu[2 - b])
        s.q[rows], lse[:, rows] = float("nan"), float("inf")
        for c in range(pm.pages_of(s.lens[1 - b] + new[1 - b], 16)):
            s.k_pages[s.table[1 - b][c]] = float("nan")
        w, _, _ = run(s, max(new), lse=lse)
        assert torch.equal(w[b], want[b])
        s.q, lse, s.k_pages = q, l, keys


@pytest.mark.gpu
@pytest.mark.parametrize("new,H,Hkv,d,page", [([1], 8, 2, 128, 16), ([60], 8, 2, 64, 32), ([9], 4, 4, 256, 128)])
def test_places_without_a_page_get_nothing(new, H, Hkv, d, page):
    s = pm.Setup([5 * page + 3], new, page, Hkv, d, seed=5, H=H)
    for c, junk in ((1, -1), (3, s.num_pages), (0, 2**31 - 1)):
        s.table[0][c] = junk
    s.t_table = torch.tensor(s.table, dtype=torch.int32, device="cuda")
    w, before, lse = run(s, new[0], decay=0.5)
    check(s, w, reference(s, s.q, lse, before, decay=0.5), before, "dropped pages")


@pytest.mark.gpu
def test_fewer_columns_than_places_and_old_rubbish():
    s = pm.Setup([300, 10], [4, 3], 16, 2, 128, seed=6, H=4)
    w, before, lse = run(s, 4, places=133)
    check(s, w, reference(s, s.q, lse, before), before, "narrow")
    # decay 0 does not read what was there
    w = torch.full((2, 2, 133), float("nan"), device="cuda")
    fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, 4, lse, w, decay=0.0)
    zero = torch.zeros_like(w)
    fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, 4, lse, zero)
    for b in range(2):
        assert torch.equal(w[b, :, : s.lens[b] + s.new[b]], zero[b, :, : s.lens[b] + s.new[b]])
        assert torch.isnan(w[b, :, s.lens[b] + s.new[b] :]).all()


@pytest.mark.gpu
def test_lengths_and_offsets_outside_their_contract():
    s = pm.Setup([100, 40, 8], [3, 2, 4], 16, 2, 64, seed=8, H=4, fill=0.5)
    lse = torch.zeros((4, s.total), device="cuda")
    for lens in ([-5, 2**31 - 1, -(2**31)], [0, 0, 0], [2**30, 63, 1]):
        for cu in ([0, 3, 5, 9], [5, 0, 900, -4], [2**31 - 1, -(2**31), 3, 9]):
            store = torch.full((3 * 2 * 200 + 64,), 7.0, device="cuda")
            w = store[32:-32].view(3, 2, 200)
            fa.attention_weights_paged(s.q, s.k_pages, s.t_table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                       torch.tensor(cu, dtype=torch.int32, device="cuda"), 4, lse, w)
            torch.cuda.synchronize()
            assert fa.fa_last_device_status() == fa.FA_OK and (store[:32] == 7).all() and (store[-32:] == 7).all()


@pytest.mark.gpu
def test_repeatable_and_captured():
    s = pm.Setup([4000, 700, 0, 90], [9, 40, 0, 1], 32, 4, 128, seed=4, H=16)
    first, before, lse = run(s, 40)
    again, _, _ = run(s, 40, lse=lse)
    assert torch.equal(first, again)
    w = before.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, 40, lse, w)
    for _ in range(3):
        w.copy_(before)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(w, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w.copy_(before)
    torch.cuda.synchronize()
    fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, 40, lse, w, stream=side)
    side.synchronize()
    assert torch.equal(w, first)


# ------------------------------------------------------------------ refusals
@pytest.mark.parametrize("args,code", [
    (dict(q=None), INV), (dict(k_pages=None), INV), (dict(page_table=None), INV), (dict(cache_lens=None), INV),
    (dict(cu_seqlens=None), INV), (dict(lse=None), INV), (dict(weights=None), INV), (dict(places=0), INV), (dict(places=-1), INV),
    (dict(decay=-0.5), INV), (dict(decay=float("nan")), INV), (dict(decay=float("inf")), INV), (dict(scale=0.0), INV),
    (dict(scale=float("inf")), INV), (dict(H=3), INV), (dict(H=0), INV), (dict(Hkv=0), INV), (dict(H=258), UNS), (dict(d=96), UNS),
    (dict(max_new=0), INV), (dict(max_new=257), UNS), (dict(total=-1), INV), (dict(total=2**31 - 1), UNS), (dict(B=0), INV),
    (dict(B=65536), UNS), (dict(page_size=24), UNS), (dict(max_pages=1 << 27), UNS), (dict(q=A + 8), ALI), (dict(k_pages=A + 4), ALI),
    (dict(lse=A + 2), ALI), (dict(weights=A + 1), ALI), (dict(cu_seqlens=A + 2), ALI), (dict(tree_mask=A, mask_words=0), INV),
    (dict(tree_mask=A + 4, mask_words=1), ALI), (dict(B=65535, H=65535, Hkv=65535, num_pages=1, places=2**31 - 1), UNS)],
    ids=lambda x: str(x) if isinstance(x, dict) else None)
def test_refusals(args, code):
    a = dict(q=A, k_pages=A, page_table=A, cache_lens=A, cu_seqlens=A, tree_mask=None, mask_words=0, lse=A, weights=A, places=70,
             decay=1.0, B=2, max_pages=4, num_pages=9, page_size=16, max_new=3, total=5, H=4, Hkv=2, d=128, scale=0.1,
             stream=0) | args
    assert fa.fa_attention_weights_paged(**a) == code


def test_every_operand_is_checked():
    bf = lambda *x: torch.zeros(x, dtype=torch.bfloat16)
    i32 = lambda *x: torch.zeros(x, dtype=torch.int32)
    good = dict(q=bf(5, 4, 64), k_pages=bf(9, 16, 2, 64), page_table=i32(3, 4), cache_lens=i32(3), cu_seqlens=i32(4), max_new=3,
                lse=torch.zeros(4, 5), weights=torch.zeros(3, 2, 50), tree_mask=torch.zeros((5, 1), dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        fa.attention_weights_paged(**good)
    for name, x in good.items():
        if name == "max_new":
            continue
        wide = torch.zeros(x.shape[:-1] + (2 * x.shape[-1],), dtype=x.dtype)
        for bad in (x.double() if x.is_floating_point() else x.to(torch.int16), x[..., None], x[:-1], wide[..., ::2]):
            if name == "k_pages" and bad.shape == (8, 16, 2, 64):
                continue  # any number of pages
            with pytest.raises(ValueError, match="^(?!.*CUDA tensor)"):
                fa.attention_weights_paged(**(good | {name: bad}))
    with pytest.raises(ValueError, match="tree_mask"):
        fa.attention_weights_paged(**(good | dict(max_new=65)))
