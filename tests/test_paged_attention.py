"""Attention of new tokens over the paged cache, against a 64-bit plain form:
single tokens, chains and drafted trees, ragged batches, every page size and head
dim, rows that see nothing, and rubbish wherever a token must not look."""
import math

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm

pytestmark = pytest.mark.gpu


def run(s, max_new, mask=None, **kw):
    o, lse = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, max_new,
                                    tree_mask=None if mask is None else mask.cuda(), **kw)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    return o, lse


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
    ([60, 3], [256, 200], 32, 2, 1, 64),
    ([60, 3], [256, 131], 16, 4, 2, 256),
    ([5] * 40, [1, 2] * 20, 16, 2, 2, 64),
    ([600, 33], [90, 70], 256, 4, 2, 128),
    ([200, 15], [140, 150], 16, 2, 2, 128),
    ([700, 300], [33, 31], 128, 20, 4, 256),
    ([40, 500, 90], [4, 2, 4], 16, 12, 3, 128),
    ([40, 500, 90], [2, 2, 1], 32, 12, 2, 256),
]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("lens,new,page,H,Hkv,d", CASES)
def test_matches_64_bit_form(lens, new, page, H, Hkv, d, tree):
    s = pm.Setup(lens, new, page, Hkv, d, seed=sum(lens) + d + page, H=H)
    mask = seen = None
    if tree:
        mask, seen = pm.tree_masks(new, (max(new) + 63) // 64, seed=7 + d)
    o, lse = run(s, max(new), mask)
    pm.check_attention(s, o, lse, pm.attention(s, s.q, seen), f"{lens} {new} page {page} H{H}/{Hkv} d{d} tree={tree}")


@pytest.mark.parametrize("d,H,Hkv,new", [(128, 4, 2, [3, 5]), (64, 2, 2, [70, 90]), (256, 16, 1, [2, 40])])
def test_rows_that_see_nothing(d, H, Hkv, new):
    s = pm.Setup([0, 0], new, 16, Hkv, d, seed=3, H=H)
    seen = [set() if t % 2 else {t % new[0]} for t in range(sum(new))]
    seen = [{j for j in x if j < n} for x, n in zip(seen, [new[0]] * new[0] + [new[1]] * new[1])]
    o, lse = run(s, max(new), pm.pack_masks(seen, (max(new) + 63) // 64))
    assert (o[1::2] == 0).all() and torch.isneginf(lse[:, 1::2]).all()
    pm.check_attention(s, o, lse, pm.attention(s, s.q, seen), "half the rows see nothing")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("new,H,Hkv,d", [([6], 4, 2, 128), ([40], 8, 2, 64), ([100], 4, 2, 128), ([20], 8, 1, 256)])
def test_unseen_drafted_tokens_may_hold_anything(bad, new, H, Hkv, d):
    s = pm.Setup([37], new, 16, Hkv, d, seed=11, H=H)
    n = new[0]
    hidden = {2, n - 1}
    seen = [{j for j in range(i + 1) if j not in hidden} for i in range(n)]
    clean_k, clean_v = s.k_pages.clone(), s.v_pages.clone()
    for j in hidden:
        p, r = s.place(0, 37 + j)
        s.k_pages[p, r], s.v_pages[p, r] = bad, bad
    o, lse = run(s, n, pm.pack_masks(seen, (n + 63) // 64))
    pm.check_attention(s, o, lse, pm.attention(s, s.q, seen, k_pages=clean_k, v_pages=clean_v), f"{bad} hidden")


@pytest.mark.parametrize("new,H,Hkv,d", [([6], 4, 2, 128), ([100], 4, 2, 128), ([20], 8, 1, 256)])
def test_non_finite_values_reach_only_the_tokens_that_see_them(new, H, Hkv, d):
    s = pm.Setup([37], new, 16, Hkv, d, seed=12, H=H)
    n = new[0]
    clean = s.v_pages.clone()
    p, r = s.place(0, 37 + 3)
    s.v_pages[p, r, 0, 5], s.v_pages[p, r, 0, 6] = float("inf"), float("nan")
    o, lse = run(s, n)
    ref = pm.attention(s, s.q, None, v_pages=clean)
    G = H // Hkv
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[3:, :G, 5:7] = True
    assert torch.isposinf(o[3:, :G, 5]).all() and torch.isnan(o[3:, :G, 6]).all()
    o = torch.where(hit, ref[0].to(o.device, o.dtype), o)
    pm.check_attention(s, o, lse, ref, "the others")


@pytest.mark.parametrize("new,H,Hkv,d,page", [([1], 8, 2, 128, 16), ([60], 8, 2, 64, 32), ([9], 4, 4, 256, 128)])
def test_entries_that_name_no_page_are_not_seen(new, H, Hkv, d, page):
    s = pm.Setup([5 * page + 3], new, page, Hkv, d, seed=5, H=H)
    for c, junk in ((1, -1), (3, s.num_pages), (0, 2**31 - 1)):
        s.table[0][c] = junk
    s.t_table = torch.tensor(s.table, dtype=torch.int32, device="cuda")
    o, lse = run(s, new[0])
    pm.check_attention(s, o, lse, pm.attention(s, s.q), "dropped pages")


def test_a_table_too_narrow_for_the_lengths_sees_what_it_holds():
    s = pm.Setup([100], [4], 16, 2, 128, seed=6, H=4)
    narrow = s.t_table[:, :5].contiguous()
    o, lse = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, narrow, s.t_lens, s.t_cu, 4)
    s.table[0] = s.table[0][:5] + [-1] * 10
    pm.check_attention(s, o, lse, pm.attention(s, s.q), "narrow table")


def test_large_scores_and_a_given_scale():
    s = pm.Setup([400, 90], [3, 40], 64, 2, 128, seed=8, H=8)
    s.q *= 20
    s.k_pages[:, ::7] *= 20
    o, lse = run(s, 40, scale=0.31)
    pm.check_attention(s, o, lse, pm.attention(s, s.q, scale=0.31), "outliers")


def test_rows_of_no_sequence_and_past_max_new_are_left_alone():
    s = pm.Setup([20, 30], [4, 6], 16, 2, 128, seed=9, H=4)
    o = torch.full((10, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 10), 7.0, device="cuda")
    cu = torch.tensor([1, 4, 8], dtype=torch.int32, device="cuda")  # rows 0, 8, 9 belong to nobody
    fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, cu, 3, out=o, lse=lse)
    torch.cuda.synchronize()
    for t in (0, 7, 8, 9):  # row 7 is the fourth new token of a call that allows three
        assert (o[t] == 7).all() and (lse[:, t] == 7).all(), t
    s.new, s.cu = [3, 3], [1, 4, 7]
    ref = pm.attention(s, s.q)
    keep = [1, 2, 3, 4, 5, 6]
    s2 = s
    pm.check_attention(s2, o[keep], lse[:, keep], tuple(x[keep] if x.dim() == 3 else x[:, keep] for x in ref), "the rest")


@pytest.mark.parametrize("B,new_of,H,Hkv,d", [(700, lambda b: 1, 2, 2, 64), (1500, lambda b: 3 if b % 97 == 5 else 0, 4, 4, 128),
                                              (400, lambda b: b % 23, 4, 1, 128), (1000, lambda b: 40 if b == 999 else 0, 4, 1, 64),
                                              (370, lambda b: 70 if b % 9 == 0 else 1, 2, 1, 128)])
def test_many_sequences(B, new_of, H, Hkv, d):
    """More sequences than a block has threads, most of them without new tokens."""
    s = pm.Setup([(7 * b) % 90 for b in range(B)], [new_of(b) for b in range(B)], 16, Hkv, d, seed=B, H=H)
    o, lse = run(s, max(s.new))
    pm.check_attention(s, o, lse, pm.attention(s, s.q), f"B {B}")


def test_max_new_may_be_larger_than_any_sequence_has():
    s = pm.Setup([200, 31, 0, 77], [5, 0, 3, 1], 32, 2, 128, seed=4, H=4)
    ref = pm.attention(s, s.q)
    for most in (5, 8, 9, 17, 64, 65, 256):
        o, lse = run(s, most)
        pm.check_attention(s, o, lse, ref, f"max_new {most}")
        mask, seen = pm.tree_masks(s.new, (most + 63) // 64, seed=most)
        o, lse = run(s, most, mask)
        pm.check_attention(s, o, lse, pm.attention(s, s.q, seen), f"max_new {most}, trees")


def test_empty_batch():
    s = pm.Setup([20, 30], [0, 0], 16, 2, 128, seed=9, H=4)
    o, lse = run(s, 1)
    assert o.shape == (0, 4, 128) and lse.shape == (4, 0)


def test_long_cache_with_offsets_past_32_bits():
    # pages past element 2^31 and byte 2^32 of the pool
    page, Hkv, d = 256, 16, 128
    num_pages = 2**31 // (page * Hkv * d) + 40
    k = torch.zeros((num_pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    lens, n = [3000], 2
    table = torch.tensor([[num_pages - 1 - 3 * c for c in range(12)]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = table[0].long()
    k[ids] = torch.randn((12, page, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    v[ids] = torch.randn((12, page, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((n, 16, d), generator=g, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    o, lse = fa.attention_fwd_paged(q, k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, n)
    kk = k[ids].reshape(-1, Hkv, d)[: 3000 + n].double()
    vv = v[ids].reshape(-1, Hkv, d)[: 3000 + n].double()
    z = torch.einsum("thd,khd->htk", q.double(), kk) / math.sqrt(d)
    z[:, 0, 3001] = float("-inf")
    norm = torch.logsumexp(z, -1)
    w = torch.exp(z - norm[..., None])
    s = pm.Setup([0], [0], page, 1, d, seed=1)
    s.lens, s.new, s.d = lens, [n], d
    big = (torch.einsum("thd,khd->htk", q.double().abs(), kk.abs()) / math.sqrt(d)).amax(-1)
    pm.check_attention(s, o, lse, (torch.einsum("htk,khd->thd", w, vv).cpu(), norm.cpu(),
                                   torch.einsum("htk,khd->thd", w, vv.abs()).cpu(), big.cpu()), "far pages")


@pytest.mark.parametrize("lens,new,H,Hkv,d,page", [([20000], [1], 8, 2, 128, 64), ([9001, 17], [50, 3], 8, 2, 128, 32),
                                                   ([7000] * 3, [1] * 3, 4, 4, 64, 128), ([6001], [33], 8, 1, 256, 64),
                                                   ([4095, 0, 4096, 1, 12345], [1, 4, 2, 3, 7], 16, 4, 128, 256)])
def test_long_caches(lens, new, H, Hkv, d, page):
    B = len(lens)
    g = torch.Generator(device="cuda").manual_seed(d + H)
    held = [pm.pages_of(a + n, page) for a, n in zip(lens, new)]
    num = sum(held)
    k = torch.randn((num, page, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn((num, page, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(held)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at : at + h]
        at += h
    q = torch.randn((sum(new), H, d), generator=g, device="cuda").to(torch.bfloat16)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    o, lse = fa.attention_fwd_paged(q, k, v, table, i32(lens), i32(cu), max(new))
    again, lse2 = fa.attention_fwd_paged(q, k, v, table, i32(lens), i32(cu), max(new))
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    assert fa.fa_last_device_status() == fa.FA_OK
    for b in range(B):
        ids = table[b, : held[b]].long()
        keys = lens[b] + new[b]
        kk = k[ids].reshape(-1, Hkv, d)[:keys].double().repeat_interleave(H // Hkv, 1)
        vv = v[ids].reshape(-1, Hkv, d)[:keys].double().repeat_interleave(H // Hkv, 1)
        qq = q[cu[b] : cu[b + 1]].double()
        z = torch.einsum("thd,khd->htk", qq, kk) / math.sqrt(d)
        hide = torch.arange(keys, device="cuda")[None] > lens[b] + torch.arange(new[b], device="cuda")[:, None]
        z.masked_fill_(hide[None], float("-inf"))
        norm = torch.logsumexp(z, -1)
        w = torch.exp(z - norm[..., None])
        big = (torch.einsum("thd,khd->htk", qq.abs(), kk.abs()) / math.sqrt(d)).amax(-1)
        s = pm.Setup([0], [0], page, 1, d, seed=1)
        s.lens, s.new = [lens[b]], [new[b]]
        pm.check_attention(s, o[cu[b] : cu[b + 1]], lse[:, cu[b] : cu[b + 1]],
                           (torch.einsum("htk,khd->thd", w, vv).cpu(), norm.cpu(),
                            torch.einsum("htk,khd->thd", w, vv.abs()).cpu(), big.cpu()), f"sequence {b}")
