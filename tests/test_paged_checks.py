"""Refusals of the paged cache's entry points, without a GPU: the C entry points
check before they launch, the torch helpers check before they call."""
import pytest
import torch

import exact_attention_blackwell_gb300 as fa
from exact_attention_blackwell_gb300 import build as fa_build

A = 0x10000  # an aligned fake device address: never dereferenced
INV, UNS, ALI, WS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_ALIGNMENT, fa.FA_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()
    return fa.lib()


TABLE = [
    (dict(B=0), INV), (dict(B=-1), INV), (dict(B=65536), UNS), (dict(max_pages=0), INV), (dict(num_pages=0), INV),
    (dict(page_size=0), INV), (dict(page_size=24), UNS), (dict(page_size=8), UNS), (dict(page_size=512), UNS),
    (dict(max_pages=1 << 27), UNS), (dict(page_table=None), INV), (dict(cache_lens=None), INV),
    (dict(page_table=A + 2), ALI), (dict(cache_lens=A + 1), ALI),
]
ROWS = [
    (dict(Hkv=0), INV), (dict(Hkv=65536), UNS), (dict(d=96), UNS), (dict(d=-64), INV), (dict(num_pages=1 << 30), UNS),
    (dict(k_pages=None), INV), (dict(v_pages=None), INV), (dict(k_pages=A + 8), ALI), (dict(v_pages=A + 4), ALI),
]


def ids(x):
    return str(x) if isinstance(x, dict) else None


@pytest.mark.parametrize("args,code", TABLE + ROWS + [
    (dict(k=None), INV), (dict(v=A + 8), ALI), (dict(cu_seqlens=None), INV), (dict(cu_seqlens=A + 2), ALI),
    (dict(total=-1), INV), (dict(total=2**31 - 1, Hkv=65535, num_pages=1), UNS)], ids=ids)
def test_append(args, code):
    a = dict(k=A, v=A, k_pages=A, v_pages=A, page_table=A, cache_lens=A, cu_seqlens=A, B=2, max_pages=4, num_pages=9,
             page_size=16, total=5, Hkv=2, d=128, stream=0) | args
    assert fa.fa_cache_append(**a) == code


@pytest.mark.parametrize("args,code", TABLE + ROWS + [
    (dict(q=None), INV), (dict(q=A + 2), ALI), (dict(o=None), INV), (dict(o=A + 8), ALI), (dict(lse=A + 2), ALI),
    (dict(cu_seqlens=None), INV), (dict(cu_seqlens=A + 2), ALI), (dict(H=0), INV), (dict(H=3), INV),
    (dict(H=65536), UNS), (dict(H=258), UNS), (dict(max_new=0), INV), (dict(max_new=257), UNS), (dict(total=-1), INV),
    (dict(total=2**31 - 1), UNS), (dict(scale=0.0), INV), (dict(scale=float("nan")), INV), (dict(scale=-1.0), INV),
    (dict(tree_mask=A, mask_words=0), INV), (dict(tree_mask=A, mask_words=1, max_new=65), INV),
    (dict(tree_mask=A + 4, mask_words=1), ALI), (dict(workspace=None), WS), (dict(workspace_bytes=0), WS),
    (dict(workspace=A + 16), WS)], ids=ids)
def test_attention(args, code):
    a = dict(q=A, k_pages=A, v_pages=A, page_table=A, cache_lens=A, cu_seqlens=A, tree_mask=None, mask_words=0, o=A,
             lse=None, B=2, max_pages=4, num_pages=9, page_size=16, max_new=3, total=5, H=4, Hkv=2, d=128, scale=0.1,
             workspace=A, workspace_bytes=1 << 40, stream=0) | args
    assert fa.fa_fwd_paged(**a) == code


@pytest.mark.parametrize("args", [dict(max_pages=1 << 26, num_pages=1, H=65535, Hkv=65535, d=64),  # tiles of a sequence
                                  dict(B=65535, num_pages=1, H=65535, Hkv=65535, d=64)], ids=ids)  # items
def test_attention_counts_work_in_31_bits(args):
    test_attention(args, UNS)


def test_resize_refuses_pools_past_2_to_30_pages():
    test_resize(dict(num_pages=(1 << 30) + 1, layers=1, Hkv=1, d=64), UNS)


def test_attention_workspace():
    assert fa.fa_fwd_paged_workspace_bytes(2, 1, 4, 2, 128) > 0
    for bad in ((0, 1, 4, 2, 128), (2, 0, 4, 2, 128), (2, 257, 4, 2, 128), (2, 1, 3, 2, 128), (2, 1, 4, 2, 96)):
        assert fa.fa_fwd_paged_workspace_bytes(*bad) == 0
    need = fa.fa_fwd_paged_workspace_bytes(2, 3, 4, 2, 128)
    assert fa.fa_fwd_paged(A, A, A, A, A, A, None, 0, A, None, 2, 4, 9, 16, 3, 5, 4, 2, 128, 0.1, A, need - 1, 0) == WS


@pytest.mark.parametrize("args,code", TABLE + ROWS + [
    (dict(layers=0), INV), (dict(layers=65536), UNS), (dict(accepted=None), INV), (dict(n_accepted=None), INV),
    (dict(lens_out=None), INV), (dict(accepted=A + 2), ALI), (dict(n_accepted=A + 2), ALI), (dict(lens_out=A + 6), ALI),
    (dict(max_accepted=0), INV), (dict(lens_out=A, cache_lens=A), INV), (dict(B=65535, layers=65535, num_pages=1, Hkv=1, d=64), UNS)],
    ids=ids)
def test_compact(args, code):
    a = dict(k_pages=A, v_pages=A, page_table=A, cache_lens=A, accepted=A, n_accepted=A, lens_out=A + 64, B=2,
             max_accepted=3, max_pages=4, num_pages=9, page_size=16, layers=2, Hkv=2, d=128, stream=0) | args
    assert fa.fa_cache_compact(**a) == code


@pytest.mark.parametrize("args,code", TABLE + [
    (dict(page_refs=None), INV), (dict(parents=None), INV), (dict(lens_out=None), INV), (dict(page_refs=A + 2), ALI),
    (dict(parents=A + 2), ALI), (dict(lens_out=A + 2), ALI), (dict(lens_out=A), INV), (dict(B=4097), UNS)], ids=ids)
def test_fork(args, code):
    a = dict(page_refs=A, page_table=A, cache_lens=A, parents=A, lens_out=A + 64, B=2, max_pages=4, num_pages=9,
             page_size=16, stream=0) | args
    assert fa.fa_cache_fork(**a) == code


@pytest.mark.parametrize("args,code", TABLE + ROWS + [
    (dict(page_refs=None), INV), (dict(new_lens=None), INV), (dict(lens_out=None), INV), (dict(status=None), INV),
    (dict(page_refs=A + 2), ALI), (dict(new_lens=A + 2), ALI), (dict(status=A + 2), ALI), (dict(layers=0), INV),
    (dict(lens_out=A), INV), (dict(B=4097), UNS), (dict(workspace=None), WS), (dict(workspace=A + 16), WS),
    (dict(workspace_bytes=27), WS)], ids=ids)
def test_resize(args, code):
    a = dict(page_refs=A, k_pages=A, v_pages=A, page_table=A, cache_lens=A, new_lens=A, lens_out=A + 64, status=A + 128,
             B=2, max_pages=4, num_pages=9, page_size=16, layers=2, Hkv=2, d=128, workspace=A, workspace_bytes=1 << 20,
             stream=0) | args
    assert fa.fa_cache_resize(**a) == code


def test_resize_workspace():
    assert fa.fa_cache_resize_workspace_bytes(0) == 0 and fa.fa_cache_resize_workspace_bytes(4097) == 0
    assert fa.fa_cache_resize_workspace_bytes(4096) >= (1 + 3 * 4096) * 4


# ------------------------------------------------------------------ torch helpers
def tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    return dict(q=bf(5, 4, 64), k=bf(5, 2, 64), v=bf(5, 2, 64), k_pages=bf(9, 16, 2, 64), v_pages=bf(9, 16, 2, 64),
                page_table=i32(3, 4), cache_lens=i32(3), cu_seqlens=i32(4), accepted=i32(3, 2), n_accepted=i32(3),
                page_refs=i32(9), parents=i32(3), new_lens=i32(3), tree_mask=torch.zeros((5, 1), dtype=torch.int64))


CALLS = {
    "append": lambda t: fa.cache_append(t["k"], t["v"], t["k_pages"], t["v_pages"], t["page_table"], t["cache_lens"],
                                        t["cu_seqlens"]),
    "attention": lambda t: fa.attention_fwd_paged(t["q"], t["k_pages"], t["v_pages"], t["page_table"], t["cache_lens"],
                                                  t["cu_seqlens"], 3, tree_mask=t["tree_mask"]),
    "compact": lambda t: fa.cache_compact(t["k_pages"], t["v_pages"], t["page_table"], t["cache_lens"], t["accepted"],
                                          t["n_accepted"]),
    "fork": lambda t: fa.cache_fork(t["page_refs"], t["page_table"], t["cache_lens"], t["parents"], 16),
    "resize": lambda t: fa.cache_resize(t["page_refs"], t["k_pages"], t["v_pages"], t["page_table"], t["cache_lens"],
                                        t["new_lens"]),
}
USED = {
    "append": ("k", "v", "k_pages", "v_pages", "page_table", "cache_lens", "cu_seqlens"),
    "attention": ("q", "k_pages", "v_pages", "page_table", "cache_lens", "cu_seqlens", "tree_mask"),
    "compact": ("k_pages", "v_pages", "page_table", "cache_lens", "accepted", "n_accepted"),
    "fork": ("page_refs", "page_table", "cache_lens", "parents"),
    "resize": ("page_refs", "k_pages", "v_pages", "page_table", "cache_lens", "new_lens"),
}


@pytest.mark.parametrize("op,name", [(o, n) for o, names in USED.items() for n in names])
def test_every_operand_is_checked(op, name):
    good = tensors()
    with pytest.raises(ValueError, match="CUDA"):
        CALLS[op](good)
    x = good[name]
    for bad in (x.double() if x.is_floating_point() else x.to(torch.int16),  # type
                x[..., None], x[:0], x[:-1],  # shape
                torch.zeros(x.shape[:-1] + (2 * x.shape[-1],), dtype=x.dtype)[..., ::2]):  # layout
        if bad.shape == x.shape and bad.is_contiguous() and bad.dtype == x.dtype:
            continue
        if (op, name) == ("fork", "page_refs") and bad.dim() == 1 and bad.dtype == x.dtype and bad.is_contiguous():
            continue  # its length is the number of pages, whatever it is
        with pytest.raises(ValueError, match="^(?!.*CUDA tensor)"):
            CALLS[op](tensors() | {name: bad})


def test_mask_words_follow_max_new():
    t = tensors()
    with pytest.raises(ValueError, match="tree_mask"):
        fa.attention_fwd_paged(t["q"], t["k_pages"], t["v_pages"], t["page_table"], t["cache_lens"], t["cu_seqlens"], 65,
                               tree_mask=t["tree_mask"])
    with pytest.raises(ValueError, match="lse"):
        fa.attention_fwd_paged(t["q"], t["k_pages"], t["v_pages"], t["page_table"], t["cache_lens"], t["cu_seqlens"], 3,
                               lse=torch.zeros((4, 4)))
