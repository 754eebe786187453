"""Calls without work, on every way into the library: the ordinary call through the
binding, the call on a given stream, and the C entry point."""
import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm
from exact_attention_blackwell_gb300 import build as fa_build

A = 0x10000  # an aligned fake device address: never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()
    return fa.lib()


def test_c_append_of_no_rows_asks_for_none():
    a = dict(k=None, v=None, k_pages=A, v_pages=A, page_table=A, cache_lens=A, cu_seqlens=A, B=2, max_pages=4, num_pages=9,
             page_size=16, total=0, Hkv=2, d=128, stream=0)
    # FA_ERR_CUDA where there is no device to ask
    assert fa.fa_cache_append(**a) in (fa.FA_OK, fa.FA_ERR_CUDA)
    for bad, code in ((dict(k_pages=None), fa.FA_ERR_INVALID_ARG), (dict(page_size=24), fa.FA_ERR_UNSUPPORTED),
                      (dict(total=1), fa.FA_ERR_INVALID_ARG), (dict(total=-1), fa.FA_ERR_INVALID_ARG)):
        assert fa.fa_cache_append(**(a | bad)) == code


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(params=["ordinary", "stream"])
def where(request):
    return dict(stream=torch.cuda.Stream() if request.param == "stream" else None)


@pytest.mark.gpu
def test_append_of_no_rows(where):
    s = pm.Setup([10, 30], [0, 0], 16, 2, 64, seed=4, fill=3.0)
    before = s.k_pages.clone()
    none = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    fa.cache_append(none, none, s.k_pages, s.v_pages, s.t_table, s.t_lens, i32([0, 0, 0]), **where)
    torch.cuda.synchronize()
    assert torch.equal(s.k_pages, before)
    # nor with no sequences at all
    fa.cache_append(none, none, s.k_pages, s.v_pages, s.t_table[:0], s.t_lens[:0], i32([0]), **where)
    torch.cuda.synchronize()
    assert torch.equal(s.k_pages, before)


@pytest.mark.gpu
@pytest.mark.parametrize("layers", [None, 2])
def test_compact_of_no_tokens(where, layers):
    s = pm.Setup([10, 30], [4, 0], 16, 2, 64, seed=4, layers=layers, fill=3.0)
    k, v = s.k_pages.clone(), s.v_pages.clone()
    lens = i32([10, -4])
    path = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for counts in ([0, 0], [3, -1]):  # a path is no longer than its columns
        out = fa.cache_compact(s.k_pages, s.v_pages, s.t_table, lens, path, i32(counts), **where)
        torch.cuda.synchronize()
        assert out.tolist() == [10, -4] and out.dtype == torch.int32 and out.data_ptr() != lens.data_ptr()
    assert torch.equal(s.k_pages, k) and torch.equal(s.v_pages, v)


@pytest.mark.gpu
def test_attention_of_no_tokens(where):
    s = pm.Setup([10, 30], [0, 0], 16, 2, 64, seed=4, H=4)
    for mask in (None, torch.zeros((0, 1), dtype=torch.int64, device="cuda")):
        o, lse = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, 1, tree_mask=mask, **where)
        assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
        o, lse = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table[:0], s.t_lens[:0], s.t_cu[:1], 1, tree_mask=mask,
                                        **where)
        assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
