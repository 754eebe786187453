"""Eviction in every division of work: clusters of 8 and of 4 blocks to a row, one block to a row, rows that fill a
cluster's shared memory and rows that shared memory does not hold."""
import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm
from test_evict import check, i32, model, sums

pytestmark = pytest.mark.gpu


def cache(lens, page, Hkv, d, layers=None, seed=0):
    """Like pm.Setup, filled whole (a row at a time takes long for many places)."""
    s = pm.Setup([1] * len(lens), [0] * len(lens), page, Hkv, d, seed=seed, layers=layers)
    g = torch.Generator().manual_seed(seed)
    held = [pm.pages_of(n, page) for n in lens]
    order = torch.randperm(sum(held) + 2, generator=g).tolist()
    cols = max(held) + 1
    s.lens, s.table, s.num_pages = list(lens), [], sum(held) + 2
    for h in held:
        s.table.append([order.pop() for _ in range(h)] + [-1] * (cols - h))
    shape = (() if layers is None else (layers,)) + (s.num_pages, page, Hkv, d)
    s.k_pages, s.v_pages = (torch.randint(-(2**15), 2**15, shape, generator=g, dtype=torch.int16).view(torch.bfloat16).cuda()
                            for _ in range(2))
    s.t_lens, s.t_table, s.t_refs = i32(s.lens), i32(s.table), i32([1] * s.num_pages)
    return s


# lens, Hkv, layers, columns of sums, keep, recent
SHAPES = [
    # 20 to 38 rows with 4096 columns and more: clusters of 4
    ([5000, 4097, 100, 9000, 0], 4, None, 9003, 700, 64),
    ([5000, 4097, 100, 9000, 7777], 2, 2, 9001, 4096, 0),
    ([4500] * 19, 2, None, 4500, 4499, 4499),
    ([4100, 33] * 10, 1, None, 4100, 1, 1),
    ([196608] + [50] * 19, 1, None, 196608, 5000, 100),  # all that four blocks hold
    # up to 19 rows: clusters of 8
    ([4096, 4099, 5000], 3, 2, 5003, 2000, 50),
    ([4096] * 19, 1, None, 4096, 0, 0),
    ([393216], 1, None, 393216, 70000, 10),  # all that eight blocks hold
    # one block to a row: more rows, and more columns than clusters hold
    ([4200, 8193, 77] * 7, 2, None, 8193, 1500, 20),
    ([400000], 1, None, 400000, 30000, 64),
    ([300000, 20], 1, None, 393217, 299999, 299999),
    ([200000] + [60] * 19, 1, None, 200000, 100000, 0),
    # many short rows, above and below the small blocks' 8192 columns
    ([900, 1100, 40] * 13, 2, 2, 1101, 800, 60),
    ([900, 1100, 40] * 13, 2, 2, 8193, 800, 60),
]


@pytest.mark.parametrize("kind", ["many", "few", "odd", "same"])
@pytest.mark.parametrize("lens,Hkv,layers,places,keep,recent", SHAPES, ids=lambda x: None if isinstance(x, list) else str(x))
def test_every_division_of_work(lens, Hkv, layers, places, keep, recent, kind):
    s = cache(lens, 256 if max(lens) > 10000 else 64, Hkv, 64, layers, seed=keep)
    check(s, sums(s, places, recent, layers, kind), keep, recent)


def test_clusters_of_four_leave_alone_what_may_not_go():
    """The whole cluster of a row that stays gives up together: a place without a page, a shared page."""
    s = cache([5000, 4600, 9000, 4096, 60], 64, 4, 64, seed=5)
    s.table[1][70] = -1
    s.refs = [1] * s.num_pages
    s.refs[s.table[2][3]] = 2
    s.t_table, s.t_refs = i32(s.table), i32(s.refs)
    check(s, sums(s, 9000), 1000, 30, alone=(1, 2))


def test_clusters_of_four_replay():
    s = cache([5000, 4097, 100, 9000, 8000], 64, 4, 128, seed=6)
    w0, k0, v0 = sums(s, 9000), s.k_pages.clone(), s.v_pages.clone()
    want = model(s, w0, 2500, 100)
    w = w0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens, kept = fa.cache_evict(s.t_refs, s.k_pages, s.v_pages, s.t_table, s.t_lens, w, 2500, 100)
    for _ in range(3):
        w.copy_(w0), s.k_pages.copy_(k0), s.v_pages.copy_(v0)
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == want[3] and torch.equal(kept.cpu(), want[4]) and torch.equal(w.cpu(), want[2])
        assert torch.equal(s.k_pages.cpu().view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(s.v_pages.cpu().view(torch.int16), want[1].view(torch.int16))
