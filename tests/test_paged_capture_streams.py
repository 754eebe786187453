"""Captured steps whose kernels depend on work of several streams, and on copies and fills: a
kernel that may begin early still follows all of it."""
import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("new,H,Hkv,d", [(1, 8, 2, 128), (30, 8, 2, 128), (70, 4, 2, 64), (20, 4, 1, 256)])
def test_step_over_two_streams(new, H, Hkv, d):
    """Keys are appended on one stream, queries and lengths come from another, and the attention of two layers runs
    on both at once; then the accepted path is compacted behind both."""
    page, B, layers = 16, 5, 2
    s = pm.Setup([300, 0, 17, 95, 128], [new] * B, page, Hkv, d, seed=new, H=H, layers=layers)
    total = new * B
    src = [torch.zeros((layers, total, n, d), dtype=torch.bfloat16, device="cuda") for n in (H, Hkv, Hkv)]
    q, k, v = (torch.empty_like(x) for x in src)
    lens_src, lens = i32(s.lens), i32([0] * B)
    path, kept = i32([[0]] * B), i32([1] * B)
    big = torch.zeros(16 << 20, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        a.wait_stream(here), b.wait_stream(here)
        with torch.cuda.stream(b):
            big.add_(1)
            q.copy_(src[0])
            lens.copy_(lens_src)
        with torch.cuda.stream(a):
            k.copy_(src[1]), v.copy_(src[2])
            a.wait_stream(b)
            for layer in range(layers):
                fa.cache_append(k[layer], v[layer], s.k_pages[layer], s.v_pages[layer], s.t_table, lens, s.t_cu)
        b.wait_stream(a)
        out = []
        for layer, stream in ((0, a), (1, b)):
            with torch.cuda.stream(stream):
                out += fa.attention_fwd_paged(q[layer], s.k_pages[layer], s.v_pages[layer], s.t_table, lens, s.t_cu, new)
        here.wait_stream(a), here.wait_stream(b)
        out.append(fa.cache_compact(s.k_pages, s.v_pages, s.t_table, lens, path, kept))
        return out

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for x in src:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        lens_src.copy_(i32([(n * (seed + 1)) % (n + 1) for n in s.lens]))

    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(1, 6):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        want = step()
        torch.cuda.synchronize()
        assert fa.fa_last_device_status() == fa.FA_OK
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and len(got) == len(want)
        held = lens_src.tolist()
        for layer in range(layers):
            s.lens = held
            pm.check_attention(s, got[2 * layer], got[2 * layer + 1],
                               pm.attention(s, src[0][layer], None, k_pages=s.k_pages[layer], v_pages=s.v_pages[layer]),
                               f"layer {layer}")
        assert got[-1].tolist() == [n + 1 for n in held]


def test_calls_between_fills_and_copies():
    """Fills and copies of the tables between the calls, captured: each call reads what the one just before it set."""
    s = pm.Setup([40, 0, 17, 95], [3, 1, 2, 4], 16, 2, 128, seed=1, H=8)
    lens, refs = i32([0] * 4), s.t_refs.clone()
    want = [fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, x, s.t_cu, 4) for x in (s.t_lens, i32([0] * 4))]

    def step():
        out = []
        for _ in range(3):
            lens.copy_(s.t_lens)
            out.append(fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, lens, s.t_cu, 4))
            lens.zero_()
            out.append(fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, lens, s.t_cu, 4))
        refs.copy_(s.t_refs)
        lens.copy_(s.t_lens)
        table = s.t_table.clone()
        up = fa.cache_fork(refs, table, lens, i32_parents, 16)
        return out, up, refs.clone(), table

    i32_parents = i32([0, 0, 2, -1])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, up, counts, table = step()
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, lse) in enumerate(out):
            assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
        books, book_lens = list(s.refs), [40, 0, 17, 95]
        rows, new_lens = pm.fork([list(r) for r in s.table], book_lens, books, [0, 0, 2, -1], 16)
        assert up.tolist() == new_lens
        assert [r[: pm.pages_of(n, 16)] for r, n in zip(table.tolist(), new_lens)] == \
            [r[: pm.pages_of(n, 16)] for r, n in zip(rows, new_lens)]
