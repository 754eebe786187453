"""Kernels of the paged cache begin while the kernel before them still runs; none may read
what that one has yet to write, at once or through a pointer that promises constant
contents."""
import os
import random
import re

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm

CSRC = os.path.join(os.path.dirname(fa.__file__), "csrc")


@pytest.mark.parametrize("source", ["fa_cache.cu", "fa_paged.cu"])
def test_early_kernels_promise_no_constant_contents(source):
    text = open(os.path.join(CSRC, source)).read()
    kernels = re.findall(r"__global__[^;{]*?(\w+_kernel)\(([^{]*?)\)\s*\{", text)
    assert len(kernels) >= 3, kernels
    for name, params in kernels:
        assert "__restrict__" not in params, f"{name} reads what an earlier kernel may still be writing"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(x):
    return x.view(torch.int16)


@pytest.mark.gpu
@pytest.mark.parametrize("B,page,layers,Hkv,d,seed", [(1, 16, 2, 1, 64, 0), (24, 16, 12, 4, 128, 1), (64, 64, 6, 8, 64, 2),
                                                      (200, 16, 1, 2, 256, 3)])
def test_fork_and_resize_follow_one_another_without_waiting(B, page, layers, Hkv, d, seed):
    """Rows are shared, grown (with copies of the last pages), shrunk and emptied, each call on the results of
    the one before and nothing between the launches."""
    r = random.Random(seed)
    cols = 6
    num = B * cols + 4
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (layers, num, page, Hkv, d)
    k0, v0 = (torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    want_k, want_v = k0.clone(), v0.clone()
    table, lens, refs = [[-1] * cols for _ in range(B)], [0] * B, [0] * num
    steps, copied = [], 0
    for i in range(10):
        if i % 2:
            parents = [r.choice([b, r.randrange(B), r.randrange(B), b ^ 1 if b ^ 1 < B else 0, -1 if i == 7 else b])
                       for b in range(B)]
            table, lens = pm.fork(table, lens, refs, parents, page)
            steps.append(("fork", i32(parents)))
        new = [r.choice([n, min(n + r.randint(1, page), cols * page), r.randint(0, n) if i % 3 == 2 else n + (n % page != 0)])
               for n in lens]
        if i == 0:
            new = [r.randint(1, 3 * page) for _ in range(B)]
        lens, said, copies = pm.resize(table, lens, refs, new, page)
        assert said == [0, 0]
        copied += len(copies)
        for f, t, m in copies:
            want_k[:, t, :m], want_v[:, t, :m] = want_k[:, f, :m], want_v[:, f, :m]
        steps.append(("resize", i32(new)))
    assert copied > 0 or B == 1
    k, v = k0.clone(), v0.clone()
    t_table, t_refs, zero = i32([[-1] * cols] * B), i32([0] * num), i32([0] * B)

    def play():
        said, n = [], zero
        for what, x in steps:
            if what == "fork":
                n = fa.cache_fork(t_refs, t_table, n, x, page)
            else:
                n, status = fa.cache_resize(t_refs, k, v, t_table, n, x)
                said.append(status)
        return n, said

    def reset():
        k.copy_(k0), v.copy_(v0), t_table.fill_(-1), t_refs.zero_()

    def check(n, said):
        assert all(x.tolist() == [0, 0] for x in said)
        assert n.tolist() == lens and t_refs.tolist() == refs and t_table.tolist() == table
        assert torch.equal(bits(k), bits(want_k)) and torch.equal(bits(v), bits(want_v))

    for _ in range(10):
        reset()
        check(*play())
    graph = torch.cuda.CUDAGraph()
    reset()
    with torch.cuda.graph(graph):
        out = play()
    for _ in range(10):
        reset()
        graph.replay()
        check(*out)


@pytest.mark.gpu
def test_append_reads_the_keys_of_the_kernel_before():
    """cache_append begins while cache_compact still moves rows of many layers; what it copies are rows that those
    moves leave behind."""
    page, B, layers, Hkv, d = 16, 8, 32, 8, 128
    s = pm.Setup([64] * B, [32] * B, page, Hkv, d, seed=5)
    deep = s.k_pages[None].repeat(layers, 1, 1, 1, 1), s.v_pages[None].repeat(layers, 1, 1, 1, 1)
    path, kept = i32([list(range(1, 31))] * B), i32([30] * B)
    cu = i32([0, page])
    # one row's first drafted page in the last layer, as packed keys
    p, _ = s.place(B - 1, 64)
    to_k, to_v = torch.zeros((1, page, Hkv, d), dtype=torch.bfloat16, device="cuda"), \
        torch.zeros((1, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    start = [x.clone() for x in deep]
    want = s.k_pages.clone()
    for i in range(page):
        pf, rf = s.place(B - 1, 64 + i + 1)
        want[p, i] = s.k_pages[pf, rf]
    for _ in range(10):
        deep[0].copy_(start[0]), deep[1].copy_(start[1]), to_k.zero_()
        fa.cache_compact(*deep, s.t_table, s.t_lens, path, kept)
        fa.cache_append(deep[0][-1, p], deep[1][-1, p], to_k, to_v, i32([[0]]), i32([0]), cu)
        assert torch.equal(bits(to_k[0]), bits(want[p]))


def test_the_join_reads_the_lengths_from_l2_before_its_wait():
    """The join looks at cu_seqlens and cache_lens before it waits for the main kernel: past L1, which may still
    hold lines from before these arrays were written."""
    text = open(os.path.join(CSRC, "fa_paged.cu")).read()
    join = text[text.index("paged_combine_kernel(const __grid_constant__"):]
    early = join[: join.index("grid_wait();")]
    assert "warp_units<true>(p)" in early
    assert not re.search(r"paged_seq\(|warp_units\(|p\.cu\b|cache_lens|page_table|p\.mask|prefix\[", early)
    seq = text[text.index("PagedSeq paged_seq(const PagedParams"):]
    assert "EARLY ? __ldcg(x) : *x" in seq[: seq.index("\n}\n")]
