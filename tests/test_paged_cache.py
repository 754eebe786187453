"""The paged cache's own operators against a plain model of the page table, and a
decoding loop of them together with the attention."""
import random

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(x):
    return x.view(torch.int16)


def rows(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("lens,new,page,Hkv,d", [
    ([0], [1], 16, 1, 64), ([5, 16, 31], [1, 1, 1], 16, 8, 128), ([0, 7, 100, 0], [130, 0, 33, 300], 64, 3, 256),
    ([17] * 40, [0, 3] * 20, 32, 2, 64), ([3] * 1100, [1] * 1100, 16, 1, 64), ([250, 0], [7, 600], 256, 16, 128),
])
def test_append(lens, new, page, Hkv, d):
    s = pm.Setup(lens, new, page, Hkv, d, seed=1, fill=3.0)
    k, v = rows((s.total, Hkv, d), 2), rows((s.total, Hkv, d), 3)
    want_k, want_v = s.k_pages.clone(), s.v_pages.clone()
    for b in range(s.B):
        for i in range(new[b]):
            p, r = s.place(b, lens[b] + i)
            want_k[p, r], want_v[p, r] = k[s.cu[b] + i], v[s.cu[b] + i]
    fa.cache_append(k, v, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu)
    assert torch.equal(bits(s.k_pages), bits(want_k)) and torch.equal(bits(s.v_pages), bits(want_v))


def test_append_drops_rows_without_a_place():
    s = pm.Setup([10, 30], [20, 20], 16, 2, 64, seed=4, fill=3.0)
    s.table[0][1] = -1  # the second page of sequence 0 was dropped
    s.table[1] = s.table[1][:]
    k, v = rows((50, 2, 64), 5), rows((50, 2, 64), 6)
    want = s.k_pages.clone()
    narrow = i32([row[:3] for row in s.table])  # sequence 1: places 48 and 49 are past the table
    cu = i32([2, 22, 42])  # rows 0, 1 and 42.. belong to nobody
    for b in range(2):
        for i in range(20):
            pos = s.lens[b] + i
            if pos < 48 and s.table[b][pos // 16] >= 0:
                want[s.table[b][pos // 16], pos % 16] = k[2 + 20 * b + i]
    fa.cache_append(k, v, s.k_pages, s.v_pages, narrow, s.t_lens, cu)
    assert torch.equal(bits(s.k_pages), bits(want))
    before = s.k_pages.clone()
    fa.cache_append(k[:0], v[:0], s.k_pages, s.v_pages, narrow, s.t_lens, i32([0, 0, 0]))
    fa.cache_append(k, v, s.k_pages, s.v_pages, narrow, i32([-1, -5]), cu)  # lengths outside the contract
    assert torch.equal(bits(s.k_pages), bits(before))


def test_append_past_32_bit_offsets():
    page, Hkv, d = 256, 16, 128
    num = 2**31 // (page * Hkv * d) + 8
    kp = torch.zeros((num, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    k, v = rows((300, Hkv, d), 1), rows((300, Hkv, d), 2)
    fa.cache_append(k, v, kp, vp, i32([[num - 1, num - 3]]), i32([0]), i32([0, 300]))
    assert torch.equal(kp[num - 1], k[:256]) and torch.equal(vp[num - 3, :44], v[256:])
    assert (kp[: num - 3] == 0).all() and (kp[num - 2] == 0).all() and (kp[num - 3, 44:] == 0).all()


# ------------------------------------------------------------------ compact
@pytest.mark.parametrize("layers", [None, 1, 3])
@pytest.mark.parametrize("lens,draft,page,Hkv,d,paths", [
    ([5], 8, 16, 2, 64, [[0, 2, 3, 7]]),
    ([0, 15, 16, 40], 20, 16, 8, 128, [[], [19], [0, 1, 2], [1, 3, 5, 7, 9, 11, 13, 15, 17, 19]]),
    ([100, 3], 200, 64, 3, 256, [list(range(0, 200, 1)), list(range(60, 200))]),
    ([7], 250, 32, 1, 64, [sorted(random.Random(1).sample(range(250), 140))]),
])
def test_compact(lens, draft, page, Hkv, d, paths, layers):
    s = pm.Setup(lens, [draft] * len(lens), page, Hkv, d, seed=2, layers=layers)
    most = max(max(len(x) for x in paths), 1)
    path = i32([x + [-9] * (most - len(x)) for x in paths])
    want = [s.k_pages.clone(), s.v_pages.clone()]
    for got, w in zip((s.k_pages, s.v_pages), want):
        for b, x in enumerate(paths):
            for i, e in enumerate(x):
                (pf, rf), (pt, rt) = s.place(b, lens[b] + e), s.place(b, lens[b] + i)
                w[..., pt, rt, :, :] = got[..., pf, rf, :, :]
    out = fa.cache_compact(s.k_pages, s.v_pages, s.t_table, s.t_lens, path, i32([len(x) for x in paths]))
    assert out.tolist() == [a + len(x) for a, x in zip(lens, paths)]
    assert torch.equal(bits(s.k_pages), bits(want[0])) and torch.equal(bits(s.v_pages), bits(want[1]))


def test_compact_ends_a_path_that_does_not_ascend_or_leaves_the_table():
    paths = [[1, 1, 2], [0, 5, 4, 6], [-1, 2], [2, 10**9], [3, 2**31 - 1], [2, 4, 5], [2, 4, 5], [0]]
    counts = [3, 4, 2, 2, 2, 7, -3, 1]
    kept = [1, 2, 0, 1, 1, 3, 0, 1]
    s = pm.Setup([9] * 8, [8] * 8, 16, 2, 64, seed=3)
    most = 4
    out = fa.cache_compact(s.k_pages, s.v_pages, s.t_table, s.t_lens,
                           i32([x + [-1] * (most - len(x)) for x in paths]), i32(counts))
    assert out.tolist() == [9 + m for m in kept]
    p, r = s.place(1, 10)
    pf, rf = s.place(1, 14)
    assert torch.equal(s.k_pages[p, r], s.k_pages[pf, rf])
    out = fa.cache_compact(s.k_pages, s.v_pages, s.t_table, i32([-4] * 8), i32([[0, 1]] * 8), i32([2] * 8))
    assert out.tolist() == [-4] * 8


# ------------------------------------------------------------------ fork
def check_books(s, table, lens, refs):
    assert s.t_refs.tolist() == refs
    for b, n in enumerate(lens):
        h = pm.pages_of(n, s.page)
        assert s.t_table[b].tolist()[:h] == table[b][:h], b
    return True


@pytest.mark.parametrize("B,page,most,seed", [(1, 16, 100, 0), (7, 16, 900, 1), (64, 64, 2000, 2), (300, 16, 60, 3),
                                              (130, 16, 40000, 4), (4096, 32, 40, 5)])
def test_fork(B, page, most, seed):
    r = random.Random(seed)
    lens = [r.randint(0, most) for _ in range(B)]
    cols = pm.pages_of(most, page) + r.randint(0, 3)
    refs = [0] * (sum(pm.pages_of(n, page) for n in lens) + 5)
    ids = list(range(len(refs)))
    r.shuffle(ids)
    table, at = [], 0
    for n in lens:
        h = pm.pages_of(n, page)
        table.append(ids[at : at + h] + [-1] * (cols - h))
        at += h
    for x in ids[:at]:
        refs[x] = 1
    t_table, t_refs, t_lens = i32(table), i32(refs), i32(lens)
    for step in range(3):
        parents = [r.choice([b, r.randrange(B), r.randrange(B), -1, -5, B, 2**31 - 1]) for b in range(B)]
        table, lens = pm.fork(table, lens, refs, parents, page)
        t_lens = fa.cache_fork(t_refs, t_table, t_lens, i32(parents), page)
        assert t_lens.tolist() == lens and t_refs.tolist() == refs and t_table.tolist() == table, step
    t_lens = fa.cache_fork(t_refs, t_table, t_lens, i32([-1] * B), page)
    assert t_lens.tolist() == [0] * B and t_refs.tolist() == [0] * len(refs) and (t_table == -1).all()


def test_fork_with_rubbish_in_the_tables_stays_in_bounds():
    refs, table = i32([1, 1, 1, 1]), i32([[0, 99, -3], [2, 1, 2**31 - 1], [-(2**31), 3, 0]])
    lens = fa.cache_fork(refs, table, i32([40, -5, 10**9]), i32([2, 0, 1]), 16)
    assert lens.tolist() == [10**9, 40, -5]
    assert table.tolist() == [[-(2**31), 3, 0], [0, 99, -3], [-1, -1, -1]]


# ------------------------------------------------------------------ resize
@pytest.mark.parametrize("B,page,cols,spare,layers,seed", [
    (1, 16, 4, 10, None, 0), (5, 16, 9, 30, 2, 1), (40, 32, 6, 60, 1, 2), (64, 16, 12, 20, None, 3),
    (1500, 16, 5, 3000, None, 4), (20, 256, 3, 60, 2, 5), (4096, 16, 3, 20000, None, 6), (9, 64, 2000, 40000, None, 7),
])
def test_resize(B, page, cols, spare, layers, seed):
    r = random.Random(seed)
    Hkv, d = (1, 64) if spare > 1000 else (3, 64)
    num = spare + 7
    shape = ((layers,) if layers else ()) + (num, page, Hkv, d)
    if num * page > 10**6:
        shape = (num, page, 1, 64)
    k, v = rows(shape, seed + 1), rows(shape, seed + 2)
    want_k, want_v = k.clone(), v.clone()
    table, lens, refs = [[-1] * cols for _ in range(B)], [0] * B, [0] * num
    t_table, t_lens, t_refs = i32(table), i32(lens), i32(refs)
    outcomes = set()
    cap = cols * page
    for step in range(8):
        if step % 3 == 2:  # share rows, so that last pages have to be copied
            parents = [r.randrange(B) if r.random() < 0.7 else b for b in range(B)]
            table, lens = pm.fork(table, lens, refs, parents, page)
            t_lens = fa.cache_fork(t_refs, t_table, t_lens, i32(parents), page)
        top = min(cap, 3 * spare * page // B + 5)
        new = [r.choice([a, min(a + 1, cap), r.randint(0, a), r.randint(0, top), r.randint(a, min(cap, a + page))])
               for a in lens]
        if step % 4 == 3:
            new[r.randrange(B)] = r.choice([-1, cap + 1, 2**31 - 1])
        lens, said, copies = pm.resize(table, lens, refs, new, page)
        for f, t, m in copies:
            want_k[..., t, :m, :, :] = want_k[..., f, :m, :, :]
            want_v[..., t, :m, :, :] = want_v[..., f, :m, :, :]
        t_lens, status = fa.cache_resize(t_refs, k, v, t_table, t_lens, i32(new))
        assert status.tolist() == said, step
        assert t_lens.tolist() == lens and t_refs.tolist() == refs and t_table.tolist() == table, step
        assert torch.equal(bits(k), bits(want_k)) and torch.equal(bits(v), bits(want_v)), step
        outcomes |= {("copy", bool(copies)), ("missing", said[0] > 0), ("refused", said[1] > 0)}
    assert ("refused", True) in outcomes


def test_resize_takes_nothing_when_pages_are_missing():
    page, Hkv, d = 16, 1, 64
    k, v = rows((6, page, Hkv, d), 1), rows((6, page, Hkv, d), 2)
    refs, table = i32([1, 0, 1, 0, 1, 1]), i32([[0, 2, -1], [4, 5, -1], [-1, -1, -1]])
    lens = i32([20, 32, 0])
    # row 1 gives page 5 back; rows 0 and 2 want four pages of the three free ones
    out, status = fa.cache_resize(refs, k, v, table, lens, i32([48, 16, 48]))
    assert out.tolist() == [20, 16, 0] and status.tolist() == [1, 0]
    assert refs.tolist() == [1, 0, 1, 0, 1, 0] and table.tolist() == [[0, 2, -1], [4, -1, -1], [-1, -1, -1]]
    out, status = fa.cache_resize(refs, k, v, table, out, i32([48, 16, 32]))
    assert out.tolist() == [48, 16, 32] and status.tolist() == [0, 0]
    assert refs.tolist() == [1] * 6 and table.tolist() == [[0, 2, 1], [4, -1, -1], [3, 5, -1]]


def test_resize_counts_needs_past_32_bits():
    """4096 rows that want 2^20 pages each: 2^32 in all, which wraps to 0 in 32 bits."""
    cols = 1 << 20
    k = v = rows((5, 16, 1, 64), 1)
    table = torch.full((4096, cols), -1, dtype=torch.int32, device="cuda")
    refs = i32([0, 1, 0, 0, 1])
    lens = torch.zeros(4096, dtype=torch.int32, device="cuda")
    out, status = fa.cache_resize(refs, k, v, table, lens, torch.full_like(lens, cols * 16))
    assert status.tolist() == [2**31 - 1, 0] and int(out.sum()) == 0 and refs.tolist() == [0, 1, 0, 0, 1]
    want = lens.clone()
    want[4095] = 48
    out, status = fa.cache_resize(refs, k, v, table, lens, want)
    assert status.tolist() == [0, 0] and out.tolist() == want.tolist() and refs.tolist() == [1] * 5
    assert table[4095, :4].tolist() == [0, 2, 3, -1]


def test_resize_with_rubbish_in_the_table_stays_in_bounds():
    k, v = rows((4, 16, 1, 64), 1), rows((4, 16, 1, 64), 2)
    refs, table = i32([2, 2, 0, 0]), i32([[99, -1], [-7, 2**31 - 1], [0, 1]])
    out, status = fa.cache_resize(refs, k, v, table, i32([5, 20, 30]), i32([7, 3, 31]))
    assert out.tolist() == [7, 3, 31] and status.tolist() == [0, 0]
    assert table.tolist() == [[99, -1], [-7, -1], [0, 2]] and refs.tolist() == [2, 1, 1, 0]


# ------------------------------------------------------------------ together
class Sequence:
    """What one row of the batch should hold: its keys and values in every layer, in order."""

    def __init__(self, layers, Hkv, d):
        self.k = torch.zeros((layers, 0, Hkv, d), dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()

    def copy(self):
        s = Sequence.__new__(Sequence)
        s.k, s.v = self.k.clone(), self.v.clone()
        return s


def plain(q, k, v, seen):
    n, H, d = q.shape
    G = H // k.shape[1]
    kk, vv = k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    z = torch.einsum("thd,khd->htk", q.double(), kk) * d**-0.5
    z = z.masked_fill(~seen[None], float("-inf"))
    return torch.einsum("htk,khd->thd", torch.softmax(z, -1), vv), torch.logsumexp(z, -1), \
        torch.einsum("htk,khd->thd", torch.softmax(z, -1), vv.abs())


@pytest.mark.parametrize("page,H,Hkv,d,draft", [(16, 4, 2, 64, 5), (64, 8, 2, 128, 12), (32, 8, 8, 256, 20)])
def test_speculative_decoding_loop(page, H, Hkv, d, draft):
    """Prompt, drafted trees, acceptance, forks and frees on one pool; after every step the attention
    of every row is that over the rows it should hold."""
    layers, B, cols, num = 2, 6, 40, 120
    r = random.Random(page)
    k_pages = torch.full((layers, num, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v_pages = k_pages.clone()
    refs, table, lens = i32([0] * num), i32([[-1] * cols] * B), i32([0] * B)
    want = [Sequence(layers, Hkv, d) for _ in range(B)]
    seed = [0]

    def fresh(*shape):
        seed[0] += 1
        return rows(shape, 1000 + seed[0])

    for step in range(7):
        n = [r.randint(1, 3 * page) for _ in range(B)] if step == 0 else [r.randint(0, draft) for _ in range(B)]
        if sum(n) == 0:
            n[0] = 1
        cu, total = [0], sum(n)
        for x in n:
            cu.append(cu[-1] + x)
        up, status = fa.cache_resize(refs, k_pages, v_pages, table, lens, lens + i32(n))
        assert status.tolist() == [0, 0]
        masks, seen = pm.tree_masks(n, (max(n) + 63) // 64, seed=step)
        for layer in range(layers):
            k, v, q = fresh(total, Hkv, d), fresh(total, Hkv, d), fresh(total, H, d)
            fa.cache_append(k, v, k_pages[layer], v_pages[layer], table, lens, i32(cu))
            chain = step == 0
            o, lse = fa.attention_fwd_paged(q, k_pages[layer], v_pages[layer], table, lens, i32(cu), max(n),
                                            tree_mask=None if chain else masks.cuda())
            for b in range(B):
                if n[b] == 0:
                    continue
                at = slice(cu[b], cu[b + 1])
                have = want[b].k.shape[1] if layer == 0 else want[b].k.shape[1] - n[b]
                kk = torch.cat([want[b].k[layer, :have], k[at]])
                vv = torch.cat([want[b].v[layer, :have], v[at]])
                see = torch.ones((n[b], have + n[b]), dtype=torch.bool, device="cuda")
                for i in range(n[b]):
                    for j in range(n[b]):
                        see[i, have + j] = j <= i if chain else j in seen[cu[b] + i]
                o64, l64, mag = plain(q[at], kk, vv, see)
                # rounding of O and of the weights, 2^-8 each; scores of a few units in fp32 well below that
                assert ((o[at] - o64).abs() <= 2.0**-8 * o64.abs() + 1.01 * 2.0**-8 * mag + 1e-4).all()
                assert (lse[:, at] - l64).abs().max() <= 1e-4
                if layer == 0:  # the other layer's rows get their place
                    for x, y in (("k", k), ("v", v)):
                        old = getattr(want[b], x)
                        setattr(want[b], x, torch.cat([old, torch.zeros((layers, n[b], Hkv, d), dtype=old.dtype,
                                                                        device="cuda")], 1))
                want[b].k[layer, have:], want[b].v[layer, have:] = k[at], v[at]
        if step == 0:
            lens = up
        else:  # accept the path to a random drafted token
            paths = [sorted(seen[cu[b] + r.randrange(n[b])]) if n[b] else [] for b in range(B)]
            most = max(len(x) for x in paths)
            kept = fa.cache_compact(k_pages, v_pages, table, lens, i32([x + [0] * (most - len(x)) for x in paths]),
                                    i32([len(x) for x in paths]))
            lens, status = fa.cache_resize(refs, k_pages, v_pages, table, up, kept)
            assert torch.equal(lens, kept) and status.tolist() == [0, 0]
            for b in range(B):
                base = want[b].k.shape[1] - n[b]
                keep = torch.tensor(list(range(base)) + [base + j for j in paths[b]], device="cuda", dtype=torch.long)
                want[b].k, want[b].v = want[b].k[:, keep], want[b].v[:, keep]
        if step % 2 == 1:
            parents = [r.choice([b, r.randrange(B), r.randrange(B), -1]) for b in range(B)]
            lens = fa.cache_fork(refs, table, lens, i32(parents), page)
            want = [want[p].copy() if p >= 0 else Sequence(layers, Hkv, d) for p in parents]
        assert lens.tolist() == [w.k.shape[1] for w in want]
        held = torch.zeros(num, dtype=torch.int32)
        for row, m in zip(table.tolist(), lens.tolist()):
            for x in row[: pm.pages_of(m, page)]:
                held[x] += 1
        assert torch.equal(held, refs.cpu())
    assert fa.fa_last_device_status() == fa.FA_OK


def test_captured_step_replays_on_other_contents():
    """A whole step captured in a graph on static buffers, replayed with other lengths and keys."""
    page, H, Hkv, d, B, cols, num = 16, 8, 2, 128, 3, 30, 100
    k_pages, v_pages = rows((num, page, Hkv, d), 1), rows((num, page, Hkv, d), 2)
    refs, table, lens = i32([0] * num), i32([[-1] * cols] * B), i32([0] * B)
    lens, _ = fa.cache_resize(refs, k_pages, v_pages, table, lens, i32([40, 7, 300]))
    k, v, q = rows((B, Hkv, d), 3), rows((B, Hkv, d), 4), rows((B, H, d), 5)
    cu = i32([0, 1, 2, 3])

    def step():
        up, status = fa.cache_resize(refs, k_pages, v_pages, table, lens, lens + 1)
        fa.cache_append(k, v, k_pages, v_pages, table, lens, cu)
        o, lse = fa.attention_fwd_paged(q, k_pages, v_pages, table, lens, cu, 1)
        lens.copy_(up)
        return o, lse, status

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(20):
        k.copy_(rows((B, Hkv, d), 100 + i))
        v.copy_(rows((B, Hkv, d), 200 + i))
        q.copy_(rows((B, H, d), 300 + i))
        before = lens.clone()
        graph.replay()
        assert out[2].tolist() == [0, 0] and torch.equal(lens, before + 1)
        o, lse = fa.attention_fwd_paged(q, k_pages, v_pages, table, before, cu, 1)
        assert torch.equal(o, out[0]) and torch.equal(lse, out[1])
        for b in range(B):
            n = int(lens[b])
            ids = table[b, : pm.pages_of(n, page)].long()
            assert torch.equal(k_pages[ids].reshape(-1, Hkv, d)[n - 1], k[b])
    assert lens.tolist() == [61, 28, 321]


@pytest.mark.parametrize("new,H,Hkv,d", [(1, 8, 4, 128), (30, 8, 2, 128), (70, 4, 2, 64)])
def test_lengths_of_one_call_feed_the_next_at_once(new, H, Hkv, d):
    """cache_compact's lengths go straight into the attention while the moves of many layers still run:
    each kernel may start early but must not read what the one before it has yet to write."""
    page, B, layers = 16, 24, 48
    s = pm.Setup([120] * B, [new] * B, page, Hkv, d, seed=new, H=H)
    deep = s.k_pages[None].repeat(layers, 1, 1, 1, 1), s.v_pages[None].repeat(layers, 1, 1, 1, 1)
    base = i32([10 + b for b in range(B)])
    paths = i32([list(range(40))] * B)
    counts = [i32([(7 * b + 13 * r) % 41 for b in range(B)]) for r in range(6)]

    def step(kept, wait):
        lens = fa.cache_compact(*deep, s.t_table, base, paths, kept)
        if wait:
            torch.cuda.synchronize()
        o, lse = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, lens, s.t_cu, new)
        if wait:
            torch.cuda.synchronize()
        return lens, o, lse

    want = [step(c, True) for c in counts]
    for _ in range(20):
        for c, w in zip(counts, want):
            got = step(c, False)
            assert all(torch.equal(x, y) for x, y in zip(got, w))
        got = [step(c, False) for c in counts]
        assert all(torch.equal(x, y) for g, w in zip(got, want) for x, y in zip(g, w))


def test_calls_on_a_given_stream_and_two_at_once():
    s = [pm.Setup([700, 33], [9, 20], 32, 2, 128, seed=20 + i, H=8) for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for x, y, z in zip(s, streams, got):
            z.append(fa.attention_fwd_paged(x.q, x.k_pages, x.v_pages, x.t_table, x.t_lens, x.t_cu, 20, stream=y))
    got[0].append(fa.attention_fwd_paged(s[0].q, s[0].k_pages, s[0].v_pages, s[0].t_table, s[0].t_lens, s[0].t_cu, 20,
                                         stream=streams[1].cuda_stream))
    torch.cuda.synchronize()
    for x, z in zip(s, got):
        want = fa.attention_fwd_paged(x.q, x.k_pages, x.v_pages, x.t_table, x.t_lens, x.t_cu, 20)
        for o, lse in z:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    x = s[0]
    k = rows((29, 2, 128), 1)
    fa.cache_append(k, k, x.k_pages, x.v_pages, x.t_table, x.t_lens, x.t_cu, stream=streams[0])
    out = fa.cache_compact(x.k_pages, x.v_pages, x.t_table, x.t_lens, i32([[0], [0]]), i32([1, 1]), stream=streams[0])
    assert out is not None
    streams[0].synchronize()
    p, r = x.place(0, 708)
    assert torch.equal(x.k_pages[p, r], k[8]) and out.tolist() == [701, 34]
