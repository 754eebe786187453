"""cache_resize in pools of several stretches (the block that keeps the books looks at
16384 counts at a time), and the outcomes that a run of calls has to reach."""
import random

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm

pytestmark = pytest.mark.gpu

STRETCH = 16384


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(x):
    return x.view(torch.int16)


def rows(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def resize(table, lens, refs, new, page, t, want):
    """One call and the model's -> (lengths, [missing, refused], copies, pages taken)."""
    before = [list(row) for row in table]
    lens, said, copies = pm.resize(table, lens, refs, new, page)
    for f, to, m in copies:
        for w in want:
            w[..., to, :m, :, :] = w[..., f, :m, :, :]
    t["lens"], status = fa.cache_resize(t["refs"], t["k"], t["v"], t["table"], t["lens"], i32(new))
    assert status.tolist() == said and t["lens"].tolist() == lens and t["refs"].tolist() == refs
    assert t["table"].tolist() == table
    assert torch.equal(bits(t["k"]), bits(want[0])) and torch.equal(bits(t["v"]), bits(want[1]))
    taken = [x for row, old in zip(table, before) for x, y in zip(row, old) if x != y and x >= 0]
    return lens, said, copies, taken


@pytest.mark.parametrize("num", [2 * STRETCH, 2 * STRETCH + 1, 3 * STRETCH - 5, 50000])
@pytest.mark.parametrize("aligned", [True, False])
def test_pages_from_several_stretches_in_one_call(num, aligned):
    """Few free pages in every stretch, so that a call takes pages of two or three, with copies; the counts
    begin on a 16-byte boundary or not."""
    page, B, cols = 16, 40, 12
    r = random.Random(num)
    refs = [1 + (i % 3 == 0) for i in range(num)]  # pages that rows elsewhere hold
    stretches = -(-num // STRETCH)
    for s in range(stretches):
        here = range(s * STRETCH, min((s + 1) * STRETCH, num))
        free = r.sample(here, min(90, len(here)))
        for p in {here[0], here[-1], *free}:  # at both ends of a stretch too
            refs[p] = 0
    k, v = rows((num, page, 1, 64), 1), rows((num, page, 1, 64), 2)
    store = torch.zeros(num + 4, dtype=torch.int32, device="cuda")
    at = 0 if aligned else 1
    store[at : at + num] = i32(refs)
    store[at + num :] = -99
    table, lens = [[-1] * cols for _ in range(B)], [0] * B
    t = dict(refs=store[at : at + num], k=k, v=v, table=i32(table), lens=i32(lens))
    assert (t["refs"].data_ptr() % 16 == 0) == aligned
    want = [k.clone(), v.clone()]
    # 84 pages: within the first stretch
    lens, said, copies, taken = resize(table, lens, refs, [page + 5] * 2 + [2 * page + 3] * 20 + [page + 9] * 10 + [0] * 8,
                                       page, t, want)
    assert said == [0, 0] and len(taken) == 84 and max(taken) < STRETCH
    # the last rows get others' pages: shared, partly filled last pages
    parents = list(range(32)) + [2, 2, 3, 24, 24, 25, 31, 31]
    table[:], lens = pm.fork(table, lens, refs, parents, page)
    t["lens"] = fa.cache_fork(t["refs"], t["table"], t["lens"], i32(parents), page)
    # all grow: 2 or 3 pages a row and the copies, over the first stretch's end into the others
    lens, said, copies, taken = resize(table, lens, refs, [n + 2 * page + b % page for b, n in enumerate(lens)], page, t, want)
    assert said == [0, 0] and len(copies) == 8
    assert {x // STRETCH for x in taken} >= {0, 1} and any(to >= STRETCH for _, to, _ in copies)
    if num > 2 * STRETCH + 100:  # what is left of the second stretch and some of the third
        lens, said, copies, taken = resize(table, lens, refs, [n + 2 * page for n in lens], page, t, want)
        assert said == [0, 0] and {x // STRETCH for x in taken} >= {1, 2}
    # more than all free pages: nothing moves; then exactly all of them
    free = sum(x == 0 for x in refs)
    cap = cols * page
    lens, said, copies, taken = resize(table, lens, refs, [cap] * B, page, t, want)
    assert said[0] == B * cols - sum(pm.pages_of(n, page) for n in lens) - free and said[0] > 0 and not taken
    new, left = list(lens), free
    for b in range(B):
        n = min(left, cols - pm.pages_of(lens[b], page))
        if n > 0:
            new[b], left = (pm.pages_of(lens[b], page) + n) * page, left - n
    assert left == 0
    lens, said, copies, taken = resize(table, lens, refs, new, page, t, want)
    assert said == [0, 0] and len(taken) == free and 0 not in refs
    # and all of it back
    lens, said, copies, taken = resize(table, lens, refs, [0] * B, page, t, want)
    assert lens == [0] * B and (store[at + num :] == -99).all() and (aligned or int(store[0]) == 0)


@pytest.mark.parametrize("B,page,cols,num,layers,seed,expect", [
    (64, 16, 12, 900, None, 3, {"copy", "grown"}), (64, 16, 12, 300, 2, 4, {"copy", "grown", "missing"}),
    (2, 16, 6, 12, 3, 10, {"copy", "grown"}), (1, 32, 9, 9, None, 6, {"grown"}),
    (1, 32, 9, 4, None, 7, {"grown", "missing"}), (1100, 16, 4, 4000, None, 8, {"copy", "grown", "missing"}),
])
def test_every_outcome_is_reached(B, page, cols, num, layers, seed, expect):
    r = random.Random(seed)
    shape = ((layers,) if layers else ()) + (num, page, 2, 64)
    k, v = rows(shape, seed), rows(shape, seed + 50)
    table, lens, refs = [[-1] * cols for _ in range(B)], [0] * B, [0] * num
    t = dict(refs=i32(refs), k=k, v=v, table=i32(table), lens=i32(lens))
    want, cap, reached = [k.clone(), v.clone()], cols * page, set()
    for step in range(12):
        if step % 3 == 2 and B > 1:
            parents = [r.randrange(B) if r.random() < 0.6 else b for b in range(B)]
            table[:], lens = pm.fork(table, lens, refs, parents, page)
            t["lens"] = fa.cache_fork(t["refs"], t["table"], t["lens"], i32(parents), page)
        new = [r.choice([n, min(n + 1, cap), r.randint(0, n), r.randint(n, max(3 * page, n))]) for n in lens]
        if step % 4 == 3:
            new = [cap] * B
        had = lens
        lens, said, copies, taken = resize(table, lens, refs, new, page, t, want)
        reached |= {w for w, x in (("copy", copies), ("missing", said[0] > 0), ("grown", any(a > b for a, b in zip(lens, had))))
                    if x}
    assert reached == expect
