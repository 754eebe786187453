"""New tokens' queries, keys and values made ready and put into the paged cache in one call,
and a serving loop of the calls around such a cache: append, attention, weight sums, eviction,
pages given back."""
import math

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm
import rope_model as rm

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(x):
    return x.view(torch.int16)


class Step:
    def __init__(self, lens, new, page, H, Hkv, d, rot=None, axes=None, pairs=False, norm="float32", fused=True, positions=None,
                 seed=0):
        self.s = s = pm.Setup(lens, new, page, Hkv, d, seed=seed + d, fill=0.125)
        g = torch.Generator().manual_seed(seed + H)
        rot = d if rot is None else rot
        x = torch.randn((s.total, H + 2 * Hkv, d), generator=g).to(torch.bfloat16).cuda()
        self.q, self.k, self.v = x.split([H, Hkv, Hkv], 1)
        if not fused:
            self.q, self.k, self.v = self.q.contiguous(), self.k.contiguous(), self.v.contiguous()
        self.inv_freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
        weight = lambda: (1 + 0.3 * torch.randn(d, generator=g)).to(getattr(torch, norm)).cuda() if norm else None
        self.qw, self.kw, self.axes, self.pairs = weight(), weight(), axes, pairs
        self.positions = positions
        places = torch.tensor([max(lens[b], 0) + i for b in range(s.B) for i in range(new[b])], dtype=torch.int32)
        at = places if positions is None else positions.cpu()
        if positions is None and axes is not None:
            at = at.expand(max(axes) + 1, -1)
        self.angle = rm.angles(at, self.inv_freq.cpu(), axes)

    def run(self, **kw):
        s = self.s
        return fa.cache_append_rope(self.q, self.k, self.v, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, self.inv_freq,
                                    positions=self.positions, q_weight=self.qw, k_weight=self.kw, axes=self.axes,
                                    interleaved=self.pairs, **kw)

    def check(self, q, k0, v0, gone=()):
        """gone: (sequence, place) that no page holds."""
        s = self.s
        rm.check_forward(q, self.q, self.qw, self.angle, self.pairs, what="q")
        k, v = s.k_pages.cpu(), s.v_pages.cpu()
        at = [(t, *s.place(b, s.lens[b] + i)) for b in range(s.B) for i, t in enumerate(range(s.cu[b], s.cu[b + 1]))
              if (b, s.lens[b] + i) not in gone and s.lens[b] >= 0]
        t, p, r = (list(x) for x in zip(*at)) if at else ([], [], [])
        rm.check_forward(k[p, r], self.k[t], self.kw, self.angle[t], self.pairs, what="k")
        assert torch.equal(bits(v[p, r]), bits(self.v.cpu()[t]))
        k0, v0 = k0.cpu(), v0.cpu()
        k[p, r], v[p, r] = k0[p, r], v0[p, r]
        assert torch.equal(bits(k), bits(k0)) and torch.equal(bits(v), bits(v0)), "rows that are not new have changed"


CASES = [
    dict(lens=[0], new=[1], page=16, H=1, Hkv=1, d=64),
    dict(lens=[777], new=[1], page=64, H=32, Hkv=8, d=128, norm="bfloat16"),
    dict(lens=[15, 16, 17, 0, 300], new=[1] * 5, page=16, H=8, Hkv=2, d=128, pairs=True, norm=""),
    dict(lens=[200, 31, 0, 77], new=[5, 0, 33, 1], page=32, H=6, Hkv=3, d=64, rot=32, fused=False),
    dict(lens=[60, 3, 0], new=[130, 200, 0], page=256, H=4, Hkv=4, d=256, rot=64, axes=tuple(i % 3 for i in range(32))),
    dict(lens=[5] * 70, new=[1, 2] * 35, page=16, H=2, Hkv=2, d=64, axes=(0,) * 20 + (1,) * 12),
    dict(lens=[0, 0], new=[900, 1400], page=128, H=16, Hkv=2, d=128),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['lens'][:3]}-{c['new'][:3]}-d{c['d']}")
@pytest.mark.parametrize("given", [False, True])
def test_matches_the_model(case, given):
    total = sum(case["new"])
    positions = None
    if given:
        positions = (torch.arange(total, dtype=torch.int32) * 1000003 - 77).cuda()
        if case.get("axes"):
            positions = torch.stack([positions, -positions, positions // 7])[: max(case["axes"]) + 1].contiguous()
    c = Step(**case, positions=positions)
    k0, v0 = c.s.k_pages.clone(), c.s.v_pages.clone()
    q = c.run()
    torch.cuda.synchronize()
    c.check(q, k0, v0)


def test_rows_without_a_page_are_dropped_and_rows_of_no_sequence_left_alone():
    c = Step([20, -9, 40], [30, 2, 3], 16, 4, 2, 64)
    s = c.s
    s.table[0][2], s.table[2][2] = -1, s.num_pages  # places 32..47 of each
    s.t_table = i32(s.table)
    k0, v0 = s.k_pages.clone(), s.v_pages.clone()
    q = torch.full((35, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out = c.run(q_out=q)
    torch.cuda.synchronize()
    assert out is q
    c.check(q, k0, v0, gone={(b, p) for b in (0, 2) for p in range(32, 48)})
    s.t_cu = i32([0, 30, 32, 33])  # two rows behind the last sequence
    q.fill_(3.0)
    c.run(q_out=q)
    assert (q[33:] == 3).all() and not (q[:33] == 3).all()


def test_tables_outside_their_contract_write_nothing_elsewhere():
    c = Step([20, 0, 40], [3, 2, 30], 16, 4, 2, 64)
    s = c.s
    k0 = s.k_pages.clone()
    for lens in ([2**31 - 1, -5, 2**31 - 2], [2**30, 2**20, 63]):
        for cu in ([0, 3, 5, 35], [5, 0, 900, -4], [2**31 - 1, -(2**31), 3, 9]):
            s.t_lens, s.t_cu = i32(lens), i32(cu)
            c.run()
            torch.cuda.synchronize()
    s.t_table.fill_(-1)
    s.k_pages.copy_(k0)
    s.t_lens, s.t_cu = i32([1, 2, 3]), i32(s.cu)
    c.run()
    assert torch.equal(bits(s.k_pages), bits(k0))


def test_in_place_of_the_two_calls():
    """The same values, bit for bit, as the two calls that it replaces."""
    c = Step([100, 7], [40, 3], 32, 8, 2, 128, fused=False)
    s = c.s
    k_two, v_two = s.k_pages.clone(), s.v_pages.clone()
    q = c.run()
    at = i32([100 + i for i in range(40)] + [7, 8, 9])
    q2, k2 = fa.qk_norm_rope(c.q, c.k, at, c.inv_freq, q_weight=c.qw, k_weight=c.kw)
    fa.cache_append(k2, c.v, k_two, v_two, s.t_table, s.t_lens, s.t_cu)
    assert torch.equal(q, q2) and torch.equal(bits(k_two), bits(s.k_pages)) and torch.equal(bits(v_two), bits(s.v_pages))


def test_no_tokens():
    c = Step([10, 30], [0, 0], 16, 4, 2, 64)
    k0 = c.s.k_pages.clone()
    assert c.run().shape == (0, 4, 64) and torch.equal(bits(k0), bits(c.s.k_pages))


# ------------------------------------------------------------------ a serving loop
class Loop:
    """Sequences whose cache is cut to `keep` places whenever it has grown past it by `slack`; everything on the
    device.  The tokens' own positions go on counting, whatever was evicted."""

    def __init__(self, B, H, Hkv, d, page, keep, recent, slack, layers, seed=0):
        self.B, self.H, self.Hkv, self.d, self.page, self.layers = B, H, Hkv, d, page, layers
        self.keep, self.recent, self.slack = keep, recent, slack
        self.cols = pm.pages_of(keep + slack + 64, page) + 1
        pool = B * self.cols + 2
        self.k = torch.full((layers, pool, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.refs = i32([0] * pool)
        self.table = i32([[-1] * self.cols] * B)
        self.lens = i32([0] * B)
        self.weights = torch.zeros((layers, B, Hkv, self.cols * page), device="cuda")
        self.inv_freq = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.qw, self.kw = (1 + 0.1 * torch.randn((2, d), generator=self.g, device="cuda")).unbind()

    def step(self, qkv, cu, grown, positions, max_new, evict):
        """qkv [layers, total, H + 2 Hkv, d]; grown: int32 [B], new tokens -> (o, lse, q of each layer, kept, sums
        as they were before the eviction)."""
        held, said = fa.cache_resize(self.refs, self.k, self.v, self.table, self.lens, self.lens + grown)
        out = []
        for l in range(self.layers):
            q, k, v = qkv[l].split([self.H, self.Hkv, self.Hkv], 1)
            q = fa.cache_append_rope(q, k, v, self.k[l], self.v[l], self.table, self.lens, cu, self.inv_freq, positions,
                                     q_weight=self.qw, k_weight=self.kw)
            o, lse = fa.attention_fwd_paged(q, self.k[l], self.v[l], self.table, self.lens, cu, max_new)
            fa.attention_weights_paged(q, self.k[l], self.table, self.lens, cu, max_new, lse, self.weights[l])
            out.append((q, o, lse))
        kept = sums = None
        self.lens.copy_(held)
        if evict:
            sums = self.weights.clone()
            lens, kept = fa.cache_evict(self.refs, self.k, self.v, self.table, held, self.weights, self.keep, self.recent)
            lens, _ = fa.cache_resize(self.refs, self.k, self.v, self.table, held, lens)
            self.lens.copy_(lens)
        return out, kept, sums, said


def test_serving_loop():
    """Against a model that holds, for each head, the rows it has kept."""
    B, H, Hkv, d, page, layers = 3, 4, 2, 64, 16, 2
    loop = Loop(B, H, Hkv, d, page, keep=70, recent=9, slack=20, layers=layers)
    G, scale = H // Hkv, 1.0 / math.sqrt(d)
    held = {(l, b, h): ([], []) for l in range(layers) for b in range(B) for h in range(Hkv)}  # keys, values
    sums = {key: torch.zeros(0, dtype=torch.float64) for key in held}
    where = [0] * B
    for n_step, new in enumerate([[60, 33, 1], [20, 30, 70], [1, 1, 1], [5, 0, 2], [40, 7, 1], [1, 1, 1]]):
        total = sum(new)
        qkv = torch.randn((layers, total, H + 2 * Hkv, d), generator=loop.g, device="cuda").to(torch.bfloat16)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        positions = [where[b] + i for b in range(B) for i in range(new[b])]
        evict = n_step % 2 == 1
        before = loop.lens.tolist()
        out, kept, w_before, said = loop.step(qkv, i32(cu), i32(new), i32(positions), max(new), evict)
        torch.cuda.synchronize()
        assert said.tolist() == [0, 0] and fa.fa_last_device_status() == fa.FA_OK
        angle = rm.angles(torch.tensor(positions), loop.inv_freq.cpu(), None)
        for l in range(layers):
            q, k, v = qkv[l].cpu().double().split([H, Hkv, Hkv], 1)
            got_q, got_o, got_lse = out[l]
            rm.check_forward(got_q, q, loop.qw, angle, False, what=f"step {n_step} q")
            q64 = got_q.cpu().double()
            k64 = rm.forward(k, loop.kw.cpu().double(), angle, False).to(torch.bfloat16).double()
            for b in range(B):
                rows = slice(cu[b], cu[b + 1])
                for h in range(Hkv):
                    keys, values = held[l, b, h]
                    keys += list(k64[rows, h])
                    values += list(v[rows, h])
                    sums[l, b, h] = torch.cat([sums[l, b, h], torch.zeros(new[b], dtype=torch.float64)])
                    if new[b] == 0:
                        continue
                    kk, vv = torch.stack(keys), torch.stack(values)
                    z = torch.einsum("igd,kd->gik", q64[rows, h * G : (h + 1) * G], kk) * scale
                    hidden = torch.arange(len(keys))[None] - before[b] > torch.arange(new[b])[:, None]
                    z = z.masked_fill(hidden, float("-inf"))
                    p = z.softmax(-1)
                    o = torch.einsum("gik,kd->igd", p, vv)
                    err = (got_o[rows, h * G : (h + 1) * G].cpu().double() - o).norm() / o.norm()
                    assert err <= 2.0**-6, (n_step, l, b, h, float(err))  # keys, weights and result in bf16: 2^-8 each
                    sums[l, b, h] += p.sum((0, 1))
                    n = len(keys)
                    got = (w_before if evict else loop.weights)[l, b, h].cpu().double()
                    # rounding k to bf16 here and there may differ by a step where its error straddles one
                    assert ((got[:n] - sums[l, b, h]).abs() <= 0.05 * sums[l, b, h] + 1e-3).all() and (got[n:] == 0).all()
        where = [w + n for w, n in zip(where, new)]
        if evict:
            lens = loop.lens.tolist()
            for (l, b, h), (keys, values) in held.items():
                mine = kept[l, b, h].tolist()
                if len(keys) <= loop.keep:
                    assert mine[: len(keys)] == list(range(len(keys))) and set(mine[len(keys) :]) <= {-1}
                    continue
                assert lens[b] == loop.keep and mine == sorted(set(mine)) and mine[-loop.recent :] == list(range(len(keys) - loop.recent, len(keys)))
                w = w_before[l, b, h].cpu()
                older = [p for p in mine if p < len(keys) - loop.recent]
                left = sorted(set(range(len(keys) - loop.recent)) - set(older))
                assert min(w[older]) >= max(w[left])
                held[l, b, h] = ([keys[p] for p in mine], [values[p] for p in mine])
                sums[l, b, h] = sums[l, b, h][mine]
            assert int((loop.refs > 0).sum()) == sum(pm.pages_of(n, page) for n in lens)
    assert max(loop.lens.tolist()) <= loop.keep + loop.slack


def test_a_captured_loop_replays_as_it_ran():
    def make():
        loop = Loop(4, 8, 2, 128, 32, keep=90, recent=16, slack=20, layers=2, seed=3)
        qkv = torch.empty((2, 4 * 12, 12, 128), dtype=torch.bfloat16, device="cuda")
        cu, grown, positions = i32([0, 12, 24, 36, 48]), i32([12] * 4), i32(list(range(12)) * 4)
        return loop, qkv, lambda: loop.step(qkv, cu, grown, positions, 12, True)

    eager, q1, run = make()
    captured, q2, again = make()
    fresh = [x.clone() for x in (captured.k, captured.v, captured.refs, captured.table, captured.lens, captured.weights)]
    q2.normal_(generator=captured.g)
    again()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again()
    for x, y in zip((captured.k, captured.v, captured.refs, captured.table, captured.lens, captured.weights), fresh):
        x.copy_(y)
    g = torch.Generator(device="cuda").manual_seed(11)
    for _ in range(12):
        q1.normal_(generator=g)
        q2.copy_(q1)
        run()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in ((eager.lens, captured.lens), (eager.table, captured.table), (eager.weights, captured.weights)):
            assert torch.equal(x, y)
        assert torch.equal(bits(eager.k), bits(captured.k)) and torch.equal(bits(eager.v), bits(captured.v))
    assert eager.lens.tolist() == [90] * 4


# ------------------------------------------------------------------ both ways into the library, and given streams
class Declines:
    def __getattr__(self, name):
        return lambda *a: None


def calls():
    c = Step([100, 7, 0], [40, 3, 1], 32, 8, 2, 128, rot=96, axes=tuple(i % 2 for i in range(48)), seed=4)
    s, g = c.s, torch.Generator(device="cuda").manual_seed(2)
    pos = i32([list(range(44)), list(range(44, 0, -1))])
    args = dict(q_weight=c.qw, k_weight=c.kw, axes=c.axes, interleaved=True, eps=1e-5)
    w = torch.rand((3, 2, 160), generator=g, device="cuda")
    lse = torch.rand((8, 44), generator=g, device="cuda") * 3 + 3
    q = c.q.contiguous()
    return {
        "rope": (lambda **kw: fa.qk_norm_rope(c.q, c.k, pos, c.inv_freq, **args, **kw), ()),
        "rope without norms": (lambda **kw: fa.qk_norm_rope(c.q, c.k, pos[0].contiguous(), c.inv_freq, **kw), ()),
        "rope_bwd": (lambda **kw: fa.qk_norm_rope_bwd(c.q, c.k, c.q, c.k, pos, c.inv_freq, **args, **kw), ()),
        "rope_bwd of keys": (lambda **kw: fa.qk_norm_rope_bwd(c.q, c.k, None, c.k, pos[1].contiguous(), c.inv_freq,
                                                              k_weight=c.kw, **kw), ()),
        "append": (lambda **kw: fa.cache_append_rope(c.q, c.k, c.v, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, c.inv_freq,
                                                     pos, **args, **kw), (s.k_pages, s.v_pages)),
        "append at places": (lambda **kw: fa.cache_append_rope(c.q, c.k, c.v, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu,
                                                               c.inv_freq, **args, **kw), (s.k_pages, s.v_pages)),
        "weights": (lambda **kw: fa.attention_weights_paged(q, s.k_pages, s.t_table, s.t_lens, s.t_cu, 40, lse, w, decay=0.5,
                                                            scale=0.05, **kw), (w,)),
        "evict": (lambda **kw: fa.cache_evict(s.t_refs, s.k_pages, s.v_pages, s.t_table, s.t_lens, w, 33, 4, **kw),
                  (s.k_pages, s.v_pages, w)),
    }


def outcome(name, **kw):
    call, state = calls()[name]
    torch.cuda.synchronize()
    out = call(**kw)
    torch.cuda.synchronize()
    return [x for x in (out if isinstance(out, tuple) else (out,)) if x is not None] + list(state)


@pytest.mark.parametrize("name", list(calls()) if torch.cuda.is_available() else ["none"])
@pytest.mark.parametrize("how", ["no binding", "stream", "handle", "legacy"])
def test_every_way_gives_the_same(monkeypatch, name, how):
    want = outcome(name)
    if how == "no binding":
        monkeypatch.setattr(fa, "_fast", Declines())
        got = outcome(name)
    else:
        side = torch.cuda.Stream()
        got = outcome(name, stream={"stream": side, "handle": side.cuda_stream, "legacy": 0}[how])
    assert len(got) == len(want)
    for x, y in zip(want, got):
        x, y = (bits(t) if t.dtype == torch.bfloat16 else t for t in (x, y))
        assert x.dtype == y.dtype and torch.equal(x, y)


def test_the_ordinary_calls_take_the_binding(monkeypatch):
    """None of them falls back to the code that checks operand by operand."""
    module = fa._paged_binding()
    seen = []

    class Watches:
        def __getattr__(self, name):
            def call(*a):
                out = getattr(module, name)(*a)
                seen.append((name, out is not None))
                return out
            return call

    every = calls()
    monkeypatch.setattr(fa, "_fast", Watches())
    for call, _ in every.values():
        call()
    assert len(seen) == len(every) and all(ok for _, ok in seen), seen


def test_one_call_reads_what_the_one_before_writes():
    """Kernels begin while the one before still runs: a chain of calls on a big batch, again and again, against the
    same calls with waits between them."""
    def play(wait):
        loop = Loop(24, 8, 4, 128, 64, keep=100, recent=16, slack=40, layers=4, seed=5)
        g = torch.Generator(device="cuda").manual_seed(1)
        qkv = torch.randn((4, 24 * 37, 16, 128), generator=g, device="cuda").to(torch.bfloat16)
        cu, grown, pos = i32([37 * i for i in range(25)]), i32([37] * 24), i32(list(range(37)) * 24)
        out = []
        for _ in range(6):
            if wait:
                torch.cuda.synchronize()
            parts, kept, sums, _ = loop.step(qkv, cu, grown, pos, 37, True)
            out += [kept, sums, loop.lens.clone(), loop.table.clone()] + [t for p in parts for t in p]
        torch.cuda.synchronize()
        return out + [loop.weights, bits(loop.k), bits(loop.v)]

    want = play(True)
    for _ in range(3):
        got = play(False)
        assert all(torch.equal(x, y) for x, y in zip(want, got)) and len(want) == len(got)
