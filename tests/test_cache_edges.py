"""Key preparation, weight sums and eviction where sizes and orders are unusual: pools past 2^32
elements, scores far apart, calls on two streams at once, odd strides, many sequences."""
import math

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm
import rope_model as rm
from test_evict import model as evict_model
from test_weights import check as check_weights
from test_weights import reference as weights_reference

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(x):
    return x.view(torch.int16)


def test_pools_past_32_bits():
    """A pool of 2^32 + elements (8.9 GB each for keys and values), whose last pages are the sequence's."""
    page, Hkv, d, H = 256, 8, 128, 16
    num = 2**32 // (page * Hkv * d) + 400
    k, v = (torch.empty((num, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2**32
    order = [num - 1, 3, num - 2, num - 3]
    g = torch.Generator(device="cuda").manual_seed(1)
    for p in order:
        k[p].normal_(generator=g), v[p].normal_(generator=g)
    s = pm.Setup([1], [0], 16, 1, 64, seed=1)  # its books; the cache is the one above
    s.lens, s.new, s.page, s.Hkv, s.d, s.B, s.table, s.num_pages = [900], [20], page, Hkv, d, 1, [order], num
    s.total, s.cu = 20, [0, 20]
    table, lens, cu = i32([order]), i32([900]), i32([0, 20])
    x = torch.randn((20, H + 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    f = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    q, kn, vn = x.split([H, Hkv, Hkv], 1)
    q = fa.cache_append_rope(q, kn, vn, k, v, table, lens, cu, f)
    angle = rm.angles(900 + torch.arange(20), f.cpu(), None)
    for i in (0, 19):
        p, r = s.place(0, 900 + i)
        rm.check_forward(k[p, r][None], kn[i : i + 1], None, angle[i : i + 1], False, what=f"token {i}")
        assert torch.equal(v[p, r], vn[i])
    rm.check_forward(q, x[:, :H], None, angle, False, what="q")
    _, lse = fa.attention_fwd_paged(q, k, v, table, lens, cu, 20)
    w = torch.zeros((1, Hkv, 1024), device="cuda")
    before = w.clone()
    fa.attention_weights_paged(q, k, table, lens, cu, 20, lse, w)
    # the model sees the sequence's own pages only
    small = pm.Setup([1], [0], 16, 1, 64, seed=1)
    small.__dict__.update(s.__dict__)
    small.table, small.num_pages = [[0, 1, 2, 3]], 4
    small.k_pages, small.v_pages = k[order], v[order]
    check_weights(small, w, weights_reference(small, q, lse, before), before, "large pool")
    refs = torch.zeros(num, dtype=torch.int32, device="cuda")
    refs[order] = 1
    small.lens, small.new = [920], [0]
    want = evict_model(small, w, 300, 30)
    got = w.clone()
    lens, kept = fa.cache_evict(refs, k, v, table, i32([920]), got, 300, 30)
    assert lens.tolist() == [300] and torch.equal(kept.cpu(), want[4]) and torch.equal(got.cpu(), want[2])
    assert torch.equal(bits(k[order].cpu()), bits(want[0])) and torch.equal(bits(v[order].cpu()), bits(want[1]))


@pytest.mark.parametrize("new,H,Hkv,d", [([40, 9], 8, 2, 128), ([256], 8, 2, 64), ([256, 30], 4, 1, 256), ([3, 1], 8, 2, 128)])
@pytest.mark.parametrize("spread", [1.0, 12.0, 60.0])
def test_rows_whose_scores_lie_far_apart(new, H, Hkv, d, spread):
    """Rows with lse of very different sizes meet in one set of rows: up to 2^64 apart they share a base, past it each
    has its own."""
    s = pm.Setup([700, 30][: len(new)], new, 32, Hkv, d, seed=21, H=H)
    grow = torch.logspace(0, math.log10(spread), s.total).to(torch.bfloat16).cuda()
    s.q *= grow[torch.randperm(s.total, generator=torch.Generator().manual_seed(1)).cuda(), None, None]
    _, lse = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, max(new))
    w = torch.rand((s.B, Hkv, 1000), device="cuda")
    before = w.clone()
    fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, max(new), lse, w)
    check_weights(s, w, weights_reference(s, s.q, lse, before), before, f"spread {spread}")


@pytest.mark.parametrize("lse", [float("-inf"), float("inf"), float("nan")])
def test_lse_that_is_not_finite(lse):
    """-inf: the token saw nothing and gives nothing; inf: e^(s - inf) is 0; NaN: NaN for its own places only."""
    s = pm.Setup([300, 40], [40, 40], 32, 2, 128, seed=2, H=8)
    _, real = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, 40)
    one = real.clone()
    one[2, 5] = lse  # token 5 of the first sequence, kv head 0
    w = torch.zeros((2, 2, 340), device="cuda")
    before = w.clone()
    fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, 40, one, w)
    clean = torch.zeros_like(w)
    fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, 40, real, clean)
    assert torch.equal(w[1], clean[1]) and torch.equal(w[0, 1], clean[0, 1])
    if math.isnan(lse):
        assert torch.isnan(w[0, 0, :306]).all() and torch.isfinite(w[0, 0, 306:]).all()
    else:
        one[2, 5] = float("-inf")
        check_weights(s, w, weights_reference(s, s.q, one, before), before, f"lse {lse}")


@pytest.mark.parametrize("B", [1, 32, 33, 128, 129, 1500])
def test_many_sequences(B):
    r = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 60, (B,), generator=r).tolist()
    new = torch.randint(0, 4, (B,), generator=r).tolist()
    new[0] = 3
    s = pm.Setup(lens, new, 16, 1, 64, seed=B, H=2)
    _, lse = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, 3)
    w = torch.rand((B, 1, 70), device="cuda")
    before = w.clone()
    fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, 3, lse, w, decay=0.5)
    check_weights(s, w, weights_reference(s, s.q, lse, before, decay=0.5), before, f"{B} sequences")


def test_calls_on_two_streams_at_once():
    """The same operators on other data, side by side: nothing is shared between calls."""
    def make(seed):
        s = pm.Setup([3000, 800], [40, 3], 32, 4, 128, seed=seed, H=16, fill=0.5)
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn((3000, 24, 128), generator=g, device="cuda").to(torch.bfloat16)
        f = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).float().cuda()
        pos = torch.arange(3000, dtype=torch.int32, device="cuda")
        weight = torch.rand(128, generator=g, device="cuda")
        lse = torch.rand((16, 43), generator=g, device="cuda") + 8
        w = torch.rand((2, 4, 3100), generator=g, device="cuda")
        q, k, _ = x.split([16, 4, 4], 1)

        def run():
            out = list(fa.qk_norm_rope(q, k, pos, f, q_weight=weight, k_weight=weight))
            out += fa.qk_norm_rope_bwd(q, k, q, k, pos, f, q_weight=weight, k_weight=weight)
            sums = w.clone()
            fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, 40, lse, sums)
            kp, vp = s.k_pages.clone(), s.v_pages.clone()
            return out + [sums.clone(), *fa.cache_evict(s.t_refs, kp, vp, s.t_table, s.t_lens, sums, 500, 16), kp, vp, sums]

        return run

    runs = [make(1), make(2)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for run, stream in zip(runs, streams):
            with torch.cuda.stream(stream):
                got.append(run())
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert all(torch.equal(a.float(), b.float()) for a, b in zip(x, y)) and len(x) == len(y)


def test_two_graphs_replayed_in_turn():
    """Two captured backward passes, each with a workspace from its own graph's memory."""
    f = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).float().cuda()
    pos = torch.arange(500, dtype=torch.int32, device="cuda")
    data, graphs, out, want = [], [], [], []
    for seed in range(2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        q, k, gq, gk = (torch.randn((500, n, 128), generator=g, device="cuda").to(torch.bfloat16) for n in (8, 2, 8, 2))
        w = torch.rand(128, generator=g, device="cuda")
        call = lambda q=q, k=k, gq=gq, gk=gk, w=w: fa.qk_norm_rope_bwd(gq, gk, q, k, pos, f, q_weight=w, k_weight=w)
        want.append([x.clone() for x in call()])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out.append(call())
        graphs.append(graph)
        data.append((q, k, gq, gk, w))
    for _ in range(3):
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, out):
            assert all(torch.equal(a, b) for a, b in zip(x, y))


@pytest.mark.parametrize("pairs", [False, True])
def test_strides_of_every_kind(pairs):
    """Heads before tokens, every second head, tokens far apart, one token for all, a batch of one token each."""
    g = torch.Generator(device="cuda").manual_seed(3)
    f = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()
    w = torch.rand(64, generator=g, device="cuda") + 0.5
    big = torch.randn((9, 12, 70, 64), generator=g, device="cuda").to(torch.bfloat16)
    for q, k in ((big[0].transpose(0, 1), big[1, :3].transpose(0, 1)), (big[:, ::2, 5], big[:, 1::3, 6]),
                 (big[:, :, ::10].transpose(1, 2)[:1], big[:1, 3:5, ::10].transpose(1, 2)), (big[2, 0, :1].expand(30, 1, 64),
                 big[2, 0, :1].expand(30, 1, 64)), (big[:, 3:4, :5], big[:, 4:5, 5:7])):
        lead = q.shape[:-2]
        pos = torch.arange(lead.numel(), dtype=torch.int32, device="cuda").reshape(lead) * 37
        angle = rm.angles(pos.cpu(), f.cpu(), None)
        got = fa.qk_norm_rope(q, k, pos, f, q_weight=w, interleaved=pairs)
        rm.check_forward(got[0], q, w, angle, pairs, what=f"q {q.stride()}")
        rm.check_forward(got[1], k, None, angle, pairs, what=f"k {k.stride()}")
        grads = fa.qk_norm_rope_bwd(q, k, q, k, pos, f, k_weight=w, interleaved=pairs)
        rm.check_backward(grads[0], grads[2], q, q, None, angle, pairs, what=f"dq {q.stride()}")
        rm.check_backward(grads[1], grads[3], k, k, w, angle, pairs, what=f"dk {k.stride()}")


def test_misaligned_views_are_refused():
    x = torch.zeros((10, 8, 72), dtype=torch.bfloat16, device="cuda")
    f = torch.ones(16, device="cuda")
    pos = torch.arange(10, dtype=torch.int32, device="cuda")
    good = torch.zeros((10, 2, 64), dtype=torch.bfloat16, device="cuda")
    fa.qk_norm_rope(x[:, :, 8:], good, pos, f)  # heads 144 bytes apart
    for bad in (x[:, :, 1:65], torch.zeros((10, 8, 68), dtype=torch.bfloat16, device="cuda")[..., :64]):
        with pytest.raises(fa.FaError) as e:
            fa.qk_norm_rope(bad, good, pos, f)
        assert e.value.status == fa.FA_ERR_ALIGNMENT


