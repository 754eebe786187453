"""The torch helpers of the paged cache reach the library in two ways: through the binding
(the ordinary call) and through ctypes (a given stream, out, workspace, another device, no
binding).  Both accept and refuse the same calls and give the same results; and the given
workspaces and streams of every helper."""
import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm

pytestmark = pytest.mark.gpu


class Declines:
    def __getattr__(self, name):
        return lambda *a: None


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def setup(layers=None, d=128, seed=1):
    s = pm.Setup([40, 0, 17, 95], [9, 1, 0, 3], 16, 2, d, seed=seed, H=8, layers=layers, fill=0.5, spare=9)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s.k, s.v = (torch.randn((s.total, 2, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    return s


def append(s, **kw):
    fa.cache_append(s.k, s.v, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, **kw)
    return ()


def attend(s, **kw):
    kw = dict(dict(scale=None, tree_mask=None), **kw)
    return fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, 9, **kw)


def compact(s, **kw):
    return (fa.cache_compact(s.k_pages, s.v_pages, s.t_table, s.t_lens, i32([[0, 3, 8], [0, 0, 0], [0, 0, 0], [1, 2, 0]]),
                             i32([3, 1, 0, 2]), **kw),)


def fork(s, **kw):
    return (fa.cache_fork(s.t_refs, s.t_table, s.t_up, i32([1, 1, 0, -1]), 16, **kw),)


def resize(s, **kw):
    return fa.cache_resize(s.t_refs, s.k_pages, s.v_pages, s.t_table, s.t_up, i32([100, 1, 20, 90]), **kw)


CALLS = [("append", append, {}), ("attention", attend, {}), ("attention, trees", attend, dict(tree="9")),
         ("attention, scale", attend, dict(scale=0.25)), ("attention, scale as a whole number", attend, dict(scale=1)),
         ("compact", compact, {}), ("compact, layers", compact, dict(layers=3)), ("fork", fork, {}), ("resize", resize, {}),
         ("resize, layers", resize, dict(layers=2))]


def play(call, kw):
    kw = dict(kw)
    s = setup(kw.pop("layers", None))
    s.t_up = s.t_lens + i32(s.new)
    if kw.pop("tree", None):
        kw["tree_mask"] = pm.tree_masks(s.new, 1, seed=3)[0].cuda()
    out = call(s, **kw)
    torch.cuda.synchronize()
    return [x.clone() for x in (*out, s.k_pages, s.v_pages, s.t_table, s.t_refs)]


@pytest.mark.parametrize("what,call,kw", CALLS, ids=[c[0] for c in CALLS])
def test_both_ways_agree(monkeypatch, what, call, kw):
    want = play(call, kw)
    monkeypatch.setattr(fa, "_fast", Declines())
    got = play(call, kw)
    assert len(want) == len(got) and all(x.dtype == y.dtype and torch.equal(x, y) for x, y in zip(want, got))


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def pages(s, x):
    s.k_pages = s.v_pages = x
    if x.shape[0] != s.num_pages:
        s.t_refs = s.t_refs[: x.shape[0]]
    return []


BAD = {
    "pages of 24 rows": lambda s: pages(s, bf(9, 24, 2, 128)),
    "head dim 96": lambda s: pages(s, bf(9, 16, 2, 96)) + [setattr(s, n, getattr(s, n)[..., :96].contiguous())
                                                           for n in ("k", "v", "q")],
    "lengths of another batch": lambda s: setattr(s, "t_lens", s.t_lens[:3]) or setattr(s, "t_up", s.t_up[:3]),
    "tables of 64 bits": lambda s: setattr(s, "t_table", s.t_table.long()),
    "no sequences": lambda s: [setattr(s, n, x) for n, x in (("t_table", s.t_table[:0]), ("t_lens", s.t_lens[:0]),
                                                             ("t_up", s.t_up[:0]), ("t_cu", s.t_cu[:1]))],
    "no columns": lambda s: setattr(s, "t_table", s.t_table[:, :0]),
    "a misaligned page": lambda s: pages(s, bf(9 * 16 * 2 * 128 + 1)[1:].view(9, 16, 2, 128)),
    "lengths on the CPU": lambda s: [setattr(s, n, getattr(s, n).cpu()) for n in ("t_lens", "t_up")],
}


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("call", [append, attend, compact, fork, resize], ids=lambda c: c.__name__)
def test_both_ways_refuse_alike(monkeypatch, call, bad):
    def outcome():
        s = setup()
        s.t_up = s.t_lens + i32(s.new)
        BAD[bad](s)
        try:
            call(s)
        except (ValueError, fa.FaError) as e:
            return type(e), str(e)
        return None

    want = outcome()
    monkeypatch.setattr(fa, "_fast", Declines())
    assert outcome() == want
    if not (call is fork and bad in ("pages of 24 rows", "head dim 96", "a misaligned page")):  # it sees no pages
        assert want is not None


# ------------------------------------------------------------------ given streams and workspaces
@pytest.mark.parametrize("what,call,kw", CALLS, ids=[c[0] for c in CALLS])
@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_every_helper_on_a_given_stream(what, call, kw, kind):
    want = play(call, kw)
    side = torch.cuda.Stream()
    kw = dict(kw)
    s = setup(kw.pop("layers", None))
    s.t_up = s.t_lens + i32(s.new)
    if kw.pop("tree", None):
        kw["tree_mask"] = pm.tree_masks(s.new, 1, seed=3)[0].cuda()
    busy = torch.zeros(64 << 20, device="cuda")
    real = [(x, x.clone()) for x in (s.k, s.v, s.q)]
    for x, _ in real:
        x.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):  # the rows come last of all on that stream, and the call has to wait for them
        for _ in range(20):
            busy += 1
        for x, y in real:
            x.copy_(y)
    out = call(s, stream=side if kind == "stream" else side.cuda_stream, **kw)
    side.synchronize()
    got = [*out, s.k_pages, s.v_pages, s.t_table, s.t_refs]
    assert all(torch.equal(x, y) for x, y in zip(want, got)) and len(want) == len(got)


@pytest.mark.parametrize("max_new,H,Hkv,d", [(1, 8, 2, 128), (3, 4, 2, 64), (60, 8, 2, 128), (60, 4, 1, 256), (200, 4, 2, 64)])
def test_attention_with_a_given_workspace_and_outputs(max_new, H, Hkv, d):
    """The workspace may hold anything before and is not read past its size; too small a one is refused."""
    s = pm.Setup([900, 3, 0, 444], [max_new, 1, 0, max_new], 32, Hkv, d, seed=d, H=H)
    want = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, max_new)
    need = fa.fa_fwd_paged_workspace_bytes(s.B, max_new, H, Hkv, d)
    store = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    for junk in (0xFF, 0x7F, 0):
        store.fill_(junk)
        got = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, max_new, out=o, lse=lse,
                                     workspace=store[256 : 256 + need])
        assert got[0] is o and got[1] is lse and torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert (store[:256] == junk).all() and (store[256 + need :] == junk).all()
    for bad in (store[256 : 255 + need], store[16 : 16 + need], store[:0]):
        with pytest.raises(fa.FaError):
            fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, max_new, workspace=bad)
    with pytest.raises(ValueError):
        fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, max_new, workspace=store[::2])


@pytest.mark.parametrize("layers", [None, 3])
def test_resize_with_a_given_workspace(layers):
    want = play(resize, dict(layers=layers))
    need = fa.fa_cache_resize_workspace_bytes(4)
    store = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    got = play(resize, dict(layers=layers, workspace=store[256 : 256 + need]))
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert (store[:256] == 0xFF).all() and (store[256 + need :] == 0xFF).all()
    for bad in (store[256 : 255 + need], store[16 : 16 + need], store[:0]):
        with pytest.raises(fa.FaError):
            play(resize, dict(workspace=bad))


def test_two_graphs_share_workspaces():
    """Two captured calls on one workspace, replayed in turn on other contents."""
    s = [pm.Setup([700, 33], [9, 20], 32, 2, 128, seed=30 + i, H=8) for i in range(2)]
    need = fa.fa_fwd_paged_workspace_bytes(2, 20, 8, 2, 128)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def call(x):
        return fa.attention_fwd_paged(x.q, x.k_pages, x.v_pages, x.t_table, x.t_lens, x.t_cu, 20, workspace=ws)

    call(s[0])
    torch.cuda.synchronize()
    graphs, out = [], []
    for x in s:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out.append(call(x))
        graphs.append(g)
    for i in range(4):
        for x in s:
            x.q.copy_(torch.randn(x.q.shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda"))
        for g in graphs:
            g.replay()
        for x, (o, lse) in zip(s, out):
            want = fa.attention_fwd_paged(x.q, x.k_pages, x.v_pages, x.t_table, x.t_lens, x.t_cu, 20)
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
