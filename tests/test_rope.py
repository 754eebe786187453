"""Norms of queries and keys with the rotation by positions, forward and backward, against
64-bit forms: head dims, partly rotated heads, both kinds of pairs, several axes, views
into a projection's output, odd sizes, far positions, values that are not finite."""
import math

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import rope_model as rm

pytestmark = pytest.mark.gpu


class Case:
    """Random rows and tables; lead: (total,) or (B, N)."""

    def __init__(self, lead, H, Hkv, d, rot=None, norm="float32", axes=None, pairs=False, fused=False, first=0, seed=0,
                 which="qk"):
        g = torch.Generator().manual_seed(seed + d + H)
        rot = d if rot is None else rot
        x = torch.randn(lead + (H + 2 * Hkv, d), generator=g).to(torch.bfloat16).cuda()
        grads = torch.randn(lead + (H + 2 * Hkv, d), generator=g).to(torch.bfloat16).cuda()
        self.q, self.k, self.v = x.split([H, Hkv, Hkv], -2)
        self.gq, self.gk, _ = grads.split([H, Hkv, Hkv], -2)
        if not fused:
            self.q, self.k, self.v, self.gq, self.gk = (t.contiguous() for t in (self.q, self.k, self.v, self.gq, self.gk))
        self.inv_freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
        total = math.prod(lead)
        pos = first + torch.arange(total).reshape(lead)
        self.axes = axes
        if axes is not None:
            pos = torch.stack([pos, pos // 3 - 5, -pos, pos * 7 % 11][: max(axes) + 1])
        self.positions = pos.to(torch.int32).cuda()
        weight = lambda n: (1 + 0.3 * torch.randn(d, generator=g)).to(getattr(torch, norm)).cuda() if norm and n in which else None
        self.qw, self.kw = weight("q"), weight("k")
        self.pairs = pairs
        self.angle = rm.angles(self.positions.cpu(), self.inv_freq.cpu(), axes)

    def kw_args(self):
        return dict(q_weight=self.qw, k_weight=self.kw, axes=self.axes, interleaved=self.pairs)

    def forward(self, **kw):
        return fa.qk_norm_rope(self.q, self.k, self.positions, self.inv_freq, **self.kw_args(), **kw)

    def backward(self, **kw):
        return fa.qk_norm_rope_bwd(self.gq, self.gk, self.q, self.k, self.positions, self.inv_freq, **self.kw_args(), **kw)

    def check(self, what=""):
        q, k = self.forward()
        torch.cuda.synchronize()
        rm.check_forward(q, self.q, self.qw, self.angle, self.pairs, what=f"{what} q")
        rm.check_forward(k, self.k, self.kw, self.angle, self.pairs, what=f"{what} k")
        assert q.is_contiguous() and k.is_contiguous()

    def check_bwd(self, what=""):
        dq, dk, dwq, dwk = self.backward()
        torch.cuda.synchronize()
        rm.check_backward(dq, dwq, self.gq, self.q, self.qw, self.angle, self.pairs, what=f"{what} q")
        rm.check_backward(dk, dwk, self.gk, self.k, self.kw, self.angle, self.pairs, what=f"{what} k")


def runs(half, n):  # a run of pairs for each of n axes
    return tuple(i * n // half for i in range(half))


CASES = [
    dict(lead=(1,), H=1, Hkv=1, d=64),
    dict(lead=(1,), H=32, Hkv=8, d=128, norm="bfloat16"),
    dict(lead=(7,), H=5, Hkv=3, d=64, rot=32, pairs=True),
    dict(lead=(33,), H=9, Hkv=1, d=128, rot=16, norm=""),
    dict(lead=(33,), H=9, Hkv=1, d=128, rot=112, norm="bfloat16", fused=True, first=131072),
    dict(lead=(3, 41), H=16, Hkv=4, d=128, axes=runs(64, 3), fused=True),
    dict(lead=(3, 41), H=6, Hkv=2, d=256, rot=64, which="k", axes=tuple(i % 4 for i in range(32)), pairs=True),
    dict(lead=(1, 50), H=4, Hkv=2, d=256, pairs=True, fused=True, which="q", first=2**31 - 60),
    dict(lead=(50, 1), H=4, Hkv=4, d=256, norm="", fused=True, first=-(2**31)),
    dict(lead=(1500,), H=16, Hkv=16, d=128, axes=runs(64, 2)),
    dict(lead=(777,), H=71, Hkv=1, d=64, rot=48, pairs=True, norm="bfloat16", fused=True),
    dict(lead=(3001,), H=17, Hkv=2, d=256, rot=240),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items() if k != "axes"))
def test_forward(case):
    Case(**case).check()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items() if k != "axes"))
def test_backward(case):
    Case(**case).check_bwd()


def test_angles_are_exact_at_any_position():
    """Frequencies of every size, negative and zero ones among them, against 64 bits; a position of 2^31 turns by up to
    2^31 f radians, whose fraction has to be right."""
    c = Case((40,), 2, 1, 64, norm="")
    c.inv_freq = torch.tensor([1.0, 0.0, -1.0, 3.0, 1e-3, 1e-9, 1e-30, 1e-41, 0.5, 6.2831855, 100.0, 1000.5, 0.1, 0.3, 0.7, 0.9]
                              + [2.0**-i for i in range(16)], dtype=torch.float32, device="cuda")
    pos = [0, 1, -1, 2**31 - 1, -(2**31), 2**24 + 1, 12345678, 99999999] + [int(1.7**i) for i in range(32)]
    c.positions = torch.tensor(pos, dtype=torch.int32, device="cuda")
    c.angle = rm.angles(c.positions.cpu(), c.inv_freq.cpu(), None)
    c.check()
    c.check_bwd()


def test_gradients_against_differences():
    """The loss <G, forward(x, w)> in 64 bits, differenced along random directions, against the kernel's gradients."""
    c = Case((40,), 4, 2, 128, rot=64, pairs=True, axes=runs(32, 3), fused=True)
    dq, dk, dwq, dwk = c.backward()
    g = torch.Generator().manual_seed(3)
    for x, w, dy, dx, dw in ((c.q, c.qw, c.gq, dq, dwq), (c.k, c.kw, c.gk, dk, dwk)):
        x, w, dy = x.cpu().double(), w.cpu().double(), dy.cpu().double()
        loss = lambda x, w: (rm.forward(x, w, c.angle, c.pairs) * dy).sum()
        for i in range(4):
            vx, vw = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(w.shape, generator=g, dtype=torch.float64)
            h = 1e-5  # the difference's own error is of the order h^2 and 2^-52 / h
            want = (loss(x + h * vx, w) - loss(x - h * vx, w)) / (2 * h)
            size = (dx.cpu().double() * vx).norm()
            got = (dx.cpu().double() * vx).sum()
            assert abs(got - want) <= 2.0**-8 * 6 * size, (i, float(got), float(want))  # independent roundings: 6 sigma
            want = (loss(x, w + h * vw) - loss(x, w - h * vw)) / (2 * h)
            assert abs((dw.cpu().double() * vw).sum() - want) <= 1e-5 * (dw.cpu().double() * vw).abs().sum() + 1e-6 * abs(want)


@pytest.mark.parametrize("pairs", [False, True])
def test_columns_that_are_not_rotated_and_other_rows_keep_their_values(pairs):
    c = Case((30,), 4, 2, 128, rot=64, norm="", pairs=pairs)
    clean = c.forward()
    odd = [(3, 1, 100, float("inf")), (4, 0, 127, float("nan")), (5, 3, 64, float("-inf")), (9, 2, 5, float("nan"))]
    for t, h, col, x in odd:
        c.q[t, h, col] = x
    q, k = c.forward()
    assert torch.equal(k, clean[1])
    for t, h, col, x in odd[:3]:
        assert torch.equal(torch.isnan(q[t, h, col]).cpu(), torch.tensor(math.isnan(x))) and (math.isnan(x) or q[t, h, col] == x)
        clean[0][t, h, col] = q[t, h, col] = 0
    assert torch.isnan(q[9, 2, 5])
    pair = [5, 4] if pairs else [5, 37]
    clean[0][9, 2, pair] = 0
    q[9, 2, pair] = 0
    assert torch.equal(q, clean[0])


def test_a_row_that_is_not_finite_stays_alone():
    c = Case((30,), 4, 2, 64, fused=True)
    clean, cleaner = c.forward(), c.backward()
    c.q[7, 2, 11] = float("nan")
    q, k = c.forward()
    assert torch.isnan(q[7, 2]).all()
    q[7, 2] = clean[0][7, 2]
    assert torch.equal(q, clean[0]) and torch.equal(k, clean[1])
    dq, dk, dwq, dwk = c.backward()
    assert torch.isnan(dq[7, 2]).all() and torch.isnan(dwq).all()
    dq[7, 2] = cleaner[0][7, 2]
    assert torch.equal(dq, cleaner[0]) and torch.equal(dk, cleaner[1]) and torch.equal(dwk, cleaner[3])


def test_rows_of_zeros_and_of_the_largest_values():
    """eps keeps rows of zeros at zero; the squares of values up to 2^60 stay inside fp32."""
    c = Case((8,), 2, 1, 64)
    c.q[:4] = 0
    c.k[:] = c.k * 2.0**60
    c.check()
    assert (c.forward()[0][:4] == 0).all()
    c.check_bwd()


def test_in_place_and_given_outputs():
    c = Case((2, 90), 6, 2, 128, rot=96)
    want = c.forward()
    q, k = c.q.clone(), c.k.clone()
    got = fa.qk_norm_rope(q, k, c.positions, c.inv_freq, **c.kw_args(), q_out=q, k_out=k)
    assert got[0] is q and got[1] is k and torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_no_tokens():
    c = Case((0,), 4, 2, 64)
    q, k = c.forward()
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    dq, dk, dwq, dwk = c.backward()
    assert dq.shape == (0, 4, 64) and (dwq == 0).all() and (dwk == 0).all() and dwq.shape == (64,)


def test_gradients_are_reproducible_and_the_workspace_may_hold_anything():
    c = Case((4000,), 16, 4, 128, fused=True)
    want = c.backward()
    need = fa.fa_qk_norm_rope_bwd_workspace_bytes(128)
    store = torch.empty(need + 512, dtype=torch.uint8, device="cuda")
    for junk in (0xFF, 0x7F, 0):
        store.fill_(junk)
        got = c.backward(workspace=store[256 : 256 + need])
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        assert (store[:256] == junk).all() and (store[256 + need :] == junk).all()
    for bad in (store[256 : 255 + need], store[16 : 16 + need], store[:0]):
        with pytest.raises(fa.FaError):
            c.backward(workspace=bad)


@pytest.mark.parametrize("which", ["", "q", "k"])
def test_rows_without_a_norm_need_no_inputs(which):
    c = Case((20,), 4, 2, 64, which=which)
    want = c.backward()
    q, k = (c.q if "q" in which else None), (c.k if "k" in which else None)
    got = fa.qk_norm_rope_bwd(c.gq, c.gk, q, k, c.positions, c.inv_freq, **c.kw_args())
    for x, y in zip(want, got):
        assert (x is None and y is None) or torch.equal(x, y)
    assert (got[2] is None) == ("q" not in which) and (got[3] is None) == ("k" not in which)


def test_training_step():
    """Norm and rotation, attention and both backward passes, against 64-bit automatic differentiation."""
    B, N, H, Hkv, d = 2, 150, 4, 2, 64
    c = Case((B, N), H, Hkv, d, rot=32, fused=True)
    v = c.v.contiguous()
    dO = torch.randn((B, N, H, d), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()

    def step():
        q, k = c.forward()
        o, lse = fa.attention_fwd(q, k, v, causal=True)
        dq, dk, dv = fa.attention_bwd(q, k, v, o, lse, dO, causal=True)
        return (o, dv) + fa.qk_norm_rope_bwd(dq, dk, c.q, c.k, c.positions, c.inv_freq, **c.kw_args())

    got = step()
    ins = [t.detach().cpu().double().requires_grad_() for t in (c.q, c.k, v, c.qw, c.kw)]
    q, k = rm.forward(ins[0], ins[3], c.angle, False), rm.forward(ins[1], ins[4], c.angle, False)
    s = torch.einsum("bihd,bjhd->bhij", q, k.repeat_interleave(H // Hkv, 2)) / math.sqrt(d)
    s = s.masked_fill(torch.ones(N, N).triu(1).bool(), float("-inf"))
    o = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), ins[2].repeat_interleave(H // Hkv, 2))
    grads = torch.autograd.grad(o, ins, dO.cpu().double())
    o = o.detach()
    for name, x, y in (("o", got[0], o), ("dv", got[1], grads[2]), ("dq", got[2], grads[0]), ("dk", got[3], grads[1]),
                       ("dq_weight", got[4], grads[3]), ("dk_weight", got[5], grads[4])):
        rel = float((x.cpu().double() - y).norm() / y.norm())
        # q, k, o, dq, dk rounded to bf16 on the way and the weights in P V: each 2^-8 at most, one after another
        assert rel <= 6 * 2.0**-8, (name, rel)
    # captured, while results of an eager step are held, and replayed on other inputs
    c.forward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    c.q.copy_(torch.roll(c.q, 1, 1))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [x.clone() for x in out]
    assert all(torch.equal(x, y) for x, y in zip(replayed, step()))
