"""Gradients of key preparation hold numbers: the comparison with the 64-bit form asks whether an error lies past its
bound, which a NaN does not, so every case of it is run here with a look at the values too."""
import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import rope_model as rm
import test_cache_edges as edges
import test_rope as tr

compare = rm.check_backward


def check_backward(dx, dw, *rest, what="", **kw):
    """rope_model's comparison, and no NaN or infinity in dx or dw."""
    assert torch.isfinite(dx).all(), f"{what}: dx holds {int((~torch.isfinite(dx)).sum())} values that are no numbers"
    assert dw is None or torch.isfinite(dw).all(), f"{what}: dw holds {int((~torch.isfinite(dw)).sum())} values that are no numbers"
    compare(dx, dw, *rest, what=what, **kw)


@pytest.fixture
def strict(monkeypatch):
    monkeypatch.setattr(rm, "check_backward", check_backward)


@pytest.mark.parametrize("weight", [False, True])
def test_the_check_takes_right_gradients_and_no_others(weight):
    g = torch.Generator().manual_seed(1)
    dy, x = (torch.randn((7, 3, 64), generator=g, dtype=torch.float64).to(torch.bfloat16) for _ in range(2))
    w = torch.rand(64, generator=g) + 0.5 if weight else None
    angle = rm.angles(torch.arange(7), 10000.0 ** (-torch.arange(0, 64, 2) / 64.0), None)
    x64 = x.double().requires_grad_()
    w64 = None if w is None else w.double().requires_grad_()
    ins = [x64] if w is None else [x64, w64]
    got = torch.autograd.grad(rm.forward(x64, w64, angle, False), ins, dy.double())
    dx, dw = got[0].to(torch.bfloat16), got[1].float() if weight else None
    check_backward(dx, dw, dy, x, w, angle, False)
    for bad in (float("nan"), float("inf"), 1e3):
        wrong = dx.clone()
        wrong[3, 1, 5] = bad
        with pytest.raises(AssertionError):
            check_backward(wrong, dw, dy, x, w, angle, False)
        if weight:
            wrong = dw.clone()
            wrong[11] = bad
            with pytest.raises(AssertionError):
                check_backward(dx, wrong, dy, x, w, angle, False)


@pytest.mark.gpu
@pytest.mark.parametrize("case", tr.CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items() if k != "axes"))
def test_backward(case, strict):
    tr.Case(**case).check_bwd()


@pytest.mark.gpu
def test_far_positions(strict):
    tr.test_angles_are_exact_at_any_position()


@pytest.mark.gpu
def test_zeros_and_the_largest_values(strict):
    tr.test_rows_of_zeros_and_of_the_largest_values()


@pytest.mark.gpu
@pytest.mark.parametrize("pairs", [False, True])
def test_strides(pairs, strict):
    edges.test_strides_of_every_kind(pairs)


@pytest.mark.gpu
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("d,H,Hkv", [(64, 5, 3), (64, 9, 1), (128, 5, 3), (128, 3, 1), (256, 3, 1), (256, 1, 3)])
def test_lanes_without_a_head_keep_what_they_hold_to_themselves(d, H, Hkv, pairs, strict):
    """Heads that do not fill a warp's step, after a call that leaves NaN in every place a lane may have kept."""
    per = 32 // (d // 16)
    before = tr.Case((3000,), 4 * per, 4 * per, d, pairs=pairs)
    before.gq[:], before.gk[:], before.q[:], before.k[:] = (float("nan"),) * 4
    c = tr.Case((901,), H, Hkv, d, pairs=pairs, fused=True)
    for _ in range(3):
        before.backward()
        dq, dk, dwq, dwk = c.backward()
        torch.cuda.synchronize()
        rm.check_backward(dq, dwq, c.gq, c.q, c.qw, c.angle, pairs, what="q")
        rm.check_backward(dk, dwk, c.gk, c.k, c.kw, c.angle, pairs, what="k")
