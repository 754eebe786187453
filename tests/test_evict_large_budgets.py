"""Eviction with the largest numbers its arguments hold: a budget that means "no limit", and rows of sums with
room for 2^31 - 1 places."""
import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm
from test_evict import bits, check, model, sums

pytestmark = pytest.mark.gpu

MOST = 2**31 - 1


def left_alone(s, w, keep):
    """A call that no sequence is long enough for: everything as it was, kept the places there are and then -1."""
    k, v, before = s.k_pages.clone(), s.v_pages.clone(), w.clone()
    lens, kept = fa.cache_evict(s.t_refs, s.k_pages, s.v_pages, s.t_table, s.t_lens, w, keep, 7)
    torch.cuda.synchronize()
    assert lens.tolist() == s.lens and kept.shape == (s.B, s.Hkv, keep)
    for b, a in enumerate(s.lens):
        assert (kept[b, :, :a] == torch.arange(a, dtype=torch.int32, device="cuda")).all()
        for h in range(s.Hkv):
            for at in range(a, keep, 2**28):  # a piece at a time
                assert (kept[b, h, at : at + 2**28] == -1).all(), (b, h, at)
    assert torch.equal(bits(k), bits(s.k_pages)) and torch.equal(bits(v), bits(s.v_pages)) and torch.equal(w, before)


@pytest.mark.parametrize("keep", [MOST, MOST - 1, MOST - 1023, MOST - 1024, 2**30 + 1])
def test_a_budget_without_limit(keep):
    """The steps over kept pass 2^31 - 1 behind its end (8.6 GB)."""
    s = pm.Setup([40], [0], 16, 1, 64, seed=1)
    left_alone(s, sums(s, 50), keep)


def test_a_budget_without_limit_in_clusters():
    """Sums of 4096 places and more are looked at by clusters of 8 blocks: their step is 8192."""
    s = pm.Setup([40], [0], 16, 1, 64, seed=1)
    left_alone(s, sums(s, 5000), MOST)


@pytest.mark.parametrize("places", [MOST, MOST - 3, 2**30])
def test_sums_with_room_for_any_number_of_places(places):
    s = pm.Setup([100], [0], 16, 1, 64, seed=2)
    w = torch.zeros((1, 1, places), device="cuda")
    few = sums(s, 120)
    w[..., :120] = few
    want = model(s, few, 30, 4)
    lens, kept = fa.cache_evict(s.t_refs, s.k_pages, s.v_pages, s.t_table, s.t_lens, w, 30, 4)
    torch.cuda.synchronize()
    assert lens.tolist() == want[3] and torch.equal(kept.cpu(), want[4]) and torch.equal(w[..., :120].cpu(), want[2])
    for at in range(120, places, 2**28):
        assert (w[..., at : at + 2**28] == 0).all()
    assert torch.equal(bits(s.k_pages.cpu()), bits(want[0])) and torch.equal(bits(s.v_pages.cpu()), bits(want[1]))


def test_ordinary_budgets_are_as_they_were():
    s = pm.Setup([300, 17], [0, 0], 16, 2, 64, seed=3)
    check(s, sums(s, 310), 299, 20)
