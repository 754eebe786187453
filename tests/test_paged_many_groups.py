"""Batches of more than 32 sequences whose new tokens fill several row groups: the join then
finds its parts through the table of units that the main kernel leaves, with groups."""
import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm

pytestmark = pytest.mark.gpu


def new_tokens(B, most):
    """Mostly none or one, some over one, two and all groups."""
    return [most if b % 19 == 4 else most // 2 + 3 if b % 13 == 7 else most // 4 if b % 11 == 3 else b % 3 == 0 for b in range(B)]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,most,H,Hkv,d,page,long", [
    (40, 200, 4, 2, 64, 16, 400), (33, 160, 4, 1, 128, 32, 900), (45, 140, 2, 1, 256, 16, 300), (64, 20, 32, 2, 128, 64, 700),
    (34, 12, 71, 1, 64, 16, 500), (50, 256, 4, 2, 128, 256, 60), (300, 9, 64, 1, 256, 16, 40),
])
def test_many_sequences_of_several_row_groups(B, most, H, Hkv, d, page, long, tree):
    G = H // Hkv
    rows = (128 // G) * (2 if d <= 128 else 1)
    assert B > 32 and most > rows  # tokens of a row group
    new = [int(x) for x in new_tokens(B, most)]
    lens = [long if b % 19 == 4 else (37 * b) % (long // 3 + 1) for b in range(B)]
    s = pm.Setup(lens, new, page, Hkv, d, seed=B + d, H=H)
    mask = seen = None
    if tree:
        mask, seen = pm.tree_masks(new, (most + 63) // 64, seed=d)
        mask = mask.cuda()
    o, lse = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, most, tree_mask=mask)
    again = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, most, tree_mask=mask)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    pm.check_attention(s, o, lse, pm.attention(s, s.q, seen), f"B {B} most {most} H{H}/{Hkv} d{d} tree={tree}")
