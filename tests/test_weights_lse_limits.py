"""Weight sums of rows that are left out by their lse (minus or plus infinity), whatever their scores are."""
import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm
from test_weights import check, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("grow", [1.0, 64.0, 4096.0])
@pytest.mark.parametrize("lse", [float("-inf"), float("inf")])
@pytest.mark.parametrize("new,H,Hkv,d", [([40, 40], 8, 2, 128), ([64, 1], 8, 2, 128), ([200, 50], 4, 2, 64), ([30, 9], 8, 1, 256),
                                         ([3, 2], 8, 2, 128)])
def test_rows_left_out_may_have_any_score(new, H, Hkv, d, lse, grow):
    """-inf: nothing; inf: e^(s - inf) is 0.  With q grown by 64 scores reach e^190 and more, past fp32 beside the lse
    of the other rows."""
    s = pm.Setup([300, 90], new, 32, Hkv, d, seed=2, H=H)
    _, real = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, max(new))
    for head, token in ((2, 1), (H - 1, new[0] - 1)):
        s.q[token, head] *= grow
        real[head, token] = lse
    w = torch.rand((2, Hkv, 300 + max(new)), device="cuda")
    before = w.clone()
    fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, max(new), real, w)
    left_out = torch.where(torch.isinf(real), float("-inf"), real)
    check(s, w, reference(s, s.q, left_out, before), before, f"lse {lse}, scores times {grow}")
