"""Weight sums where each weight is known to nearly 32 bits: rows of one set whose lse lie far apart must not cost
one another accuracy."""
import math

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm

pytestmark = pytest.mark.gpu

LSE, PLACES = 0.37, 1500


@pytest.mark.parametrize("new,H,Hkv,d", [(33, 1, 1, 64), (20, 8, 2, 128), (128, 1, 1, 128), (36, 1, 1, 256), (200, 2, 1, 64)])
@pytest.mark.parametrize("spread", [0.0, 3.9, 7.9, 8.1, 16.0, 40.0, 63.5, 63.9, 64.5, 100.0, -7.9, -40.0, -63.5])
def test_a_row_keeps_its_accuracy_beside_others(spread, new, H, Hkv, d):
    """One row of each kv head gives a place its weight, all others give nothing (a score of -100), and the last token's
    lse lies `spread` above or below (in powers of two).  Scores are sums of two products with 21 bits in all: exact.

    The weight's error, relative: scale log2(e) rounded, |z| 2^-24 with |z| < 1.1; the exponent's argument below 8 (its
    row's own below 2, a base at most 4 away), 2^-22 ln 2; 2^x, 2^-22 each for the weight and for its factor; the
    factor's rounding twice and the sum's once, 2^-24 each; with the others' terms below 2^-70 of it the sum of all of them
    adds no more.  In all (1.1 / 4 + 0.7 + 2 + 3 / 4) 2^-22 < 2^-20."""
    s = pm.Setup([PLACES], [new], 64, Hkv, d, seed=1, H=H)
    g = torch.Generator().manual_seed(int(abs(spread) * 10) + d)
    # z - lse in powers of two from -2 to -0.6, in steps of 2^-19
    z = ((LSE - math.log(2) * (0.6 + 1.4 * torch.rand((PLACES, Hkv), generator=g, dtype=torch.float64))) * 2.0**19).round() / 2.0**19
    coarse = (z * 2.0**7).round() / 2.0**7
    keys = torch.zeros((PLACES, Hkv, d), dtype=torch.float64)
    keys[..., 0], keys[..., 1], keys[..., 2] = coarse, (z - coarse) * 2.0**4, 1.0
    keys = keys.to(torch.bfloat16)
    q = torch.zeros((new, H, d), dtype=torch.bfloat16)
    q[..., 2] = -100.0
    first = torch.arange(0, H, H // Hkv)  # the first head of each group, of the first token
    q[0, first, 2], q[0, first, 0], q[0, first, 1] = 0.0, 1.0, 2.0**-4
    lse = torch.full((H, new), LSE)
    lse[:, -1] += spread * math.log(2)
    at = torch.tensor([s.place(0, p)[0] * s.page + s.place(0, p)[1] for p in range(PLACES + new)])
    pool = s.k_pages.cpu()
    pool.view(-1, Hkv, d)[at[:PLACES]] = keys
    pool.view(-1, Hkv, d)[at[PLACES:]] = 0  # the new tokens' own places, which are not looked at here
    s.k_pages = pool.cuda()
    w = torch.zeros((1, Hkv, PLACES + new), device="cuda")
    fa.attention_weights_paged(q.cuda(), s.k_pages, s.t_table, s.t_lens, s.t_cu, new, lse.cuda(), w, decay=0.0, scale=1.0)
    torch.cuda.synchronize()
    k64, q64 = keys.double(), q.double()
    assert torch.equal(k64[..., 0] + k64[..., 1] * 2.0**-4, (keys[..., 0].float() + keys[..., 1].float() * 2.0**-4).double())
    scores = torch.einsum("ihgd,phd->pihg", q64.view(new, Hkv, H // Hkv, d), k64)
    own = torch.exp(scores - lse.double().t().view(new, Hkv, H // Hkv)[None])
    want = own.sum((1, 3)).t()  # [Hkv, PLACES]
    rel = ((w[0, :, :PLACES].cpu().double() - want) / want).abs()
    assert float(rel.max()) <= 2.0**-20, f"{float(rel.max()):.3e} relative at a spread of {spread}"
