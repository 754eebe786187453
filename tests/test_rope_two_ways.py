"""The helpers of key preparation, weight sums and eviction refuse the same calls, in the same
words, through the binding and without it."""
import pytest
import torch

import exact_attention_blackwell_gb300 as fa

pytestmark = pytest.mark.gpu


class Declines:
    def __getattr__(self, name):
        return lambda *a: None


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def operands():
    f32 = lambda *s: torch.zeros(s, device="cuda")
    return dict(q=bf(6, 4, 64), k=bf(6, 2, 64), v=bf(6, 2, 64), dq_out=bf(6, 4, 64), dk_out=bf(6, 2, 64), positions=i32(6),
                inv_freq=f32(16), q_weight=f32(64) + 1, k_weight=f32(64) + 1, eps=1e-6, axes=None, interleaved=False,
                k_pages=bf(9, 16, 2, 64), v_pages=bf(9, 16, 2, 64), page_table=i32(3, 3), cache_lens=i32(3), cu_seqlens=i32(4),
                max_new=2, lse=f32(4, 6), weights=f32(3, 2, 48), tree_mask=None, decay=1.0, scale=None, page_refs=i32(9), keep=5,
                recent=1)


ROPE = ("positions", "inv_freq", "q_weight", "k_weight", "eps", "axes", "interleaved")
CACHE = ("page_table", "cache_lens")
CALLS = {
    "rope": (fa.qk_norm_rope, ("q", "k") + ROPE),
    "rope_bwd": (fa.qk_norm_rope_bwd, ("dq_out", "dk_out", "q", "k") + ROPE),
    "append": (fa.cache_append_rope, ("q", "k", "v", "k_pages", "v_pages") + CACHE + ("cu_seqlens",) + ROPE),
    "weights": (fa.attention_weights_paged, ("q", "k_pages") + CACHE + ("cu_seqlens", "max_new", "lse", "weights", "tree_mask",
                                                                        "decay", "scale")),
    "evict": (fa.cache_evict, ("page_refs", "k_pages", "v_pages") + CACHE + ("weights", "keep", "recent")),
}
BAD = {
    "as it should be": lambda t: {},
    "no norms": lambda t: dict(q_weight=None, k_weight=None),
    "norms of two types": lambda t: dict(q_weight=t["q_weight"].bfloat16()),
    "norms of half precision": lambda t: dict(q_weight=t["q_weight"].half(), k_weight=t["k_weight"].half()),
    "a short norm": lambda t: dict(k_weight=t["k_weight"][:32]),
    "eps below zero": lambda t: dict(eps=-1.0),
    "eps as a whole number": lambda t: dict(eps=0),
    "eight frequencies": lambda t: dict(inv_freq=t["inv_freq"][:4]),
    "more frequencies than columns": lambda t: dict(inv_freq=torch.zeros(40, device="cuda")),
    "axes without positions for them": lambda t: dict(axes=(0,) * 8 + (1,) * 8),
    "an axis too many": lambda t: dict(axes=(2,) + (0,) * 15, positions=i32(2, 6)),
    "a negative axis": lambda t: dict(axes=(-1,) * 16, positions=i32(2, 6)),
    "five axes": lambda t: dict(axes=tuple(range(5)) + (0,) * 11, positions=i32(5, 6)),
    "axes as a list": lambda t: dict(axes=[0, 1] * 8, positions=i32(2, 6)),
    "positions of other tokens": lambda t: dict(positions=i32(5)),
    "positions of 64 bits": lambda t: dict(positions=t["positions"].long()),
    "positions on the CPU": lambda t: dict(positions=t["positions"].cpu()),
    "fp32 rows": lambda t: {n: t[n].float() for n in ("q", "dq_out")},
    "rows of dim 96": lambda t: dict(q=bf(6, 4, 96), k=bf(6, 2, 96), v=bf(6, 2, 96), dq_out=bf(6, 4, 96), dk_out=bf(6, 2, 96),
                                     q_weight=None, k_weight=None),
    "misaligned rows": lambda t: {n: bf(6 * 4 * 64 + 1)[1:].view(6, 4, 64) for n in ("q", "dq_out")},
    "columns apart": lambda t: {n: bf(6, 4, 128)[..., ::2] for n in ("q", "dq_out")},
    "keys of other tokens": lambda t: dict(k=bf(5, 2, 64), dk_out=bf(5, 2, 64)),
    "values of other heads": lambda t: dict(v=bf(6, 3, 64)),
    "no rows": lambda t: dict(q=bf(0, 4, 64), k=bf(0, 2, 64), v=bf(0, 2, 64), dq_out=bf(0, 4, 64), dk_out=bf(0, 2, 64),
                              positions=i32(0), lse=torch.zeros((4, 0), device="cuda")),
    "batches that do not follow one another": lambda t: {n: bf(2, 6, 4, 64)[:, :3] for n in ("q", "dq_out")},
    "pages of 24 rows": lambda t: dict(k_pages=bf(9, 24, 2, 64), v_pages=bf(9, 24, 2, 64)),
    "one tensor for keys and values": lambda t: dict(v_pages=t["k_pages"]),
    "lengths of another batch": lambda t: dict(cache_lens=t["cache_lens"][:2]),
    "a table of no columns": lambda t: dict(page_table=t["page_table"][:, :0]),
    "no sequences": lambda t: dict(page_table=t["page_table"][:0], cache_lens=t["cache_lens"][:0], cu_seqlens=i32(1),
                                   weights=t["weights"][:0]),
    "too many new tokens": lambda t: dict(max_new=257),
    "no new tokens": lambda t: dict(max_new=0),
    "decay below zero": lambda t: dict(decay=-1.0),
    "decay as a whole number": lambda t: dict(decay=1),
    "scale of zero": lambda t: dict(scale=0.0),
    "a mask of other words": lambda t: dict(tree_mask=torch.zeros((6, 2), dtype=torch.int64, device="cuda")),
    "lse of other heads": lambda t: dict(lse=t["lse"][:2]),
    "no columns of sums": lambda t: dict(weights=t["weights"][..., :0]),
    "sums of other heads": lambda t: dict(weights=torch.zeros((3, 4, 48), device="cuda")),
    "sums with layers": lambda t: dict(weights=t["weights"][None]),
    "pages with layers": lambda t: dict(k_pages=t["k_pages"][None], v_pages=t["v_pages"][None]),
    "pages and sums with layers": lambda t: dict(k_pages=t["k_pages"][None], v_pages=t["v_pages"][None], weights=t["weights"][None]),
    "recent past keep": lambda t: dict(recent=6),
    "keep below zero": lambda t: dict(keep=-1, recent=-1),
    "keep as another whole number": lambda t: dict(keep=True, recent=0),
    "counts of other pages": lambda t: dict(page_refs=t["page_refs"][:8]),
}


@pytest.mark.parametrize("call", CALLS)
def test_both_ways_accept_and_refuse_alike(monkeypatch, call):
    f, names = CALLS[call]

    def outcome(bad):
        t = operands()
        t |= BAD[bad](t)
        try:
            out = f(**{n: t[n] for n in names})
        except (ValueError, fa.FaError) as e:
            return type(e).__name__, str(e)
        torch.cuda.synchronize()
        return [None if x is None else (x.dtype, tuple(x.shape)) for x in (out if isinstance(out, tuple) else (out,))]

    want = {bad: outcome(bad) for bad in BAD}
    monkeypatch.setattr(fa, "_fast", Declines())
    got = {bad: outcome(bad) for bad in BAD}
    assert got == want
    assert not isinstance(want["as it should be"][0], str)
    refused = [bad for bad, x in want.items() if isinstance(x[0], str)]
    assert len(refused) >= (10 if call in ("rope", "rope_bwd") else 6), refused
