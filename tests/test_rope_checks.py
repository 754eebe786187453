"""Refusals of the calls that make queries and keys ready, without a GPU."""
import ctypes

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
from exact_attention_blackwell_gb300 import build as fa_build

A = 0x10000  # an aligned fake device address: never dereferenced
INV, UNS, ALI, WS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_ALIGNMENT, fa.FA_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()
    return fa.lib()


def ids(x):
    return str(x) if isinstance(x, dict) else None


ROWS = dict(q=A, q_token=256, q_head=64, k=A, k_token=128, k_head=64)
ANGLES = dict(positions=A, n_axes=1, inv_freq=A, rot=64, axes=None, q_weight=A, k_weight=A, bf16_weights=0, eps=1e-6,
              interleaved=0)
COMMON = [
    (dict(total=-1), INV), (dict(H=0), INV), (dict(Hkv=0), INV), (dict(d=0), INV), (dict(d=96), UNS), (dict(H=65536), UNS),
    (dict(Hkv=65536), UNS), (dict(rot=0), INV), (dict(rot=-16), INV), (dict(rot=80), INV), (dict(rot=24), UNS), (dict(rot=8), UNS),
    (dict(n_axes=0), INV), (dict(n_axes=2), INV), (dict(n_axes=5, axes=(0,) * 32), UNS), (dict(axes=(0,) * 31 + (1,)), INV),
    (dict(n_axes=2, axes=(2,) + (0,) * 31), INV), (dict(n_axes=2, axes=(-1,) * 32), INV), (dict(inv_freq=None), INV),
    (dict(inv_freq=A + 2), ALI), (dict(positions=A + 1), ALI), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(total=2**31 - 1, H=65535), UNS), (dict(total=2**31 - 1, Hkv=65535), UNS),
    (dict(q_weight=A + 2), ALI), (dict(k_weight=A + 1), ALI), (dict(k_weight=A + 1, bf16_weights=1), ALI),
]


@pytest.mark.parametrize("args,code", COMMON + [
    (dict(q=None), INV), (dict(k=None), INV), (dict(positions=None), INV), (dict(q_out=None), INV), (dict(k_out=None), INV),
    (dict(q=A + 8), ALI), (dict(k=A + 2), ALI), (dict(q_out=A + 8), ALI), (dict(k_out=A + 4), ALI), (dict(q_token=4), ALI),
    (dict(q_head=65), ALI), (dict(k_token=12), ALI), (dict(k_head=1), ALI)], ids=ids)
def test_forward(args, code):
    a = ROWS | ANGLES | dict(q_out=A, k_out=A, total=5, H=4, Hkv=2, d=64, stream=0) | args
    assert fa.fa_qk_norm_rope(**a) == code


@pytest.mark.parametrize("args,code", COMMON + [
    (dict(dq_out=None), INV), (dict(dk_out=None), INV), (dict(positions=None), INV), (dict(dq=None), INV), (dict(dk=None), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(dq_weight=None), INV), (dict(dk_weight=None), INV), (dict(dq_out=A + 8), ALI),
    (dict(dk_out=A + 2), ALI), (dict(dq=A + 8), ALI), (dict(dk=A + 8), ALI), (dict(q=A + 8), ALI), (dict(k=A + 8), ALI),
    (dict(dq_token=4), ALI), (dict(dk_head=3), ALI), (dict(q_token=4), ALI), (dict(k_head=3), ALI), (dict(dq_weight=A + 2), ALI),
    (dict(dk_weight=A + 2), ALI), (dict(workspace=None), WS), (dict(workspace=A + 16), WS), (dict(workspace_bytes=99), WS)], ids=ids)
def test_backward(args, code):
    a = dict(dq_out=A, dq_token=256, dq_head=64, dk_out=A, dk_token=128, dk_head=64) | ROWS | ANGLES | dict(
        dq=A, dk=A, dq_weight=A, dk_weight=A, total=5, H=4, Hkv=2, d=64, workspace=A, workspace_bytes=1 << 30, stream=0) | args
    assert fa.fa_qk_norm_rope_bwd(**a) == code


def test_backward_workspace():
    for d in (64, 128, 256):
        need = fa.fa_qk_norm_rope_bwd_workspace_bytes(d)
        a = dict(dq_out=A, dq_token=0, dq_head=d, dk_out=A, dk_token=0, dk_head=d, q=A, q_token=0, q_head=d, k=A, k_token=0,
                 k_head=d, **ANGLES, dq=A, dk=A, dq_weight=A, dk_weight=A, total=1, H=1, Hkv=1, d=d, workspace=A,
                 workspace_bytes=need - 1, stream=0)
        assert need > 0 and fa.fa_qk_norm_rope_bwd(**a) == WS
    assert fa.fa_qk_norm_rope_bwd_workspace_bytes(96) == 0


@pytest.mark.parametrize("args,code", COMMON + [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(q_out=None), INV), (dict(q=A + 8), ALI), (dict(k=A + 8), ALI),
    (dict(v=A + 8), ALI), (dict(q_out=A + 8), ALI), (dict(k_pages=A + 8), ALI), (dict(v_pages=A + 8), ALI), (dict(v_token=4), ALI),
    (dict(v_head=4), ALI), (dict(k_pages=None), INV), (dict(v_pages=None), INV), (dict(v_pages=A), INV), (dict(page_table=None), INV),
    (dict(cache_lens=None), INV), (dict(cu_seqlens=None), INV), (dict(cu_seqlens=A + 2), ALI), (dict(page_table=A + 2), ALI),
    (dict(cache_lens=A + 2), ALI), (dict(B=0), INV), (dict(B=65536), UNS), (dict(page_size=24), UNS), (dict(max_pages=0), INV),
    (dict(num_pages=0), INV), (dict(max_pages=1 << 27), UNS)], ids=ids)
def test_append(args, code):
    a = ROWS | dict(v=A, v_token=128, v_head=64, k_pages=A, v_pages=A + 4096, page_table=A, cache_lens=A, cu_seqlens=A) | ANGLES | dict(
        q_out=A, B=2, max_pages=4, num_pages=9, page_size=16, total=5, H=4, Hkv=2, d=64, stream=0) | args
    assert fa.fa_cache_append_rope(**a) == code


# ------------------------------------------------------------------ torch helpers
def tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    f32 = lambda *s: torch.zeros(s, dtype=torch.float32)
    return dict(q=bf(5, 4, 64), k=bf(5, 2, 64), v=bf(5, 2, 64), dq_out=bf(5, 4, 64), dk_out=bf(5, 2, 64), k_pages=bf(9, 16, 2, 64),
                v_pages=bf(9, 16, 2, 64), page_table=i32(3, 4), cache_lens=i32(3), cu_seqlens=i32(4), positions=i32(5),
                inv_freq=f32(16), q_weight=f32(64), k_weight=f32(64))


NORMS = ("q_weight", "k_weight")
CALLS = {
    "forward": (fa.qk_norm_rope, ("q", "k", "positions", "inv_freq") + NORMS),
    "backward": (fa.qk_norm_rope_bwd, ("dq_out", "dk_out", "q", "k", "positions", "inv_freq") + NORMS),
    "append": (fa.cache_append_rope, ("q", "k", "v", "k_pages", "v_pages", "page_table", "cache_lens", "cu_seqlens", "inv_freq",
                                      "positions") + NORMS),
}


def call(op, t):
    f, names = CALLS[op]
    return f(**{n: t[n] for n in names})


@pytest.mark.parametrize("op,name", [(o, n) for o, (_, names) in CALLS.items() for n in names])
def test_every_operand_is_checked(op, name):
    good = tensors()
    with pytest.raises(ValueError, match="CUDA"):
        call(op, good)
    x = good[name]
    wide = torch.zeros(x.shape[:-1] + (2 * x.shape[-1],), dtype=x.dtype)
    for bad in (x.double() if x.is_floating_point() else x.to(torch.int16), x[..., None], x[:-1], wide[..., ::2], wide):
        if (name, bad.shape) in (("inv_freq", (15,)), ("inv_freq", (32,))):
            continue  # its length is the number of pairs
        if name == "page_table" and bad is wide:
            continue  # any number of columns
        if op == "backward" and bad.shape[:1] != x.shape[:1] and name in ("dq_out",):
            continue
        with pytest.raises((ValueError, fa.FaError), match="^(?!.*CUDA tensor)"):
            call(op, good | {name: bad})
    if name not in NORMS + (("positions",) if op == "append" else ()):
        with pytest.raises((ValueError, AttributeError)):
            call(op, good | {name: None})


def test_views_are_taken_as_they_are_and_refused_where_tokens_have_no_stride():
    x = torch.zeros((2, 6, 8, 64), dtype=torch.bfloat16)
    _, token, head = fa._rows("q", x[:, :, 2:6])
    assert (token, head) == (8 * 64, 64)
    _, token, head = fa._rows("q", x.transpose(1, 2)[:1])  # heads before tokens
    assert (token, head) == (64, 8 * 64)
    _, token, head = fa._rows("q", x[:, 3:4])  # one token of each batch
    assert (token, head) == (6 * 8 * 64, 64)
    _, token, head = fa._rows("q", x[:1, 3:4, 5:6])
    assert (token, head) == (0, 0)
    _, token, head = fa._rows("q", x[0, 0].expand(5, 8, 64))
    assert (token, head) == (0, 64)
    with pytest.raises(ValueError, match="batches"):
        fa._rows("q", x[:, :3])
    with pytest.raises(ValueError, match="last dimension"):
        fa._rows("q", x.transpose(2, 3), None)


def test_axes_and_weights():
    t = tensors()
    base = {n: t[n] for n in CALLS["forward"][1]}
    many = torch.zeros((3, 5), dtype=torch.int32)
    for bad in (dict(axes=(0,) * 16), dict(axes=(0,) * 15, positions=many), dict(axes=(3,) + (0,) * 15, positions=many),
                dict(axes=(-1,) * 16, positions=many), dict(positions=many), dict(q_weight=t["q_weight"].bfloat16()),
                dict(q_weight=t["q_weight"].half(), k_weight=None)):
        with pytest.raises(ValueError, match="^(?!.*CUDA tensor)"):
            fa.qk_norm_rope(**(base | bad))
    for good in (dict(axes=(0, 1, 2, 2) * 4, positions=many), dict(axes=[0] * 16, positions=many[:1]), dict(q_weight=None),
                 dict(q_weight=None, k_weight=t["k_weight"].bfloat16())):
        with pytest.raises(ValueError, match="CUDA"):
            fa.qk_norm_rope(**(base | good))


def test_axes_are_a_host_array():
    assert list(fa._axes((0, 1, 2))) == [0, 1, 2] and fa._axes(None) is None
    assert isinstance(fa._axes((0,)), ctypes.Array)
