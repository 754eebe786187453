"""Queries and keys made ready, for the tests: 64-bit torch arithmetic from the definitions."""
from __future__ import annotations

import torch

EPS = 1e-6


def angles(positions, inv_freq, axes):
    """[..., rot / 2] radians; positions [...] or, with axes, [n_axes, ...]."""
    pos, f = positions.double(), inv_freq.double()
    if axes is None:
        return pos[..., None] * f
    return torch.stack([pos[a] * f[i] for i, a in enumerate(axes)], -1)


def columns(half, interleaved):
    """Columns of the first and of the second half of each pair."""
    if interleaved:
        return torch.arange(0, 2 * half, 2), torch.arange(1, 2 * half, 2)
    return torch.arange(half), torch.arange(half, 2 * half)


def rotate(y, angle, interleaved):
    a, b = columns(angle.shape[-1], interleaved)
    c, s = torch.cos(angle).unsqueeze(-2), torch.sin(angle).unsqueeze(-2)
    out = y.clone()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def spread(y, half, interleaved):
    """What a rounding of a pair's rotation is relative to: |y_a| + |y_b| in both columns, |y| elsewhere."""
    a, b = columns(half, interleaved)
    out = y.abs().clone()
    out[..., a] = out[..., b] = y[..., a].abs() + y[..., b].abs()
    return out


def forward(x, w, angle, interleaved, eps=EPS):
    y = x
    if w is not None:
        y = x * (x.square().mean(-1, keepdim=True) + eps) ** -0.5 * w
    return rotate(y, angle, interleaved)


def check_forward(got, x, w, angle, interleaved, eps=EPS, what=""):
    """The roundings: the sum of d squares, d 2^-24 of it, half of that in r; rsqrt, two products and those of the
    rotation, some 2^-22 each; cosine and sine 2^-22, their angle 2^-24 turns; at the end 2^-8 of the result."""
    x = x.detach().cpu().double()
    w = None if w is None else w.detach().cpu().double()
    want = forward(x, w, angle, interleaved, eps)
    y = x if w is None else x * (x.square().mean(-1, keepdim=True) + eps) ** -0.5 * w
    bound = 2.0**-8 * want.abs() + (x.shape[-1] * 2.0**-24 + 2.0**-19) * spread(y, angle.shape[-1], interleaved) + 2.0**-126
    off = (got.cpu().double() - want).abs()
    assert got.shape == want.shape and not (off > bound).any() and torch.isfinite(got).all(), (
        f"{what}: off by {float((off - bound).max()):.3e} past its bound, {int((off > bound).sum())} values, "
        f"first {(off > bound).nonzero()[:1].tolist()}")


def check_backward(dx, dw, dy, x, w, angle, interleaved, eps=EPS, what=""):
    """dx and dw against the formulas, with magnitudes in place of the values for the bounds: the errors of the
    forward's factors, the sum of d products in mean(x w g), a sum over all rows in dw (its depth at most their
    number), and 2^-8 of the result for dx."""
    dy, x = dy.cpu().double(), x.cpu().double()
    d, half = dy.shape[-1], angle.shape[-1]
    g, size = rotate(dy, -angle, interleaved), spread(dy, half, interleaved)
    each = d * 2.0**-23 + 2.0**-18
    if w is None:
        want, bound = g, each * size
        assert dw is None
    else:
        w = w.cpu().double()
        r = (x.square().mean(-1, keepdim=True) + eps) ** -0.5
        want = r * (w * g - x * r * r * (x * w * g).mean(-1, keepdim=True))
        bound = each * r * (w.abs() * size + x.abs() * r * r * (x * w * size).abs().mean(-1, keepdim=True))
        terms, sizes = (g * x * r).flatten(0, -2), (size * x * r).abs().flatten(0, -2)
        off = (dw.cpu().double() - terms.sum(0)).abs()
        room = (each + terms.shape[0] * 2.0**-24) * sizes.sum(0) + 2.0**-126
        assert dw.dtype == torch.float32 and dw.shape == (d,)
        assert not (off > room).any(), f"{what}: dw off by {float((off / room).max()):.2f} of its bound"
    off, room = (dx.cpu().double() - want).abs(), bound + 2.0**-8 * want.abs() + 2.0**-126
    assert dx.shape == want.shape and not (off > room).any(), f"{what}: dx off by {float((off / room).max()):.2f} of its bound"
