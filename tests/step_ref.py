"""Plain 64-bit forms of the operators of a MoE layer's step, and the error
bounds their tests use.  torch on the CPU; none of the package's code.

Bounds.  U = 2^-24 is the largest relative error of one FP32 rounding; a sum of
n FP32 terms in any order is off by at most (n - 1) U times the sum of their
magnitudes, by twice that where each addition may cut bits off instead of
rounding them, as a matrix unit may.  A value rounded to bf16 is off by 2^-8 of
itself at most, to fp16 by 2^-11, to E4M3 by 2^-4 (by 2^-10 below 2^-6).
"""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U, torch.float8_e4m3fn: 2.0 ** -4}
TINY = 2.0 ** -126
AMAX_FLOOR, FLOAT_MAX = 2.0 ** -100, 3.4028234663852886e38
D = torch.float64


def f64(t):
    return t.detach().cpu().to(D)


def assert_within(got, want, tol, what):
    """|got - want| <= tol everywhere, NaN where and only where want is NaN, the same infinities."""
    got, want = f64(got), want.to(D)
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)} != {tuple(want.shape)}"
    ok = ((got - want).abs() <= tol) | (got == want) | (got.isnan() & want.isnan())
    if not ok.all():
        i = tuple(torch.nonzero(~ok)[0].tolist())
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} off; first at {i}: got {got[i].item()!r}, want "
                             f"{want[i].item()!r}, tolerance {torch.as_tensor(tol, dtype=D).expand_as(want)[i].item()!r}")


# ---- a MoE layer for a few tokens -------------------------------------------------------

def spread(sf, rows, cols):
    """Scales of 128 x 128 blocks, for every element."""
    return sf.repeat_interleave(128, -2)[..., :rows, :].repeat_interleave(128, -1)[..., :cols]


def group_scale(h):
    """(scale, half a step of E4M3) of h [n, I] in groups of 128 columns, for every element."""
    n, I = h.shape
    amax = h.abs().view(n, I // 128, 128).amax(-1).clamp(AMAX_FLOOR, FLOAT_MAX).repeat_interleave(128, 1)
    return amax / 448


def moe_layer(x, ids, w, w13, w2, x_sf=None, w13_sf=None, w2_sf=None):
    """(out [T, H], its error bound) in 64 bits; tensors anywhere, ids outside [0, E) add nothing.
    The layer's h is not rounded here: its rounding to bf16 or E4M3 is in the bound."""
    fp8 = x_sf is not None
    (T, H), (E, I2, _) = x.shape, w13.shape
    I = I2 // 2
    xs = f64(x) * (f64(x_sf).repeat_interleave(128, 1)[:, :H] if fp8 else 1)
    out, tol = torch.zeros((T, H), dtype=D), torch.zeros((T, H), dtype=D)
    ids, w = ids.cpu(), f64(w)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        a, b = f64(w13[e]), f64(w2[e])
        if fp8:
            a, b = a * spread(f64(w13_sf[e]), I2, H), b * spread(f64(w2_sf[e]), H, I)
        both, size = xs[t] @ a.t(), xs[t].abs() @ a.abs().t()
        g, u = both[:, :I], both[:, I:]
        # products of H terms, scaled (3 more roundings); silu's slope is at most 1.1
        err = (2 * H + 8) * U * size
        sig = 1 / (1 + torch.exp(-g))
        h = g * sig * u
        e_h = 1.1 * err[:, :I] * (u.abs() + err[:, I:]) + (g * sig).abs() * err[:, I:] + 16 * U * (1 + g.abs()) * h.abs()
        if fp8:
            scale = group_scale(h.abs() + e_h)
            e_h = e_h + torch.maximum((h.abs() + e_h) * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 4 * U)
        else:
            e_h = e_h + (h.abs() + e_h) * 2.0 ** -8
        y = h @ b.t()
        e_y = e_h @ b.abs().t() + (2 * I + 8) * U * ((h.abs() + e_h) @ b.abs().t())
        out.index_add_(0, t, w[t, j][:, None] * y)
        tol.index_add_(0, t, w[t, j].abs()[:, None] * (e_y + 2 * ids.shape[1] * U * (y.abs() + e_y)))
    return out, tol + 2.0 ** -8 * (out.abs() + tol) + TINY
