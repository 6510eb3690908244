"""Plain 64-bit forms of the operators around the finalize, and the error
bounds their tests use.  NumPy / torch on the CPU; none of the package's code.

Bounds.  u = 2^-24 is the largest relative error of one FP32 rounding, and a
value rounded to bf16 is off by at most 2^-8 of itself (half a step), to E4M3
by 2^-4 (and by 2^-10 below the smallest normal 2^-6).  No FP32 sum over the
columns of a token (H <= 16384) is a chain of more than CHAIN additions: a thread
adds at most 64 products, then come 5 shuffle levels and at most 32 - 5
partial sums of warps.
"""
import numpy as np
import torch

U = 2.0 ** -24
CHAIN = 96
BF16 = 2.0 ** -8
E4M3 = 2.0 ** -4
TINY = 2.0 ** -126          # results this small may also lose bits to gradual underflow

AMAX_FLOOR, FLOAT_MAX = 2.0 ** -100, float(np.finfo(np.float32).max)


def route(ids, E, align, R=None):
    """(row_of [T, k], slot_of [R], offsets [E + 1], counts [E]) by looking at the pairs one by one."""
    ids = np.asarray(ids)
    T, k = ids.shape
    N = T * k
    counts = np.array([(ids == e).sum() for e in range(E)], dtype=np.int64)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    if R is None:
        R = N + min(E, N) * (align - 1)
    row_of = np.full(N, -1, dtype=np.int64)
    slot_of = np.where(np.arange(R) < offsets[E], -1, -2)
    nxt = offsets[:E].copy()
    for s, e in enumerate(ids.reshape(-1)):
        if 0 <= e < E:
            row_of[s] = nxt[e]
            slot_of[nxt[e]] = s
            nxt[e] += 1
    return row_of.reshape(T, k), slot_of, offsets, counts


def draw_ids(T, k, E, seed, nonlocal_share=0.0, skew=0.0):
    rng = np.random.default_rng(seed)
    score = rng.gumbel(size=(T, E)) - skew * np.log(np.arange(1, E + 1))
    ids = np.argsort(-score, axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < nonlocal_share] = -1
    return ids


def finalize_grad(d_out, E, row_of, slot_of, w):
    """(d_rows [R, H] with NaN where a row is left alone, d_w [T, k], scale of d_w's error) in 64 bits."""
    d_out, E, w = (np.asarray(a, dtype=np.float64) for a in (d_out, E, w))
    T, k = row_of.shape
    d_rows = np.full(E.shape, np.nan)
    d_rows[slot_of == -1] = 0
    d_w, size = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = row_of[t, j]
            if 0 <= r < len(slot_of) and slot_of[r] == t * k + j:
                d_rows[r] = w[t, j] * d_out[t]
                d_w[t, j] = np.sum(E[r] * d_out[t])
                size[t, j] = np.sum(np.abs(E[r] * d_out[t]))
    return d_rows, d_w, size


def residual_norm(x, residual, gamma, eps):
    """(r as FP32 rounds it, y, 1 / rms) in 64 bits from the FP32 r."""
    r = (np.asarray(residual, dtype=np.float32) + np.asarray(x, dtype=np.float32))
    r64 = r.astype(np.float64)
    inv = 1.0 / np.sqrt(np.mean(r64 * r64, axis=1, keepdims=True) + np.float64(np.float32(eps)))
    return r, r64 * inv * np.asarray(gamma, dtype=np.float64), inv


#: relative error of y: the sum of squares (positive terms, so CHAIN u), the
#: division and eps, halved by the root; rsqrtf is off by at most 2 ulp (4 u);
#: two products.
Y_REL = (CHAIN + 2) / 2 * U + 4 * U + 2 * U


def group_amax(y, size):
    T, H = y.shape
    S = -(-H // size)
    full = np.zeros((T, S * size))
    full[:, :H] = np.abs(y)
    return np.clip(full.reshape(T, S, size).max(-1), AMAX_FLOOR, FLOAT_MAX)


def residual_norm_grad(d_out, d_res, r, gamma, eps):
    """(d_r, its error's scale, d_gamma, its error's scale) in 64 bits."""
    d_out, r, gamma = (np.asarray(a, dtype=np.float64) for a in (d_out, r, gamma))
    d_res = np.zeros_like(r) if d_res is None else np.asarray(d_res, dtype=np.float64)
    inv = 1.0 / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + np.float64(np.float32(eps)))
    unit = r * inv
    dn = gamma * d_out
    d_r = d_res + inv * (dn - unit * np.mean(dn * unit, axis=1, keepdims=True))
    size = np.abs(d_res) + inv * (np.abs(dn) + np.abs(unit) * np.mean(np.abs(dn * unit), axis=1, keepdims=True))
    return d_r, size, np.sum(d_out * unit, axis=0), np.sum(np.abs(d_out * unit), axis=0)


#: relative to residual_norm_grad's scale: three powers of inv, each off by
#: Y_REL, the sum of CHAIN products, and eight more roundings.
GRAD_REL = 3 * Y_REL + CHAIN * U + 8 * U


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def assert_within(got, want, tol, what):
    """|got - want| <= tol everywhere, NaN where and only where want is NaN, the same infinities."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape, f"{what}: shape {got.shape} != {want.shape}"
    with np.errstate(invalid="ignore"):
        ok = (np.abs(got - want) <= tol) | (got == want) | (np.isnan(got) & np.isnan(want))
    if not ok.all():
        i = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{what}: {(~ok).sum()} of {ok.size} off; first at {i}: got {got[i]!r}, want {want[i]!r}, "
                             f"tolerance {np.broadcast_to(tol, want.shape)[i]!r}")
