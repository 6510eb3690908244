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


# ---- gate ---------------------------------------------------------------------------------

def _scores(l, sigmoid):
    """Scores over all experts, dead ones (-infinity, NaN) 0."""
    dead = ~(l > -torch.inf)
    l = l.clamp(max=FLOAT_MAX)
    if sigmoid:
        p = torch.where(l >= 0, 1 / (1 + torch.exp(-l)), torch.exp(l) / (1 + torch.exp(l)))
    else:
        p = torch.softmax(torch.where(dead, torch.full_like(l, -1e300), l), 1)
    return torch.where(dead, torch.zeros_like(p), p)


def _shares(q, l, taken, sigmoid):
    """The chosen scores q of logits l divided by their sum.  Sigmoids by their logarithms: far
    negative ones are 0 in 64 bits too, and still have proportions."""
    if sigmoid:
        log_q = torch.nn.functional.logsigmoid(l.clamp(max=FLOAT_MAX))
        share = torch.softmax(torch.where(taken, log_q, torch.full_like(log_q, -1e300)), 1)
        return torch.where(taken, share, torch.zeros_like(share))
    total = q.sum(1, keepdim=True)
    return torch.where(total > 0, q / total, torch.zeros_like(q))


def gate(logits, k, sigmoid, renormalize, scale=1.0, bias=None):
    """(ids [T, k], weights, error bound of the weights) by looking at the tokens one by one."""
    l = f64(logits)
    T, E = l.shape
    p = _scores(l, sigmoid)
    key = p + f64(bias) if bias is not None else l
    ids, w = torch.full((T, k), -1, dtype=torch.int64), torch.zeros((T, k), dtype=D)
    for t in range(T):
        live = [e for e in range(E) if l[t, e] > -torch.inf and key[t, e] > -torch.inf]
        live.sort(key=lambda e: (-key[t, e].item(), e))
        for j, e in enumerate(live[:k]):
            ids[t, j], w[t, j] = e, p[t, e]
    span = (l.clamp(max=FLOAT_MAX).amax(1, keepdim=True) - torch.where(ids >= 0, torch.gather(l, 1, ids.clamp(min=0)), l.amax(1, keepdim=True))).abs()
    if renormalize:
        w = _shares(w, torch.gather(l, 1, ids.clamp(min=0)), ids >= 0, sigmoid)
    w = scale * w
    # exp is off by 2 ulp (4 U) and by U for each unit of its rounded argument (a difference of
    # logits; of a lone sigmoid it is the logit itself); a sum of E terms; four more roundings
    return ids, w, (E + 20 + (0 if sigmoid and not renormalize else 2) * span.nan_to_num(0, 0, 0).clamp(max=200)) * U * w + TINY


def gate_grad(d_w, logits, ids, sigmoid, renormalize, scale=1.0):
    """(d_logits, its error's scale) in 64 bits; ids outside [0, E) take no part, repeated ones add."""
    l, g, ids = f64(logits), f64(d_w) * scale, ids.cpu().long()
    T, E = l.shape
    p = _scores(l, sigmoid)
    live = (ids >= 0) & (ids < E)
    at = ids.clamp(0, E - 1)
    g = torch.where(live, g, torch.zeros_like(g))
    q = torch.where(live, torch.gather(p, 1, at), torch.zeros_like(g))
    share = _shares(q, torch.gather(l, 1, at), live, sigmoid) if renormalize else q
    mean, size = (g * share).sum(1, keepdim=True), (g * share).abs().sum(1, keepdim=True)
    out, mag = torch.zeros((T, E), dtype=D), torch.zeros((T, E), dtype=D)
    if sigmoid and not renormalize:
        mean, size = torch.zeros_like(mean), torch.zeros_like(size)
    slope = share * (1 - q) if sigmoid else share
    if sigmoid or renormalize:
        d, m = slope * (g - mean), slope * (g.abs() + size)
    else:
        d, m = slope * g, slope * g.abs()
        out, mag = -p * mean, p * size
    return out.scatter_add(1, at, d), mag.scatter_add(1, at, m)


# ---- norms of query and key heads with the rotation -----------------------------------------

def rotate(n, table, positions, rotary, interleaved, back=False):
    """(turned, sum of the magnitudes of what is added) of [T, heads, D]."""
    cs = f64(table)[positions.cpu().long()][:, None]
    c, s = cs[..., :rotary // 2], cs[..., rotary // 2:]
    s = -s if back else s
    out, mag = n.clone(), n.abs()
    i = torch.arange(rotary // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    out[..., a], out[..., b] = n[..., a] * c - n[..., b] * s, n[..., a] * s + n[..., b] * c
    mag[..., a] = (n[..., a] * c).abs() + (n[..., b] * s).abs()
    mag[..., b] = (n[..., a] * s).abs() + (n[..., b] * c).abs()
    return out, mag


def qk_norm(x, gamma, eps, table, positions, rotary, interleaved):
    """(out, error bound without the output's rounding).  A lane adds 16 squares, then come at most 5
    levels of shuffles: 21 U of the mean and half of that for its root, 2 ulp (4 U) for rsqrtf, then 4 roundings."""
    x, gamma = f64(x), f64(gamma)
    n = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + float(torch.tensor(eps, dtype=torch.float32))) * gamma
    out, mag = rotate(n, table, positions, rotary, interleaved)
    return out, 24 * U * mag


def qk_norm_grad(d_out, x, gamma, eps, table, positions, rotary, interleaved):
    """(d_x, bound, d_gamma, bound) without the outputs' rounding."""
    x, gamma = f64(x), f64(gamma)
    d, mag = rotate(f64(d_out), table, positions, rotary, interleaved, back=True)
    inv = 1 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + float(torch.tensor(eps, dtype=torch.float32)))
    unit = x * inv
    dn = gamma * d
    d_x = inv * (dn - unit * (dn * unit).mean(-1, keepdim=True))
    dm = gamma.abs() * mag
    size = inv * (dm + unit.abs() * (dm * unit.abs()).mean(-1, keepdim=True))
    # three powers of inv (16 U each), a sum of 21 levels, 8 more roundings
    terms = d.shape[0] * d.shape[1]
    return d_x, 80 * U * size, (d * unit).sum((0, 1)), (terms + 24) * U * (mag * unit.abs()).sum((0, 1))


# ---- gradient norm and clipping ---------------------------------------------------------------

def clip(grads, max_norm, eps):
    """(norm, scaled tensors): FP32 chains are at most 128 squares and 3 sums, halved by the root."""
    norm = torch.sqrt(sum((f64(g).pow(2).sum() for g in grads), torch.zeros((), dtype=D)))
    scale = 1.0
    if torch.isfinite(norm):
        scale = min(1.0, float(max_norm) / (float(norm) + eps)) if float(norm) + eps > 0 else 1.0
    return norm, [f64(g) * scale for g in grads]


CLIP_REL = 70 * U
