"""Inputs of a MoE layer for which its first products are exact in FP32, and the
layer's output for them with a bound that shows every column of h.

x and the rows of G and U are small whole numbers times powers of two, so that every
partial sum is an FP32 number in any order, cut off or rounded: g and u have no
error, and h has that of silu alone.  What is left of the layer's error is what it
does with h.

bf16: h is the sum of two bf16 values, off by 2^-16 of itself.  Two columns a and b of
h have the same g, and u that differ by 1 around 128; a row of D_e is +1 at b and -1 at
a, so that the upper parts nearly cancel and the output is made of lower ones.
E4M3: h is quantised by the stated rule, in 64 bits; only values that lie closer to a
boundary than silu's error reach have two possible codes.

torch on the CPU; none of the package's code.
"""
import torch

from step_ref import AMAX_FLOOR, D, FLOAT_MAX, TINY, U, f64, spread

FP8 = torch.float8_e4m3fn


def _whole(g, most, *shape):
    return torch.randint(-most, most + 1, shape, generator=g).to(D)


def _power(std, wanted):
    """The power of two that brings std nearest to `wanted`."""
    return 2.0 ** round(float(torch.log2(torch.tensor(wanted / std))))


def _powers(g, *shape):
    """1/2, 1 or 2."""
    return 2.0 ** torch.randint(-1, 2, shape, generator=g).to(D)


def _pairs(g, T, E, k):
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    return ids, 0.25 + 0.75 * torch.rand((T, k), generator=g)


def inputs_bf16(T, H, I, E, k, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = _whole(g, 1, T, H)
    x[:, :2] = 1
    half = I // 2
    gates, ups, w2 = _whole(g, 2, E, I, H), _whole(g, 4, E, I, H), torch.zeros((E, H, I), dtype=D)
    gates *= _power((H * 4 / 3) ** 0.5, 1.5)
    gates[:, :, 1], ups[:, :, 1] = 0, 128
    rows = torch.arange(H)
    pair = rows % half if H >= half else rows * half // H
    for e in range(E):
        a, b = torch.randperm(I, generator=g)[:2 * half].view(2, half)
        gates[e, b], ups[e, b] = gates[e, a], ups[e, a]
        ups[e, b, 0] += 1
        w2[e, rows, a[pair]], w2[e, rows, b[pair]] = -1, 1
    ids, w = _pairs(g, T, E, k)
    B16 = torch.bfloat16
    return dict(x=x.to(B16), expert_ids=ids, topk_weights=w, w13=torch.cat([gates, ups], 1).to(B16), w2=w2.to(B16))


def inputs_e4m3(T, H, I, E, k, seed=0):
    g = torch.Generator().manual_seed(seed)
    hb, ib = -(-H // 128), I // 128
    # a mean square of 2/3 and 2 of the codes and of 7/4 of each scale
    s = _power((H * 4 / 3) ** 0.5 * 7 / 4, 1.5)
    ids, w = _pairs(g, T, E, k)
    return dict(x=_whole(g, 1, T, H).to(FP8), expert_ids=ids, topk_weights=w, w13=_whole(g, 2, E, 2 * I, H).to(FP8),
                w2=_whole(g, 4, E, H, I).to(FP8), x_sf=_powers(g, T, hb).float(), w13_sf=(_powers(g, E, 2 * ib, hb) * s).float(),
                w2_sf=_powers(g, E, hb, ib).float())


def e4m3(v):
    """The E4M3 value nearest to v, saturating."""
    return v.clamp(-448, 448).float().to(FP8).to(D)


def hidden(i, t, e):
    """(h of tokens t at expert e, its error) before any rounding of h."""
    I = i["w13"].shape[1] // 2
    x, a = f64(i["x"])[t], f64(i["w13"][e])
    if "x_sf" in i:
        x = x * f64(i["x_sf"])[t].repeat_interleave(128, 1)[:, :x.shape[1]]
        a = a * spread(f64(i["w13_sf"][e]), *a.shape)
    both = x @ a.t()
    g, u = both[:, :I], both[:, I:]
    h = g / (1 + torch.exp(-g)) * u
    return h, 16 * U * (1 + g.abs()) * h.abs()


def down(i, e):
    b = f64(i["w2"][e])
    return b * spread(f64(i["w2_sf"][e]), *b.shape) if "w2_sf" in i else b


def kept(h, err, fp8):
    """(middle, half width) of what the layer may hold for h."""
    if not fp8:
        return h, err + 2.0 ** -16 * (h.abs() + err)
    groups = (h.shape[0], -1, 128)
    lo, hi = (h.abs() - err).clamp(min=0), h.abs() + err
    least, most = (v.view(groups).amax(-1).clamp(AMAX_FLOOR, FLOAT_MAX).repeat_interleave(128, 1) for v in (lo, hi))
    # a quotient, a product; the scale is one quotient
    lo = e4m3(lo * (448 / most) * (1 - 4 * U)) * (least / 448) * (1 - 2 * U)
    hi = e4m3(hi * (448 / least) * (1 + 4 * U)) * (most / 448) * (1 + 2 * U)
    return h.sign() * (lo + hi) / 2, (hi - lo) / 2


def layer(i):
    """(out [T, H], its error bound) in 64 bits."""
    fp8 = "x_sf" in i
    (T, H), k = i["x"].shape, i["expert_ids"].shape[1]
    out, tol = torch.zeros((T, H), dtype=D), torch.zeros((T, H), dtype=D)
    w = f64(i["topk_weights"])
    for e in range(i["w13"].shape[0]):
        t, j = torch.nonzero(i["expert_ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        h, off = kept(*hidden(i, t, e), fp8)
        b = down(i, e)
        terms = int((b != 0).sum(1).max()) * (1 if fp8 else 2)        # zeros add nothing, not even an error
        y = h @ b.t()
        e_y = off @ b.abs().t() + (2 * terms + 8) * U * ((h.abs() + off) @ b.abs().t())
        out.index_add_(0, t, w[t, j][:, None] * y)
        tol.index_add_(0, t, w[t, j][:, None] * (e_y + 2 * k * U * (y.abs() + e_y)))
    return out, tol + 2.0 ** -8 * (out.abs() + tol) + TINY


def emulated(i, hold):
    """bf16 output with hold(h) in the place of what the layer holds for h."""
    out = torch.zeros(i["x"].shape, dtype=D)
    for e in range(i["w13"].shape[0]):
        t, j = torch.nonzero(i["expert_ids"] == e, as_tuple=True)
        if t.numel():
            out.index_add_(0, t, f64(i["topk_weights"])[t, j][:, None] * (hold(hidden(i, t, e)[0]) @ down(i, e).t()))
    return out.to(torch.bfloat16)
