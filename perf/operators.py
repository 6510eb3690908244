"""The operators around the MoE finalize, as cases that can be measured.

What surrounds the finalize in one MoE block, in the order a layer runs it:

  residual_norm       residual += x; y = RMSNorm(residual) * gamma, written in 8 bits (E4M3) with scales
  residual_norm_grad  its gradient: to the residual stream, to the added rows, to gamma
  route               the (token, slot) pairs sorted by expert: index maps, block offsets, counts
  dispatch            the token rows copied into expert order (16-bit rows, or 8-bit rows with scales)
  dispatch_grad       its gradient: the k rows of a token summed
  finalize_grad       the gradient of the weighted sum that the finalize takes: to the expert rows and to the weights

`run` computes a case in its plain form (elementary torch operations in 32
bits), or, with `own` set, through the package's entry points.
"""
import math

import torch

own = False

DEVICE = "cuda"
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100       # a group whose largest magnitude is below this is scaled as if it were this
FLOAT_MAX = 3.4028234663852886e38
SCALE_GROUPS = {"token": 0, "group128": 128, "mx32": 32}

# The sizes are those of the repository's own workloads (decode, prefill, wide,
# stress; hidden sizes 4096 and 8192, k = 8, 64 to 256 experts) and odd ones
# between them.
LISTED = [
    # one decode step of a small batch: 64 pairs, all latency
    {"name": "route_decode", "op": "route", "T": 8, "k": 8, "E": 128, "zipf": 0.0, "align": 1, "nonlocal_share": 0.0},
    # the stress routing: a quarter of a million pairs, very uneven experts, blocks padded for a 128-row GEMM tile
    {"name": "route_stress", "op": "route", "T": 32768, "k": 8, "E": 256, "zipf": 1.5, "align": 128, "nonlocal_share": 0.0},
    # a decode step's rows
    {"name": "dispatch_decode", "op": "dispatch", "T": 8, "H": 4096, "k": 8, "E": 128, "zipf": 0.0, "align": 1,
     "fp8": False, "nonlocal_share": 0.0},
    # a prefill's rows, blocks padded for a 128-row GEMM tile
    {"name": "dispatch_prefill", "op": "dispatch", "T": 16384, "H": 4096, "k": 8, "E": 128, "zipf": 1.2, "align": 128,
     "fp8": False, "nonlocal_share": 0.0},
    # 8-bit rows with one scale per 128 columns, wide model, an eighth of the experts elsewhere
    {"name": "dispatch_wide_fp8", "op": "dispatch", "T": 4096, "H": 8192, "k": 8, "E": 256, "zipf": 0.0, "align": 1,
     "fp8": True, "nonlocal_share": 0.125},
    # a training step's way back, one token more than a power of two
    {"name": "dispatch_grad_wide", "op": "dispatch_grad", "T": 4097, "H": 8192, "k": 8, "E": 256, "zipf": 0.0, "align": 1,
     "nonlocal_share": 0.0},
    # a short ragged micro-batch with six experts a token and a 32-bit gradient (the residual stream's own)
    {"name": "finalize_grad_ragged", "op": "finalize_grad", "T": 333, "H": 2056, "k": 6, "E": 64, "zipf": 1.2, "align": 1,
     "fp32": True, "nonlocal_share": 0.0},
    # a training step at the prefill size, blocks padded for a 128-row GEMM tile
    {"name": "finalize_grad_prefill", "op": "finalize_grad", "T": 16384, "H": 4096, "k": 8, "E": 128, "zipf": 1.2,
     "align": 128, "fp32": False, "nonlocal_share": 0.0},
    # a decode step's norm, for a GEMM that takes a scale per 128 columns
    {"name": "residual_norm_decode", "op": "residual_norm", "T": 8, "H": 4096, "scales": "group128", "tiled": False,
     "bf16_too": False},
    # a prefill's norm, for a block-scaled GEMM (a power-of-two scale per 32 columns, tiled), and in bf16 for the router
    {"name": "residual_norm_prefill", "op": "residual_norm", "T": 16384, "H": 4096, "scales": "mx32", "tiled": True,
     "bf16_too": True},
    # a training micro-batch of odd length and width
    {"name": "residual_norm_grad_ragged", "op": "residual_norm_grad", "T": 511, "H": 4104},
    # a training step, wide model
    {"name": "residual_norm_grad_wide", "op": "residual_norm_grad", "T": 8192, "H": 8192},
]


def listed():
    return [dict(c) for c in LISTED]


def _log(rng, a, b):
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "dispatch_grad", "finalize_grad", "residual_norm", "residual_norm_grad"])
    T = _log(rng, 1, 32768)
    if op == "route":
        E = _log(rng, 4, 512)
        return {"op": op, "T": T, "k": rng.randint(1, min(E, 16)), "E": E, "zipf": rng.choice([0.0, 1.2, 1.5]),
                "align": rng.choice([1, 1, 16, 128]), "nonlocal_share": rng.choice([0.0, 0.0, 0.25])}
    H = 16 * _log(rng, 4, 1024)
    if op in ("residual_norm", "residual_norm_grad"):
        T = min(T, (1 << 26) // H)      # at most the largest listed one's elements
        if op == "residual_norm_grad":
            return {"op": op, "T": T, "H": H}
        scales = rng.choice(sorted(SCALE_GROUPS))
        return {"op": op, "T": T, "H": H, "scales": scales, "tiled": scales == "mx32" and rng.random() < 0.5,
                "bf16_too": rng.random() < 0.5}
    E = _log(rng, 4, 256)
    k = rng.randint(1, min(E, 16))
    align = rng.choice([1, 1, 16])
    T = max(1, min(T, (1 << 28) // (H * k)))
    c = {"op": op, "T": T, "H": H, "k": k, "E": E, "zipf": rng.choice([0.0, 1.2]), "align": align,
         "nonlocal_share": rng.choice([0.0, 0.0, 0.25])}
    if op == "dispatch":
        c["fp8"] = rng.random() < 0.5
    if op == "finalize_grad":
        c["fp32"] = rng.random() < 0.5
    return c


# ---- inputs ------------------------------------------------------------------------

def _rows(c):
    """Rows that hold every expert's block, each padded to a multiple of align."""
    return c["T"] * c["k"] + min(c["E"], c["T"] * c["k"]) * (c["align"] - 1)


def _expert_ids(c, g):
    """k distinct experts a token by Gumbel top-k; a pair whose expert is on another GPU has id -1."""
    T, k, E = c["T"], c["k"], c["E"]
    logp = -c["zipf"] * torch.log(torch.arange(1, E + 1, device=DEVICE, dtype=torch.float32))
    u = torch.rand((T, E), generator=g, device=DEVICE).clamp_(1e-20, 1 - 1e-7)
    ids = torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices
    ids = torch.where(ids < round(E * (1 - c["nonlocal_share"])), ids, torch.full_like(ids, -1))
    return ids.to(torch.int32).contiguous()


def _weights(T, k, g):
    z = torch.randn((T, k), generator=g, device=DEVICE)
    return torch.softmax(z, dim=1).sort(dim=1, descending=True).values.contiguous()


def _normal(shape, g, dtype, scale=1.0):
    out = torch.empty(shape, device=DEVICE, dtype=dtype)
    flat, step = out.view(-1), 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEVICE) * scale
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 1000003 + 17)
    op, T = c["op"], c["T"]
    s = {"case": c}
    if op in ("residual_norm", "residual_norm_grad"):
        H = c["H"]
        s["residual"] = _normal((T, H), g, torch.float32, 2.0)
        s["gamma"] = (1.0 + _normal((H,), g, torch.float32, 0.1 ** 0.5)).to(torch.bfloat16)
        s["eps"] = 1e-6
        if op == "residual_norm":
            s["x"] = _normal((T, H), g, torch.bfloat16)
        else:
            s["d_out"] = _normal((T, H), g, torch.bfloat16)
            s["d_residual"] = _normal((T, H), g, torch.float32)
    else:
        ids = _expert_ids(c, g)
        if op == "route":
            s["ids"] = ids
        else:
            H, k, R = c["H"], c["k"], _rows(c)
            s["row_of"], s["slot_of"] = _plain_route(ids, c["E"], c["align"], R)[:2]
            if op == "dispatch":
                if c["fp8"]:
                    s["x"] = _normal((T, H), g, torch.float32, 64.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
                    s["sf"] = torch.rand((T, -(-H // 128)), generator=g, device=DEVICE) + 0.01
                else:
                    s["x"] = _normal((T, H), g, torch.bfloat16)
            elif op == "dispatch_grad":
                s["d_rows"] = _normal((R, H), g, torch.bfloat16)
            else:
                s["expert_out"] = _normal((R, H), g, torch.bfloat16)
                s["w"] = _weights(T, k, g)
                s["d_out"] = _normal((T, H), g, torch.float32 if c["fp32"] else torch.bfloat16)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The plan and the output buffers that a program keeps between calls."""
    import moe_finalize_residual_rmsnorm_gb300 as mfr
    c = s["case"]
    op, T = c["op"], c["T"]

    def new(shape, dtype):
        return torch.zeros(shape, device=DEVICE, dtype=dtype)
    if op == "route":
        s["plan"] = p = mfr.RoutePlan(T, c["k"], c["E"], align=c["align"], sentinel_skip=True)
        s["row_of"] = new((T, c["k"]), torch.int32)
        s["slot_of"] = new((p.R,), torch.int32)
        s["offsets"] = new((c["E"] + 1,), torch.int32)
        s["counts"] = new((c["E"],), torch.int32)
        s["workspace"] = new((p.workspace_bytes(),), torch.uint8)
    elif op == "dispatch":
        sf_bytes = 4 * s["sf"].shape[1] if c["fp8"] else 0
        s["plan"] = mfr.DispatchPlan(T, c["H"], c["k"], _rows(c), dtype=s["x"].dtype, sf_bytes=sf_bytes, sentinel_skip=True)
        s["rows"] = new((_rows(c), c["H"]), s["x"].dtype)
        s["sf_rows"] = new((_rows(c), s["sf"].shape[1]), torch.float32) if c["fp8"] else None
    elif op == "dispatch_grad":
        s["plan"] = mfr.DispatchPlan(T, c["H"], c["k"], _rows(c), sentinel_skip=True)
        s["d_x"] = new((T, c["H"]), torch.bfloat16)
    elif op == "finalize_grad":
        s["plan"] = mfr.FinalizeGradPlan(T, c["H"], c["k"], _rows(c), grad_dtype=s["d_out"].dtype, sentinel_skip=True)
        s["d_rows"] = new((_rows(c), c["H"]), torch.bfloat16)
        s["d_w"] = new((T, c["k"]), torch.float32)
    elif op == "residual_norm":
        quant = {"token": mfr.QUANT_TOKEN, "group128": mfr.QUANT_GROUP128, "mx32": mfr.QUANT_MX32}[c["scales"]]
        s["plan"] = p = mfr.ResidualNormPlan(T, c["H"], quant=quant,
                                             sf_layout=mfr.SF_TILED_128x4 if c["tiled"] else mfr.SF_ROW_MAJOR)
        s["residual_out"] = new((T, c["H"]), torch.float32)
        s["q"] = new((T, c["H"]), torch.float8_e4m3fn)
        s["scales"] = new(p.sf_shape(), torch.uint8 if c["scales"] == "mx32" else torch.float32)
        s["out"] = new((T, c["H"]), torch.bfloat16) if c["bf16_too"] else None
    else:
        s["plan"] = p = mfr.ResidualNormGradPlan(T, c["H"])
        s["workspace"] = new((p.workspace_bytes(),), torch.uint8)
        s["d_residual_in"] = new((T, c["H"]), torch.float32)
        s["d_x"] = new((T, c["H"]), torch.bfloat16)
        s["d_gamma"] = new((c["H"],), torch.float32)


# ---- the plain forms -----------------------------------------------------------------

def _plain_route(ids, E, align, R):
    """(row of each pair, pair of each row, block offsets, counts): pairs in order within their expert; a
    row that only pads its block holds -1, a row behind the last block -2; a pair without an expert here has row -1."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    first = torch.cumsum(counts, 0) - counts
    padded = (counts[:E] + align - 1) // align * align
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=ids.device), torch.cumsum(padded, 0)])
    sorted_key = key[order]
    row = offsets[sorted_key] + torch.arange(n, device=ids.device) - first[sorted_key]
    row = torch.where(sorted_key < E, row, torch.full_like(row, -1))
    row_of = torch.empty_like(row)
    row_of[order] = row
    slot_of = torch.where(torch.arange(R + 1, device=ids.device) < offsets[E], -1, -2)
    slot_of[torch.where(row < 0, torch.full_like(row, R), row)] = order
    return (row_of.view(ids.shape).to(torch.int32), slot_of[:R].to(torch.int32).contiguous(), offsets.to(torch.int32),
            counts[:E].to(torch.int32))


def _tile_scales(sf):
    """Scale (r, c) at byte (r % 32) * 16 + (r / 32 % 4) * 4 + c % 4 of its 128 x 4 tile, tiles row by row."""
    T, S = sf.shape
    tr, tc = -(-T // 128), -(-S // 4)
    full = torch.zeros((tr * 128, tc * 4), dtype=sf.dtype, device=sf.device)
    full[:T, :S] = sf
    return full.view(tr, 4, 32, tc, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _groups(y, size):
    """y in groups of `size` columns (0: whole rows), the last one filled up with zeros."""
    T, H = y.shape
    size = size or H
    n = -(-H // size)
    if n * size != H:
        y = torch.cat([y, torch.zeros((T, n * size - H), dtype=y.dtype, device=y.device)], 1)
    return y.view(T, n, size)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        row_of, slot_of, offsets, counts = _plain_route(s["ids"], c["E"], c["align"], _rows(c))
        return {"row_of": row_of, "slot_of": slot_of, "offsets": offsets, "counts": counts}
    if op == "dispatch":
        k, slot = c["k"], s["slot_of"].long()
        here = (slot >= 0)[:, None]
        token = torch.clamp(slot, min=0) // k
        bits = s["x"].view(torch.uint8 if c["fp8"] else torch.int16)
        rows = torch.where(here, bits[token], torch.zeros((), dtype=bits.dtype, device=bits.device)).view(s["x"].dtype)
        sf = torch.where(here, s["sf"][token], torch.zeros((), device=rows.device)) if c["fp8"] else None
        return {"rows": rows, "sf": sf}
    if op == "dispatch_grad":
        row = s["row_of"].long()
        picked = s["d_rows"][torch.clamp(row, min=0)].float()
        return {"d_x": torch.where((row >= 0)[..., None], picked, torch.zeros((), device=row.device)).sum(1).to(torch.bfloat16)}
    if op == "finalize_grad":
        k, slot, row = c["k"], s["slot_of"].long(), s["row_of"].long()
        dy = s["d_out"].float()
        at = torch.clamp(slot, min=0)
        d_rows = torch.where((slot >= 0)[:, None], s["w"].reshape(-1)[at][:, None] * dy[at // k],
                             torch.zeros((), device=row.device)).to(torch.bfloat16)
        dots = (s["expert_out"][torch.clamp(row, min=0)].float() * dy[:, None, :]).sum(-1)
        return {"d_rows": d_rows, "d_w": torch.where(row >= 0, dots, torch.zeros_like(dots))}
    gamma, eps = s["gamma"].float(), s["eps"]
    if op == "residual_norm":
        r = s["residual"] + s["x"].float()
        y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + eps) * gamma
        g = _groups(y, SCALE_GROUPS[c["scales"]])
        amax = torch.clamp(g.abs().amax(-1, keepdim=True), AMAX_FLOOR, FLOAT_MAX)
        if c["scales"] == "mx32":
            # the smallest power of two that brings the group's largest magnitude to 448 or below
            m, e = torch.frexp(amax)                                # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
            e = e - 9 + (m > 0.875).to(e.dtype)
            scale = (e + 127).to(torch.uint8)[..., 0]
            q = torch.ldexp(g, -e)
            scale = (_tile_scales(scale) if c["tiled"] else scale).view(torch.float8_e8m0fnu)
        else:
            scale = (amax / E4M3_MAX)[..., 0]
            q = g * (E4M3_MAX / amax)
        q = torch.clamp(q, -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        q = q.reshape(c["T"], -1)[:, :c["H"]].contiguous().view(torch.float8_e4m3fn)
        return {"residual": r, "q": q, "scales": scale, "out": y.to(torch.bfloat16) if c["bf16_too"] else None}
    # y = r * inv * gamma, inv = (mean(r^2) + eps)^-1/2
    r, dy = s["residual"], s["d_out"].float()
    inv = torch.rsqrt((r * r).mean(1, keepdim=True) + eps)
    dg = dy * gamma
    d_r = s["d_residual"] + inv * dg - r * (inv * inv * inv * (dg * r).mean(1, keepdim=True))
    return {"d_residual": d_r, "d_x": d_r.to(torch.bfloat16), "d_gamma": (dy * r * inv).sum(0)}


def _run_own(s):
    c, p = s["case"], s["plan"]
    op = c["op"]
    if op == "route":
        p.run(s["ids"], s["row_of"], s["slot_of"], s["offsets"], s["counts"], s["workspace"])
        return {"row_of": s["row_of"], "slot_of": s["slot_of"], "offsets": s["offsets"], "counts": s["counts"]}
    if op == "dispatch":
        p.run(s["x"], s["row_of"], s["slot_of"], s["rows"], s.get("sf"), s["sf_rows"])
        return {"rows": s["rows"], "sf": s["sf_rows"]}
    if op == "dispatch_grad":
        p.run_grad(s["d_rows"], s["row_of"], s["d_x"])
        return {"d_x": s["d_x"]}
    if op == "finalize_grad":
        p.run(s["d_out"], s["expert_out"], s["row_of"], s["slot_of"], s["w"], s["d_rows"], s["d_w"])
        return {"d_rows": s["d_rows"], "d_w": s["d_w"]}
    if op == "residual_norm":
        p.run(s["x"], s["residual"], s["residual_out"], s["gamma"], s["eps"], s["out"], s["q"], s["scales"])
        sf = s["scales"].view(torch.float8_e8m0fnu) if c["scales"] == "mx32" else s["scales"]
        return {"residual": s["residual_out"], "q": s["q"], "scales": sf, "out": s["out"]}
    p.run(s["d_out"], s["d_residual"], s["residual"], s["gamma"], s["eps"], s["d_residual_in"], s["d_gamma"],
          s["workspace"], s["d_x"])
    return {"d_residual": s["d_residual_in"], "d_x": s["d_x"], "d_gamma": s["d_gamma"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    c = case
    op, T = c["op"], c["T"]
    if op == "route":
        # ids read; row_of, slot_of, offsets and counts written
        return {"bytes": 4 * (2 * T * c["k"] + _rows(c) + 2 * c["E"] + 1), "flops": 0}
    H = c["H"]
    n = T * H
    if op == "residual_norm":
        S = n // (SCALE_GROUPS[c["scales"]] or H) * (1 if c["scales"] == "mx32" else 4)
        return {"bytes": n * (2 + 4 + 4 + 1 + (2 if c["bf16_too"] else 0)) + S + 2 * H, "flops": 8 * n}
    if op == "residual_norm_grad":
        return {"bytes": n * (2 + 4 + 4 + 4 + 2) + 2 * H + 4 * H, "flops": 14 * n}
    pairs = T * c["k"] * (1 - c["nonlocal_share"])      # rows with data (the pairs whose expert is here, on average)
    maps = 4 * T * c["k"]
    pad = 0 if c["align"] == 1 else min(c["E"], T * c["k"]) * (c["align"] - 1) / 2
    if op == "dispatch":
        row = H + 4 * -(-H // 128) if c["fp8"] else 2 * H
        return {"bytes": T * row + (pairs + pad) * row + maps + 4 * _rows(c), "flops": 0}
    if op == "dispatch_grad":
        return {"bytes": pairs * 2 * H + 2 * n + maps, "flops": pairs * H}
    return {"bytes": (2 * pairs + pad) * 2 * H + n * (4 if c["fp32"] else 2) + 3 * maps + 4 * _rows(c), "flops": 3 * pairs * H}


# ---- the definitions in 64 bits -----------------------------------------------------------

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c, op, T = case, case["op"], case["T"]
    if op == "route":
        return None                                             # whole numbers only
    H = c["H"]
    if op == "dispatch":
        out = torch.zeros((_rows(c), H), dtype=torch.float64, device=DEVICE)
        sf = torch.zeros((_rows(c), s["sf"].shape[1]), dtype=torch.float64, device=DEVICE) if c["fp8"] else None
        for j in range(c["k"]):
            row = s["row_of"][:, j].long()
            t = torch.nonzero(row >= 0)[:, 0]
            out[row[t]] = s["x"].to(torch.float64)[t]
            if sf is not None:
                sf[row[t]] = s["sf"].to(torch.float64)[t]
        return {"rows": out, "sf": sf}
    if op == "dispatch_grad":
        d_x = torch.zeros((T, H), dtype=torch.float64, device=DEVICE)
        for j in range(c["k"]):
            row = s["row_of"][:, j].long()
            t = torch.nonzero(row >= 0)[:, 0]
            d_x[t] += s["d_rows"][row[t]].to(torch.float64)
        return {"d_x": d_x}
    if op == "finalize_grad":
        d_rows = torch.zeros((_rows(c), H), dtype=torch.float64, device=DEVICE)
        d_w = torch.zeros((T, c["k"]), dtype=torch.float64, device=DEVICE)
        dy = s["d_out"].to(torch.float64)
        for j in range(c["k"]):
            row = s["row_of"][:, j].long()
            t = torch.nonzero(row >= 0)[:, 0]
            d_rows[row[t]] = dy[t] * s["w"][t, j].to(torch.float64)[:, None]
            d_w[t, j] = torch.einsum("th,th->t", s["expert_out"][row[t]].to(torch.float64), dy[t])
        return {"d_rows": d_rows, "d_w": d_w}
    gamma = s["gamma"].to(torch.float64)
    if op == "residual_norm":
        r = s["residual"].to(torch.float64) + s["x"].to(torch.float64)
        y = r / torch.sqrt(r.pow(2).sum(1, keepdim=True) / H + s["eps"]) * gamma
        size = SCALE_GROUPS[c["scales"]] or H
        q, scales = torch.empty_like(y), torch.empty((T, -(-H // size)), dtype=torch.float64, device=DEVICE)
        for n, a in enumerate(range(0, H, size)):
            top = y[:, a:a + size].abs().max(1).values.clamp(AMAX_FLOOR, FLOAT_MAX)
            scales[:, n] = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX))) if c["scales"] == "mx32" else top / E4M3_MAX
            q[:, a:a + size] = y[:, a:a + size] / scales[:, n, None]
        if c["tiled"]:
            S = scales.shape[1]
            tiled = torch.full((-(-T // 128) * 128 * (-(-S // 4) * 4),), 2.0 ** -127, dtype=torch.float64, device=DEVICE)
            t, b = torch.arange(T, device=DEVICE)[:, None], torch.arange(S, device=DEVICE)[None, :]
            tiled[(t // 128 * -(-S // 4) + b // 4) * 512 + t % 32 * 16 + t // 32 % 4 * 4 + b % 4] = scales
            scales = tiled
        return {"residual": r, "q": q, "scales": scales, "out": y if c["bf16_too"] else None}
    r, dy = s["residual"].to(torch.float64), s["d_out"].to(torch.float64)
    rms = torch.sqrt(r.pow(2).sum(1, keepdim=True) / H + s["eps"])
    unit = r / rms
    dn = dy * gamma
    d_r = s["d_residual"].to(torch.float64) + (dn - unit * (dn * unit).sum(1, keepdim=True) / H) / rms
    return {"d_residual": d_r, "d_x": d_r, "d_gamma": (dy * unit).sum(0)}
