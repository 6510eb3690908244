"""More operators of a MoE layer's step, as cases that can be measured.

  gate      router logits to the k experts of each token and their weights
  gate_grad its gradient: to the logits
  moe       a whole MoE layer for a few tokens: gated experts, their weighted sum (bf16, or E4M3 with scales)
  qk        RMSNorm of every query and key head with the position rotation in the same pass
  qk_grad   its gradient: to queries, keys and both gammas
  clip      the L2 norm of many gradient tensors together, and the gradients scaled to a largest norm

`run` computes a case in its plain form (elementary torch operations in 32
bits), or, with `own` set, through the package's entry points.
"""
import math

import torch

own = False

DEVICE = "cuda"
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
FLOAT_MAX = 3.4028234663852886e38
CLIP_EPS = 1e-6

# Hidden sizes 4096 and 8192, k = 8 and 64 to 256 experts are those of the
# repository's own workloads; the others are generic.
LISTED = [
    # one token of a decode step: eight experts' weights and nothing else
    {"name": "moe_one_token", "op": "moe", "T": 1, "H": 4096, "I": 1024, "E": 64, "k": 8, "fp8": False, "zipf": 0.0,
     "nonlocal_share": 0.0},
    # a small batch's decode step: most chosen experts have one or two tokens
    {"name": "moe_decode", "op": "moe", "T": 16, "H": 4096, "I": 1024, "E": 128, "k": 8, "fp8": False, "zipf": 0.0,
     "nonlocal_share": 0.0},
    # a ragged batch of odd sizes, popular experts, a quarter of the experts elsewhere
    {"name": "moe_ragged", "op": "moe", "T": 37, "H": 2056, "I": 712, "E": 32, "k": 6, "fp8": False, "zipf": 1.2,
     "nonlocal_share": 0.25},
    # a wide model in 8 bits, a large decode batch: every expert is read
    {"name": "moe_wide_fp8", "op": "moe", "T": 128, "H": 8192, "I": 1024, "E": 64, "k": 8, "fp8": True, "zipf": 0.0,
     "nonlocal_share": 0.0},
    # the router of a decode step
    {"name": "gate_decode", "op": "gate", "T": 8, "E": 128, "k": 8, "score": "softmax", "renormalize": True, "bias": False,
     "bf16": False, "masked": 0.0},
    # the router of a large prefill with sigmoid scores and a balancing bias
    {"name": "gate_prefill", "op": "gate", "T": 32768, "E": 256, "k": 8, "score": "sigmoid", "renormalize": True,
     "bias": True, "bf16": False, "masked": 0.0},
    # a training step's way back through the router, one token more than a power of two
    {"name": "gate_grad_train", "op": "gate_grad", "T": 16385, "E": 128, "k": 8, "score": "softmax", "renormalize": False,
     "bias": False, "bf16": False, "masked": 0.0},
    # a decode step's heads
    {"name": "qk_decode", "op": "qk", "T": 8, "heads_q": 32, "heads_k": 8, "D": 128, "rotary": 128, "interleaved": False,
     "packed": True, "fp16": False, "far": True},
    # a prefill's heads out of the packed projection
    {"name": "qk_prefill", "op": "qk", "T": 16384, "heads_q": 32, "heads_k": 8, "D": 128, "rotary": 128,
     "interleaved": False, "packed": True, "fp16": False, "far": False},
    # a training micro-batch: odd length, odd head size, a part of each head rotated in neighbouring pairs
    {"name": "qk_grad_ragged", "op": "qk_grad", "T": 4097, "heads_q": 24, "heads_k": 4, "D": 80, "rotary": 32,
     "interleaved": True, "packed": False, "fp16": False, "far": False},
    # the small tensors of an adapter-sized model
    {"name": "clip_small", "op": "clip", "tensors": 40, "total": 300000, "bf16_share": 0.5, "limit": 0.5},
    # a shard of a large model's gradients, 32 and 16 bits
    {"name": "clip_large", "op": "clip", "tensors": 60, "total": 700000000, "bf16_share": 0.7, "limit": 0.5},
]


def listed():
    return [dict(c) for c in LISTED]


def _log(rng, a, b):
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["gate", "gate_grad", "moe", "moe", "qk", "qk_grad", "clip"])
    if op in ("gate", "gate_grad"):
        E = _log(rng, 4, 512)
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "T": min(_log(rng, 1, 32768), 32768 * 256 // E), "E": E, "k": rng.randint(1, min(E, 16)),
                "score": score, "renormalize": rng.random() < 0.5, "bias": score == "sigmoid" and rng.random() < 0.7,
                "bf16": rng.random() < 0.4, "masked": rng.choice([0.0, 0.0, 0.3, 0.9])}
    if op == "moe":
        fp8 = rng.random() < 0.5
        E = _log(rng, 4, 128)
        H = 16 * _log(rng, 16, 512)
        I = 128 * _log(rng, 1, 16) if fp8 else 8 * _log(rng, 16, 256)
        T = _log(rng, 1, 256)
        most = (1 << 31) // (3 * H * I * (1 if fp8 else 2))       # experts of 2 GB of weights
        E = max(1, min(E, most))
        return {"op": op, "T": T, "H": H, "I": I, "E": E, "k": rng.randint(1, min(E, 8)), "fp8": fp8,
                "zipf": rng.choice([0.0, 1.2]), "nonlocal_share": rng.choice([0.0, 0.0, 0.25])}
    if op in ("qk", "qk_grad"):
        D = rng.choice([64, 80, 96, 128, 128, 192, 256])
        heads_k = rng.randint(1, 8)
        c = {"op": op, "T": _log(rng, 1, 16384), "heads_q": heads_k * rng.randint(1, 8), "heads_k": heads_k, "D": D,
             "rotary": rng.choice([D, D, 32, 64]), "interleaved": rng.random() < 0.4, "packed": rng.random() < 0.5,
             "fp16": rng.random() < 0.3, "far": rng.random() < 0.5}
        c["T"] = max(1, min(c["T"], (16384 * 40 * 128) // ((c["heads_q"] + c["heads_k"]) * D)))
        return c
    return {"op": op, "tensors": _log(rng, 1, 60), "total": _log(rng, 1000, 500000000),
            "bf16_share": rng.choice([0.0, 0.5, 1.0]), "limit": rng.choice([0.5, 0.9, 2.0])}


# ---- inputs ------------------------------------------------------------------------

def _normal(shape, g, dtype, scale=1.0):
    out = torch.empty(shape, device=DEVICE, dtype=dtype)
    flat, step = out.view(-1), 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        v = torch.randn(n, generator=g, device=DEVICE) * scale
        flat[i:i + n] = v.clamp_(-E4M3_MAX, E4M3_MAX) if dtype is torch.float8_e4m3fn else v
    return out


def _expert_ids(c, g):
    """k distinct experts a token by Gumbel top-k; a pair whose expert is on another GPU has id -1."""
    T, k, E = c["T"], c["k"], c["E"]
    logp = -c["zipf"] * torch.log(torch.arange(1, E + 1, device=DEVICE, dtype=torch.float32))
    u = torch.rand((T, E), generator=g, device=DEVICE).clamp_(1e-20, 1 - 1e-7)
    ids = torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices
    ids = torch.where(ids < round(E * (1 - c["nonlocal_share"])), ids, torch.full_like(ids, -1))
    return ids.to(torch.int32).contiguous()


def _clip_sizes(c):
    """Sizes of the tensors: a few matrices hold most, norms and biases of a few thousand values the rest."""
    n, total = c["tensors"], c["total"]
    share = [1.0 / (1 + i % 7) ** 3 for i in range(n)]
    return [max(1, int(total * s / sum(share)) + (i % 5) - 2) for i, s in enumerate(share)]


def _clip_types(c):
    n = c["tensors"]
    return [torch.bfloat16 if (i * 7 % 10) < 10 * c["bf16_share"] else torch.float32 for i in range(n)]


def _table(positions, rotary):
    """cos and sin of position * 10000^(-2 i / rotary), [positions, rotary]: cosines, then sines."""
    freq = 10000.0 ** (-torch.arange(0, rotary, 2, device=DEVICE, dtype=torch.float64) / rotary)
    a = torch.arange(positions, device=DEVICE, dtype=torch.float64)[:, None] * freq
    return torch.cat([torch.cos(a), torch.sin(a)], 1).to(torch.float32).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 1000003 + 29)
    op = c["op"]
    s = {"case": c}
    if op in ("gate", "gate_grad"):
        T, E = c["T"], c["E"]
        dtype = torch.bfloat16 if c["bf16"] else torch.float32
        logits = torch.randn((T, E), generator=g, device=DEVICE) * 1.5
        off = torch.rand((T, E), generator=g, device=DEVICE) < c["masked"]
        s["logits"] = torch.where(off, torch.full_like(logits, -math.inf), logits).to(dtype)
        s["bias"] = torch.randn((E,), generator=g, device=DEVICE) * 0.05 if c["bias"] else None
        if op == "gate_grad":
            s["ids"] = _plain_gate(s["logits"], s["bias"], c)[0]
            s["d_w"] = torch.randn((T, c["k"]), generator=g, device=DEVICE)
    elif op == "moe":
        T, H, I, E = c["T"], c["H"], c["I"], c["E"]
        s["ids"] = _expert_ids(c, g)
        s["w"] = torch.softmax(torch.randn((T, c["k"]), generator=g, device=DEVICE), 1).contiguous()
        if c["fp8"]:
            H128 = -(-H // 128)

            def scales(shape, typical):
                return ((0.5 + torch.rand(shape, generator=g, device=DEVICE)) * (typical / 64)).contiguous()
            s["x"], s["x_sf"] = _normal((T, H), g, torch.float8_e4m3fn, 64.0), scales((T, H128), 1.0)
            s["w13"], s["w13_sf"] = _normal((E, 2 * I, H), g, torch.float8_e4m3fn, 64.0), scales((E, 2 * I // 128, H128), H ** -0.5)
            s["w2"], s["w2_sf"] = _normal((E, H, I), g, torch.float8_e4m3fn, 64.0), scales((E, H128, I // 128), I ** -0.5)
        else:
            s["x"] = _normal((T, H), g, torch.bfloat16)
            s["w13"] = _normal((E, 2 * I, H), g, torch.bfloat16, H ** -0.5)
            s["w2"] = _normal((E, H, I), g, torch.bfloat16, I ** -0.5)
    elif op in ("qk", "qk_grad"):
        T, hq, hk, D = c["T"], c["heads_q"], c["heads_k"], c["D"]
        dtype = torch.float16 if c["fp16"] else torch.bfloat16
        if c["packed"]:                 # queries, keys and values as one projection writes them
            qkv = _normal((T, hq + 2 * hk, D), g, dtype, 2.0)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        else:
            s["q"], s["k"] = _normal((T, hq, D), g, dtype, 2.0), _normal((T, hk, D), g, dtype, 2.0)
        s["gamma_q"] = (1 + _normal((D,), g, torch.float32, 0.3)).to(dtype)
        s["gamma_k"] = (1 + _normal((D,), g, torch.float32, 0.3)).to(dtype)
        s["eps"] = 1e-6
        most = 131072 if c["far"] else 16384
        s["table"] = _table(most, c["rotary"])
        first = int(torch.randint(0, most, (1,), generator=torch.Generator().manual_seed(int(seed))))
        if c["far"]:                    # tokens of many requests, each at its own place
            s["positions"] = torch.randint(0, most, (T,), generator=g, device=DEVICE).to(torch.int32)
        else:                           # one sequence, from its start or further on
            s["positions"] = ((torch.arange(T, device=DEVICE) + first) % most).to(torch.int32)
        if op == "qk_grad":
            s["d_q_out"], s["d_k_out"] = _normal((T, hq, D), g, dtype), _normal((T, hk, D), g, dtype)
    else:
        sizes, types = _clip_sizes(c), _clip_types(c)
        s["grads"] = [_normal((n,), g, t, 1e-3) for n, t in zip(sizes, types)]
        s["max_norm"] = c["limit"] * 1e-3 * math.sqrt(sum(sizes))
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The plan and the output buffers that a program keeps between calls."""
    import moe_finalize_residual_rmsnorm_gb300 as mfr
    c = s["case"]
    op = c["op"]

    def new(shape, dtype):
        return torch.zeros(shape, device=DEVICE, dtype=dtype)
    if op in ("gate", "gate_grad"):
        T, k = c["T"], c["k"]
        s["plan"] = mfr.GatePlan(T, c["E"], k, score={"softmax": mfr.SCORE_SOFTMAX, "sigmoid": mfr.SCORE_SIGMOID}[c["score"]],
                                 renormalize=c["renormalize"], scale=1.0, dtype=s["logits"].dtype)
        if op == "gate":
            s["ids"], s["w"] = new((T, k), torch.int32), new((T, k), torch.float32)
        else:
            s["d_logits"] = new((T, c["E"]), s["logits"].dtype)
    elif op == "moe":
        s["plan"] = p = mfr.MoeLayerPlan(c["T"], c["H"], c["I"], c["E"], c["k"], dtype=s["x"].dtype, sentinel_skip=True)
        s["workspace"] = new((p.workspace_bytes(),), torch.uint8)
        s["out"] = new((c["T"], c["H"]), torch.bfloat16)
    elif op in ("qk", "qk_grad"):
        T, hq, hk, D = c["T"], c["heads_q"], c["heads_k"], c["D"]
        s["plan"] = p = mfr.QkNormRopePlan(T, hq, hk, D, rotary_dim=c["rotary"], interleaved=c["interleaved"],
                                           dtype=s["q"].dtype, max_positions=s["table"].shape[0])
        s["q_out"], s["k_out"] = new((T, hq, D), s["q"].dtype), new((T, hk, D), s["q"].dtype)
        if op == "qk_grad":
            s["d_gamma_q"], s["d_gamma_k"] = new((D,), torch.float32), new((D,), torch.float32)
            s["workspace"] = new((p.workspace_bytes(),), torch.uint8)
    else:
        s["plan"] = p = mfr.GradClipPlan([t.numel() for t in s["grads"]], [t.dtype for t in s["grads"]])
        s["workspace"] = new((p.workspace_bytes(),), torch.uint8)
        s["out"] = [torch.zeros_like(t) for t in s["grads"]]
        s["norm"] = new((1,), torch.float32)


# ---- the plain forms -----------------------------------------------------------------

def _plain_gate(logits, bias, c):
    """(ids, weights): the k largest keys, ties to the lowest index; a masked expert (-inf) is never chosen."""
    k = c["k"]
    l = logits.float()
    live = l > -math.inf
    if c["score"] == "sigmoid":
        key = torch.sigmoid(l.double())                     # in 64 bits: neighbouring keys are told apart
        key = key + bias.double() if bias is not None else l.double()
    else:
        key = l
    key = torch.where(live, key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    taken = torch.gather(live, 1, order)
    p = _plain_scores(l, c)
    w = torch.where(taken, torch.gather(p, 1, order), torch.zeros((), device=l.device))
    if c["renormalize"]:
        w = w / torch.where(taken.any(1, keepdim=True), w.sum(1, keepdim=True), torch.ones((), device=l.device))
    return torch.where(taken, order, torch.full_like(order, -1)).to(torch.int32), w


def _plain_scores(l, c):
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    top = torch.clamp(l.amax(1, keepdim=True), min=-FLOAT_MAX)
    e = torch.exp(l - top)
    if c["renormalize"]:
        return e                                            # the chosen ones' sum divides them
    return e / torch.clamp(e.sum(1, keepdim=True), min=2.0 ** -126)


def _plain_gate_grad(s):
    c, l, ids, g = s["case"], s["logits"].float(), s["ids"].long(), s["d_w"]
    live = ids >= 0
    at = torch.clamp(ids, min=0)
    p = _plain_scores(l, c)
    q = torch.where(live, torch.gather(p, 1, at), torch.zeros((), device=l.device))
    g = torch.where(live, g, torch.zeros_like(g))
    if c["renormalize"]:
        total = q.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        q = q / total
        d = g - (g * q).sum(1, keepdim=True)                # of the chosen scores, times the sum
        d = d * q if c["score"] == "softmax" else d / total
    else:
        d = g
    if c["score"] == "sigmoid":
        chosen = torch.gather(p, 1, at)
        d = d * chosen * torch.gather(1 / (1 + torch.exp(l)), 1, at)
    elif not c["renormalize"]:
        d = d * q
    d = torch.where(live, d, torch.zeros_like(d))
    out = torch.zeros_like(l).scatter_add_(1, at, d)        # the chosen of a token are distinct
    if c["score"] == "softmax" and not c["renormalize"]:
        out = out - p * (g * q).sum(1, keepdim=True)
    return out.to(s["logits"].dtype)


def _blocks(w, sf):
    """Codes [..., R, C] times their scales, one for 128 x 128 of them."""
    rows = torch.arange(w.shape[-2], device=w.device) // 128
    cols = torch.arange(w.shape[-1], device=w.device) // 128
    return w.float() * sf[:, rows][:, :, cols]


def _columns(x, sf):
    return x.float() * sf[:, torch.arange(x.shape[1], device=x.device) // 128]


def _requantised(h):
    """h in E4M3 with one scale for 128 columns, as the values it stands for."""
    y = h.reshape(*h.shape[:-1], h.shape[-1] // 128, 128)
    amax = torch.clamp(y.abs().amax(-1, keepdim=True), AMAX_FLOOR, FLOAT_MAX)
    q = torch.clamp(y * (E4M3_MAX / amax), -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float()
    return (q * (amax / E4M3_MAX)).reshape(h.shape)


def _plain_moe(s):
    c, ids, w = s["case"], s["ids"].long(), s["w"]
    T, I, E, k, fp8 = c["T"], c["I"], c["E"], c["k"], c["fp8"]
    x = _columns(s["x"], s["x_sf"]) if fp8 else s["x"].float()
    live = ids >= 0
    w = torch.where(live, w, torch.zeros_like(w))
    if T * k <= E:                      # few pairs: each with its own expert's weights
        e = torch.clamp(ids, min=0).reshape(-1)
        rows = x[torch.arange(T * k, device=x.device) // k][:, None, :]
    else:                               # every expert with every token
        e = torch.arange(E, device=x.device)
        rows = x[None]
    w13 = _blocks(s["w13"][e], s["w13_sf"][e]) if fp8 else s["w13"][e].float()
    both = torch.matmul(rows, w13.transpose(1, 2))
    del w13
    gate, up = both[..., :I], both[..., I:]
    h = gate / (1 + torch.exp(-gate)) * up
    h = _requantised(h) if fp8 else h
    w2 = _blocks(s["w2"][e], s["w2_sf"][e]) if fp8 else s["w2"][e].float()
    y = torch.matmul(h, w2.transpose(1, 2))
    if T * k <= E:
        return (y.view(T, k, -1) * w[..., None]).sum(1).to(torch.bfloat16)
    share = (torch.where(ids[..., None] == e, w[..., None], torch.zeros((), device=x.device))).sum(1)     # [T, E]
    return (y * share.t()[..., None]).sum(0).to(torch.bfloat16)


def _pairs(x, rotary, interleaved):
    """First and second members of the pairs that turn together."""
    r = x[..., :rotary]
    return (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rotary // 2], r[..., rotary // 2:])


def _joined(a, b, rest, interleaved):
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _plain_qk(s):
    c = s["case"]
    cs = s["table"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :c["rotary"] // 2], cs[..., c["rotary"] // 2:]

    def one(x, gamma):
        x = x.float()
        n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * gamma.float()
        a, b = _pairs(n, c["rotary"], c["interleaved"])
        return _joined(a * cos - b * sin, a * sin + b * cos, n[..., c["rotary"]:], c["interleaved"]).to(s["q"].dtype)
    return {"q": one(s["q"], s["gamma_q"]), "k": one(s["k"], s["gamma_k"])}


def _plain_qk_grad(s):
    c = s["case"]
    cs = s["table"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :c["rotary"] // 2], cs[..., c["rotary"] // 2:]

    def one(d_out, x, gamma):
        d, x = d_out.float(), x.float()
        a, b = _pairs(d, c["rotary"], c["interleaved"])
        d = _joined(a * cos + b * sin, b * cos - a * sin, d[..., c["rotary"]:], c["interleaved"])
        inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
        dn = d * gamma.float()
        d_x = inv * dn - x * (inv * inv * inv * (dn * x).mean(-1, keepdim=True))
        return d_x.to(s["q"].dtype), (d * x * inv).sum(1).sum(0)
    d_q, d_gamma_q = one(s["d_q_out"], s["q"], s["gamma_q"])
    d_k, d_gamma_k = one(s["d_k_out"], s["k"], s["gamma_k"])
    return {"d_q": d_q, "d_k": d_k, "d_gamma_q": d_gamma_q, "d_gamma_k": d_gamma_k}


def _plain_clip(s):
    squares = torch.stack([(t.float() * t.float()).sum() for t in s["grads"]])
    norm = torch.sqrt(squares.sum())
    scale = torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)
    scale = torch.where(torch.isfinite(norm), scale, torch.ones_like(scale))
    return {"norm": norm.reshape(1), "out": [(t.float() * scale).to(t.dtype) for t in s["grads"]]}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "gate":
        ids, w = _plain_gate(s["logits"], s["bias"], s["case"])
        return {"ids": ids, "w": w}
    if op == "gate_grad":
        return {"d_logits": _plain_gate_grad(s)}
    if op == "moe":
        return {"out": _plain_moe(s)}
    if op == "qk":
        return _plain_qk(s)
    if op == "qk_grad":
        return _plain_qk_grad(s)
    return _plain_clip(s)


def _run_own(s):
    op, p = s["case"]["op"], s["plan"]
    if op == "gate":
        p.run(s["logits"], s["ids"], s["w"], s["bias"])
        return {"ids": s["ids"], "w": s["w"]}
    if op == "gate_grad":
        p.run_grad(s["d_w"], s["logits"], s["ids"], s["d_logits"])
        return {"d_logits": s["d_logits"]}
    if op == "moe":
        p.run(s["x"], s["ids"], s["w"], s["w13"], s["w2"], s["out"], s["workspace"], s.get("x_sf"), s.get("w13_sf"),
              s.get("w2_sf"))
        return {"out": s["out"]}
    if op == "qk":
        p.run(s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["eps"], s["table"], s["positions"], s["q_out"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "qk_grad":
        p.run_grad(s["d_q_out"], s["d_k_out"], s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["eps"], s["table"],
                   s["positions"], s["q_out"], s["k_out"], s["d_gamma_q"], s["d_gamma_k"], s["workspace"])
        return {"d_q": s["q_out"], "d_k": s["k_out"], "d_gamma_q": s["d_gamma_q"], "d_gamma_k": s["d_gamma_k"]}
    p.run(s["grads"], s["max_norm"], s["norm"], s["workspace"], s["out"], eps=CLIP_EPS)
    return {"norm": s["norm"], "out": s["out"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ------------------------------------------------------

def _chosen_experts(c):
    """Experts of this GPU that at least one of the pairs chooses, on average."""
    E, local = c["E"], round(c["E"] * (1 - c["nonlocal_share"]))
    p = [(e + 1.0) ** -c["zipf"] for e in range(E)]
    total = sum(p)
    return sum(1 - max(0.0, 1 - c["k"] * p[e] / total) ** c["T"] for e in range(local))


def work(case):
    c = case
    op = c["op"]
    if op in ("gate", "gate_grad"):
        n, size = c["T"] * c["E"], 2 if c["bf16"] else 4
        pairs = 8 * c["T"] * c["k"]
        if op == "gate":
            return {"bytes": n * size + pairs + (4 * c["E"] if c["bias"] else 0), "flops": 4 * n}
        return {"bytes": 2 * n * size + pairs, "flops": 6 * n}
    if op == "moe":
        T, H, I, k, size = c["T"], c["H"], c["I"], c["k"], 1 if c["fp8"] else 2
        weights = _chosen_experts(c) * 3 * H * I * size
        return {"bytes": weights + T * H * (size + 2) + 8 * T * k,
                "flops": 6 * T * k * (1 - c["nonlocal_share"]) * H * I}
    if op in ("qk", "qk_grad"):
        n = c["T"] * (c["heads_q"] + c["heads_k"]) * c["D"]
        rows = min(c["T"], 16384) * c["rotary"] * 4 + 4 * c["T"]
        if op == "qk":
            return {"bytes": 2 * n * 2 + rows, "flops": 9 * n}
        return {"bytes": 3 * n * 2 + rows + 12 * c["D"], "flops": 16 * n}
    n = [(a, 2 if t is torch.bfloat16 else 4) for a, t in zip(_clip_sizes(c), _clip_types(c))]
    return {"bytes": 2 * sum(a * b for a, b in n) + 4, "flops": 3 * sum(a for a, _ in n)}


# ---- the definitions in 64 bits -----------------------------------------------------------

def _exact_gate(s):
    c, k = s["case"], s["case"]["k"]
    l = s["logits"].to(torch.float64)
    masked = torch.isinf(l)
    p = 1 / (1 + torch.exp(-l)) if c["score"] == "sigmoid" else torch.softmax(torch.where(masked, torch.full_like(l, -1e300), l), 1)
    p = torch.where(masked, torch.zeros_like(p), p)
    return l, masked, p


def _exact_moe(s):
    c = s["case"]
    T, H, I = c["T"], c["H"], c["I"]
    D = torch.float64
    out = torch.zeros((T, H), dtype=D, device=DEVICE)
    ids = s["ids"]
    for e in range(c["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        x, w13, w2 = s["x"][t].to(D), s["w13"][e].to(D), s["w2"][e].to(D)
        if c["fp8"]:
            x = x * torch.repeat_interleave(s["x_sf"][t].to(D), 128, 1)[:, :H]
            w13 = w13 * torch.repeat_interleave(torch.repeat_interleave(s["w13_sf"][e].to(D), 128, 0), 128, 1)[:, :H]
            w2 = w2 * torch.repeat_interleave(torch.repeat_interleave(s["w2_sf"][e].to(D), 128, 0)[:H], 128, 1)
        g, u = (x @ w13[:I].t()), (x @ w13[I:].t())
        h = g * torch.sigmoid(g) * u
        if c["fp8"]:
            for a in range(0, I, 128):
                top = h[:, a:a + 128].abs().max(1, keepdim=True).values.clamp(AMAX_FLOOR, FLOAT_MAX)
                h[:, a:a + 128] = (h[:, a:a + 128] / top * E4M3_MAX).to(torch.float8_e4m3fn).to(D) * top / E4M3_MAX
        out.index_add_(0, t, s["w"][t, j].to(D)[:, None] * (h @ w2.t()))
    return {"out": out}


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c, op, D = case, case["op"], torch.float64
    if op in ("gate", "gate_grad"):
        l, masked, p = _exact_gate(s)
        if op == "gate":
            key = p if s["bias"] is None else p + s["bias"].to(D)
            key = l if s["bias"] is None else torch.where(masked, torch.full_like(key, -math.inf), key)
            order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["k"]]
            w = torch.gather(p, 1, order)
            if c["renormalize"]:
                total = w.sum(1, keepdim=True)
                w = torch.where(total > 0, w / total, torch.zeros_like(w))
            return {"ids": None, "w": w}
        # by differentiation of the weights with the choice held fixed
        l = torch.where(masked, torch.full_like(l, -1e300), l).requires_grad_(True)
        at = s["ids"].long().clamp(min=0)
        live = (s["ids"] >= 0).to(D)
        q = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
        w = torch.gather(q, 1, at) * live
        if c["renormalize"]:
            if c["score"] == "softmax":
                w = torch.softmax(torch.where(live > 0, torch.gather(l, 1, at), torch.full_like(w, -1e300)), 1) * live
            else:
                w = w / torch.where(live.sum(1, keepdim=True) > 0, w.sum(1, keepdim=True), torch.ones_like(w[:, :1]))
        (w * s["d_w"].to(D)).sum().backward()
        return {"d_logits": l.grad}
    if op == "moe":
        return _exact_moe(s)
    if op in ("qk", "qk_grad"):
        T, rot = c["T"], c["rotary"]
        cs = s["table"].to(D)[s["positions"].long()]
        turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None, :]

        def one(x, gamma):
            n = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["D"] + s["eps"]) * gamma
            r = n[..., :rot].reshape(*n.shape[:-1], rot // 2, 2) if c["interleaved"] else \
                n[..., :rot].reshape(*n.shape[:-1], 2, rot // 2).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(r.contiguous()) * turn)
            z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
            return torch.cat([z, n[..., rot:]], -1)
        grad = op == "qk_grad"
        q, k, gq, gk = (s[n].detach().to(D).clone().requires_grad_(grad) for n in ("q", "k", "gamma_q", "gamma_k"))
        a, b = one(q, gq), one(k, gk)
        if not grad:
            return {"q": a, "k": b}
        ((a * s["d_q_out"].to(D)).sum() + (b * s["d_k_out"].to(D)).sum()).backward()
        return {"d_q": q.grad, "d_k": k.grad, "d_gamma_q": gq.grad, "d_gamma_k": gk.grad}
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(t.to(D)) for t in s["grads"]]))
    scale = min(1.0, s["max_norm"] / (float(norm) + CLIP_EPS))
    return {"norm": norm.reshape(1), "out": [t.to(D) * scale for t in s["grads"]]}
