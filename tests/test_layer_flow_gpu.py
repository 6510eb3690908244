"""The operators around the finalize as they are used: a MoE block forwards in
8 bits, a training step there and back, many calls in a row without a wait,
captured graphs, several streams."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import layer_ref as ref
import moe_finalize_residual_rmsnorm_gb300 as mfr

pytestmark = pytest.mark.gpu

I32, F32, B16, FP8 = torch.int32, torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


def new(shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def randn(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


class Route:
    def __init__(self, T, k, E, align=1, **kw):
        self.plan = mfr.RoutePlan(T, k, E, align=align, sentinel_skip=True, **kw)
        self.R = self.plan.R
        self.row_of, self.slot_of = new((T, k), I32), new((self.R,), I32)
        self.offsets, self.counts = new((E + 1,), I32), new((E,), I32)
        self.ws = new((self.plan.workspace_bytes(),), torch.uint8)

    def run(self, ids, stream=None):
        self.plan.run(ids, self.row_of, self.slot_of, self.offsets, self.counts, self.ws, stream)


@pytest.mark.parametrize("T,H,k,E,align", [(1, 4096, 8, 32, 128), (37, 1024, 4, 8, 16), (300, 2048, 8, 64, 128)])
def test_block_forward_in_8_bits(T, H, k, E, align):
    """Norm to E4M3 and bf16, sort, dispatch of codes and scales, experts that
    read them, the fused finalize."""
    eps = 1e-6
    x, res = randn((T, H), 1, B16), randn((T, H), 2)
    g1, g2 = (1 + 0.2 * randn((H,), 3)).to(B16), (1 + 0.2 * randn((H,), 4)).to(B16)
    ids = torch.from_numpy(ref.draw_ids(T, k, E, seed=5)).cuda()
    w = torch.softmax(randn((T, k), 6), 1)
    scale_of = 2.0 ** (torch.arange(E, device="cuda") % 3 - 1)        # an expert: times a power of two
    S = -(-H // 128)
    norm = mfr.ResidualNormPlan(T, H)
    r, y, q, sf = new((T, H)), new((T, H), B16), new((T, H), FP8), new((T, S))
    norm.run(x, res, r, g1, eps, y, q, sf)
    route = Route(T, k, E, align)
    route.run(ids)
    disp = mfr.DispatchPlan(T, H, k, route.R, dtype=FP8, sf_bytes=4 * S, sentinel_skip=True)
    rows, rows_sf = new((route.R, H), FP8), new((route.R, S))
    disp.run(q, route.row_of, route.slot_of, rows, sf, rows_sf)
    expert = torch.searchsorted(route.offsets[1:].long(), torch.arange(route.R, device="cuda"), right=True).clamp(max=E - 1)
    full = rows.float() * torch.repeat_interleave(rows_sf, 128, dim=1)[:, :H] * scale_of[expert][:, None]
    expert_out = full.to(B16)
    r2, z = mfr.moe_finalize_residual_rmsnorm(expert_out, route.row_of, w, r, g2, eps)
    torch.cuda.synchronize()
    # in 64 bits from the codes: the weighted sum takes bf16 rows, everything before is exact
    value = ref.f64(q) * np.repeat(ref.f64(sf), 128, axis=1)[:, :H]
    ids_h, w_h = ids.cpu().numpy(), ref.f64(w)
    terms = value[:, None, :] * ref.f64(scale_of)[ids_h][..., None] * w_h[..., None]
    want = ref.f64(r) + terms.sum(1)
    tol = (ref.BF16 + (k + 2) * ref.U) * np.abs(terms).sum(1) + (k + 2) * ref.U * np.abs(ref.f64(r)) + ref.TINY
    ref.assert_within(ref.f64(r2), want, tol, "residual_out")
    # and the codes stand for the norm: half a step of E4M3 each
    _, y64, _ = ref.residual_norm(ref.f64(x), res.cpu().numpy(), ref.f64(g1), eps)
    size = np.repeat(ref.f64(sf), 128, axis=1)[:, :H]
    ref.assert_within(value, y64, np.maximum(ref.E4M3 * np.abs(y64), size * 2.0 ** -10) * (1 + 2.0 ** -10), "codes")
    ref.assert_within(ref.f64(y), y64, (ref.BF16 + 2 * ref.Y_REL) * np.abs(y64) + ref.TINY, "bf16")
    assert norm.get_status() == route.plan.get_status() == disp.get_status() == 0


class Block:
    """r = res + x; y = norm(r) g1; rows = dispatch(y); E = rows * s[expert]; r2, z = finalize(E, w, r, g2)."""

    def __init__(self, T, H, k, E, align, pdl=True):
        self.T, self.H, self.k, self.E = T, H, k, E
        kw = dict(enable_pdl=pdl)
        self.route = Route(T, k, E, align, **kw)
        R = self.route.R
        kws = dict(sentinel_skip=True, **kw)
        self.norm = mfr.ResidualNormPlan(T, H, quant=mfr.QUANT_NONE, **kw)
        self.disp = mfr.DispatchPlan(T, H, k, R, **kws)
        self.fin = mfr.Plan(T, H, k, R, **kws)
        self.fin_grad = mfr.FinalizeGradPlan(T, H, k, R, grad_dtype=F32, **kws)
        self.norm_grad = mfr.ResidualNormGradPlan(T, H, **kw)
        self.ws = new((self.norm_grad.workspace_bytes(),), torch.uint8)
        self.b = {n: new(s, d) for n, s, d in (
            ("r", (T, H), F32), ("y", (T, H), B16), ("rows", (R, H), B16), ("r2", (T, H), F32), ("z", (T, H), B16),
            ("d_r2", (T, H), F32), ("d_g2", (H,), F32), ("d_E", (R, H), B16), ("d_w", (T, k), F32), ("d_y", (T, H), B16),
            ("d_r", (T, H), F32), ("d_x", (T, H), B16), ("d_g1", (H,), F32))}

    def forward(self, i):
        b, m = self.b, self.route
        self.norm.run(i["x"], i["res"], b["r"], i["g1"], i["eps"], b["y"])
        m.run(i["ids"])
        self.disp.run(b["y"], m.row_of, m.slot_of, b["rows"])
        b["E"] = b["rows"] * self.row_scale(i)
        self.fin.run(b["E"], m.row_of, i["w"], b["r"], b["r2"], i["g2"], i["eps"], b["z"])

    def row_scale(self, i):
        at = torch.arange(self.route.R, device="cuda")
        e = torch.searchsorted(self.route.offsets[1:].long(), at, right=True).clamp(max=self.E - 1)
        return i["s"][e][:, None].to(B16)                  # powers of two: exact

    def backward(self, i):
        b, m = self.b, self.route
        self.norm_grad.run(i["gz"], i["gr"], b["r2"], i["g2"], i["eps"], b["d_r2"], b["d_g2"], self.ws)
        self.fin_grad.run(b["d_r2"], b["E"], m.row_of, m.slot_of, i["w"], b["d_E"], b["d_w"])
        b["d_rows"] = b["d_E"] * self.row_scale(i)
        self.disp.run_grad(b["d_rows"], m.row_of, b["d_y"])
        self.norm_grad.run(b["d_y"], b["d_r2"], b["r"], i["g1"], i["eps"], b["d_r"], b["d_g1"], self.ws, b["d_x"])

    def status(self):
        return [p.get_status() for p in (self.route.plan, self.norm, self.disp, self.fin, self.fin_grad, self.norm_grad)]


def block_inputs(T, H, k, E, seed=0, share=0.0):
    return dict(x=randn((T, H), seed + 1, B16), res=randn((T, H), seed + 2), g1=(1 + 0.2 * randn((H,), seed + 3)).to(B16),
                g2=(1 + 0.2 * randn((H,), seed + 4)).to(B16), w=torch.softmax(randn((T, k), seed + 5), 1), eps=1e-5,
                ids=torch.from_numpy(ref.draw_ids(T, k, E, seed=seed + 6, nonlocal_share=share)).cuda(),
                s=2.0 ** (torch.arange(E, device="cuda") % 3 - 1), gz=randn((T, H), seed + 7, B16), gr=randn((T, H), seed + 8))


def block_in_64_bits(i, rounded):
    """The block's gradients by automatic differentiation in 64 bits on the
    CPU; with `rounded`, values and gradients rounded to bf16 where the block keeps
    them in bf16."""
    class Round(torch.autograd.Function):
        @staticmethod
        def forward(ctx, v, fwd, bwd):
            ctx.bwd = bwd
            return v.to(B16).to(torch.float64) if fwd else v.clone()

        @staticmethod
        def backward(ctx, g):
            return (g.to(B16).to(torch.float64) if ctx.bwd else g), None, None
    leaf = {n: i[n].detach().cpu().to(torch.float64).requires_grad_() for n in ("x", "res", "g1", "g2", "w")}
    ids, s = i["ids"].cpu().long(), i["s"].cpu().to(torch.float64)
    eps = float(np.float32(i["eps"]))

    def norm(r, g):
        return r * torch.rsqrt((r * r).mean(1, keepdim=True) + eps) * g
    r = leaf["res"] + leaf["x"]
    y = Round.apply(norm(r, leaf["g1"]), rounded, rounded)          # y and d_y
    acc = torch.zeros_like(r)
    for j in range(ids.shape[1]):
        here = (ids[:, j] >= 0).to(torch.float64)[:, None]
        E = Round.apply(y, False, rounded) * s[ids[:, j].clamp(min=0)][:, None]     # d_E
        acc = acc + here * leaf["w"][:, j:j + 1] * E
    r2 = r + acc
    z = norm(r2, leaf["g2"])
    loss = (z * i["gz"].cpu().to(torch.float64)).sum() + (r2 * i["gr"].cpu().to(torch.float64)).sum()
    grads = torch.autograd.grad(loss, list(leaf.values()))
    return dict(zip(leaf, (g.numpy() for g in grads)), r2=r2.detach().numpy(), z=z.detach().numpy())


@pytest.mark.parametrize("T,H,k,E,align,share,pdl", [(5, 64, 2, 4, 1, 0.0, True), (130, 1032, 8, 16, 16, 0.2, True),
                                                     (64, 4096, 6, 32, 128, 0.0, False)])
def test_training_step(T, H, k, E, align, share, pdl):
    """Every gradient of the block against automatic differentiation in 64
    bits.  What the block rounds to bf16 on its way (y, the rows' gradients,
    d_y) is rounded there too, once without: the difference of the two is what
    such roundings do, and the block, whose other steps are FP32 (1e-6 of the
    norm), may be as far from the unrounded one and a quarter more (another
    draw of the same roundings)."""
    i = block_inputs(T, H, k, E, seed=T, share=share)
    blk = Block(T, H, k, E, align, pdl)
    blk.forward(i)
    blk.backward(i)
    torch.cuda.synchronize()
    assert blk.status() == [0] * 6
    exact, rounded = block_in_64_bits(i, False), block_in_64_bits(i, True)
    b = blk.b
    for name, got in (("r2", b["r2"]), ("z", b["z"]), ("res", b["d_r"]), ("x", b["d_x"]), ("g1", b["d_g1"]),
                      ("g2", b["d_g2"]), ("w", b["d_w"])):
        off = np.linalg.norm(ref.f64(got) - exact[name])
        # z and d_x are themselves rounded to bf16 at the end
        last = ref.BF16 if got.dtype == B16 else 0.0
        allowed = 1.25 * np.linalg.norm(rounded[name] - exact[name]) + (last + 1e-5) * np.linalg.norm(exact[name])
        assert off <= allowed, (name, off, allowed)
    # and against differences: along a direction, the change of the 64-bit loss
    rng = np.random.default_rng(1)
    h = 1e-4
    v = {n: torch.from_numpy(rng.normal(size=i[n].shape)) for n in ("res", "w")}

    def loss(step):
        j = dict(i)
        for n in v:
            j[n] = i[n].cpu().to(torch.float64) + step * v[n]
        e = block_in_64_bits(j, False)
        return (e["z"] * ref.f64(i["gz"])).sum() + (e["r2"] * ref.f64(i["gr"])).sum()
    diff = (loss(h) - loss(-h)) / (2 * h)
    mine = (ref.f64(b["d_r"]) * v["res"].numpy()).sum() + (ref.f64(b["d_w"]) * v["w"].numpy()).sum()
    bound = sum((1.25 * np.linalg.norm(rounded[n] - exact[n]) + 1e-5 * np.linalg.norm(exact[n])) * np.linalg.norm(v[n].numpy())
                for n in v)
    assert abs(diff - mine) <= bound + 1e-4 * abs(diff)


def test_calls_in_a_row_without_a_wait():
    """Sort and dispatch of changing ids into the same buffers and on to a copy,
    fifty times with nothing waited for: with dependent launch a call that read
    its maps too early would see the call before's."""
    T, H, k, E = 48, 512, 4, 16
    m = Route(T, k, E, 4)
    disp = mfr.DispatchPlan(T, H, k, m.R, sentinel_skip=True)
    fg = mfr.FinalizeGradPlan(T, H, k, m.R, sentinel_skip=True)
    x = [randn((T, H), s, B16) for s in range(50)]
    ids = [torch.from_numpy(ref.draw_ids(T, k, E, seed=s, nonlocal_share=0.1)).cuda() for s in range(50)]
    w = randn((T, k), 1)
    rows, dE, dw, d_x = new((m.R, H), B16), new((m.R, H), B16), new((T, k)), new((T, H), B16)
    kept = []
    torch.cuda.synchronize()
    for s in range(50):
        m.run(ids[s])
        disp.run(x[s], m.row_of, m.slot_of, rows)
        fg.run(x[s], rows, m.row_of, m.slot_of, w, dE, dw)
        disp.run_grad(rows, m.row_of, d_x)
        kept.append((m.row_of.clone(), dw.clone(), d_x.clone()))
    torch.cuda.synchronize()
    for s, (row_of, got, got_x) in enumerate(kept):
        want = ref.route(ids[s].cpu().numpy(), E, 4)[0]
        assert np.array_equal(row_of.cpu().numpy(), want), s
        sq = (ref.f64(x[s]) ** 2).sum(1)[:, None] * (want >= 0)
        ref.assert_within(ref.f64(got), sq, ref.CHAIN * ref.U * sq, f"d_w of call {s}")
        many = (want >= 0).sum(1)[:, None] * ref.f64(x[s])
        ref.assert_within(ref.f64(got_x), many, (ref.BF16 + 2 * k * ref.U) * np.abs(many), f"d_x of call {s}")
    assert m.plan.get_status() == disp.get_status() == fg.get_status() == 0


@pytest.mark.parametrize("pdl", [True, False])
def test_two_launch_route_of_changing_ids(pdl):
    """Ids that change in place before each call of the two-launch form, whose
    second launch reads them before it waits for the first."""
    T, k, E = 5000, 8, 24
    m = Route(T, k, E, enable_pdl=pdl)
    assert m.ws.numel() > 0
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = [torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=I32) for _ in range(20)]
    at, kept = new((T, k), I32), []
    torch.cuda.synchronize()
    for i in ids:
        at.copy_(i)
        m.run(at)
        kept.append(m.row_of.clone())
    torch.cuda.synchronize()
    for i, row_of in zip(ids, kept):
        order = torch.argsort(i.view(-1).long(), stable=True)
        assert torch.equal(row_of.view(-1).long()[order], torch.arange(T * k, device="cuda"))
    assert m.plan.get_status() == 0


def test_captured_two_launch_route_and_gradient():
    """The calls of two launches (a large route, the norm's gradient) captured
    into one graph and replayed on other inputs."""
    T, k, E, H = 6000, 8, 100, 1032
    m = Route(T, k, E, 16)
    n = mfr.ResidualNormGradPlan(T, H)
    ws, d_in, d_g = new((n.workspace_bytes(),), torch.uint8), new((T, H)), new((H,))
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = new((T, k), I32)
    d, r, gamma = randn((T, H), 1, B16), randn((T, H), 2), (1 + 0.1 * randn((H,), 3)).to(B16)

    def calls():
        n.run(d, None, r, gamma, 1e-6, d_in, d_g, ws)
        m.run(ids)
        n.run(d, d_in, r, gamma, 1e-6, d_in, d_g, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            calls()
    torch.cuda.synchronize()
    for _ in range(5):
        ids.copy_(torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=I32))
        r.copy_(torch.randn((T, H), generator=g, device="cuda"))
        graph.replay()
        order = torch.argsort(ids.view(-1).long(), stable=True)
        replayed = [t.clone() for t in (m.row_of, m.slot_of, m.offsets, m.counts, d_in, d_g)]
        slots = m.slot_of[m.slot_of >= 0].long()
        assert torch.equal(slots, order)
        calls()
        assert all(torch.equal(a, b) for a, b in zip(replayed, (m.row_of, m.slot_of, m.offsets, m.counts, d_in, d_g)))
    assert m.plan.get_status() == n.get_status() == 0


def test_the_same_bits_every_time_and_in_a_graph():
    """Eager runs, a replayed graph and a graph replayed on new inputs give the
    same bits as eager runs on those inputs."""
    T, H, k, E = 700, 1032, 8, 32
    i = block_inputs(T, H, k, E, seed=3)
    blk = Block(T, H, k, E, 16)

    def outputs():
        torch.cuda.synchronize()
        return [blk.b[n].clone() for n in ("r", "y", "r2", "z", "d_r2", "d_g2", "d_w", "d_y", "d_r", "d_x", "d_g1")] + \
            [blk.route.row_of.clone(), blk.route.slot_of.clone()]
    blk.forward(i)
    blk.backward(i)
    first = outputs()
    for _ in range(3):
        blk.forward(i)
        blk.backward(i)
        assert all(torch.equal(a, b) for a, b in zip(first, outputs()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            blk.forward(i)
            blk.backward(i)
    for t in blk.b.values():
        t.zero_()
    torch.cuda.synchronize()
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, outputs()))
    j = block_inputs(T, H, k, E, seed=50)
    for n, t in i.items():
        if isinstance(t, torch.Tensor):
            t.copy_(j[n])
    torch.cuda.synchronize()
    g.replay()
    replayed = outputs()
    blk.forward(j)
    blk.backward(j)
    assert all(torch.equal(a, b) for a, b in zip(replayed, outputs()))
    assert not torch.equal(replayed[0], first[0])


@pytest.mark.parametrize("T", [64, 40000])
def test_one_plan_on_two_streams(T):
    """The same plans on two streams at once, each with its own buffers and
    workspaces (T = 40000: the two-launch route, which has one)."""
    H, k, E = 256, 8, 16
    plan = mfr.RoutePlan(T, k, E)
    norm = mfr.ResidualNormGradPlan(T, H)
    streams = [torch.cuda.Stream() for _ in range(2)]
    state = []
    for s in range(2):
        g = torch.Generator(device="cuda").manual_seed(s)
        ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=I32)
        state.append(dict(ids=ids, out=[new((T, k), I32), new((plan.R,), I32), new((E + 1,), I32), new((E,), I32)],
                          ws=new((plan.workspace_bytes(),), torch.uint8), d=randn((T, H), s, B16), r=randn((T, H), s + 2),
                          g=torch.ones(H, dtype=B16, device="cuda"), d_in=new((T, H)), d_g=new((H,)),
                          ws2=new((norm.workspace_bytes(),), torch.uint8)))
    torch.cuda.synchronize()
    for _ in range(10):
        for st, stream in zip(state, streams):
            plan.run(st["ids"], *st["out"], st["ws"], stream)
            norm.run(st["d"], None, st["r"], st["g"], 1e-6, st["d_in"], st["d_g"], st["ws2"], stream=stream.cuda_stream)
    torch.cuda.synchronize()
    for st in state:
        flat = st["ids"].view(-1).long()
        order = torch.argsort(flat, stable=True)
        assert torch.equal(st["out"][1].long(), order)
        assert torch.equal(st["out"][0].view(-1).long()[order], torch.arange(T * k, device="cuda"))
        want = (st["d"].double() * st["r"].double() * torch.rsqrt((st["r"].double() ** 2).mean(1, keepdim=True) + 1e-6)).sum(0)
        size = (st["d"].double() * st["r"].double() * torch.rsqrt((st["r"].double() ** 2).mean(1, keepdim=True) + 1e-6)).abs().sum(0)
        assert ((st["d_g"].double() - want).abs() <= (T / 152 + 200) * ref.U * size).all()
    assert plan.get_status() == norm.get_status() == 0


def test_parameters_and_slices_are_taken():
    """A gamma that is a Parameter, and rows of a larger buffer."""
    T, H = 6, 128
    big_x, big_r = randn((T + 4, H), 1, B16), randn((T + 4, H), 2)
    gamma = torch.nn.Parameter((1 + 0.1 * randn((H,), 3)).to(B16))
    plan = mfr.ResidualNormPlan(T, H, quant=mfr.QUANT_NONE)
    out = [new((T, H)), new((T, H), B16)]
    plan.run(big_x[2:2 + T], big_r[3:3 + T], out[0], gamma, 1e-6, out[1])
    again = [new((T, H)), new((T, H), B16)]
    plan.run(big_x[2:2 + T].clone(), big_r[3:3 + T].clone(), again[0], gamma.detach().clone(), 1e-6, again[1])
    torch.cuda.synchronize()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1]) and out[1].any()


CAPTURE_FIRST = r"""
import torch
import moe_finalize_residual_rmsnorm_gb300 as mfr
T, H, k, E = 50, {H}, {k}, 16
I32, F32, B16 = torch.int32, torch.float32, torch.bfloat16
def new(shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype, device="cuda")
g = torch.Generator(device="cuda").manual_seed(1)
ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=I32)
x, r = torch.randn((T, H), generator=g, device="cuda").to(B16), torch.randn((T, H), generator=g, device="cuda")
gamma, w = torch.ones(H, dtype=B16, device="cuda"), torch.rand((T, k), generator=g, device="cuda")
route, norm, back = mfr.RoutePlan(T, k, E), mfr.ResidualNormPlan(T, H, quant=mfr.QUANT_TOKEN), mfr.ResidualNormGradPlan(T, H)
disp, grad = mfr.DispatchPlan(T, H, k), mfr.FinalizeGradPlan(T, H, k)
b = dict(row=new((T, k), I32), slot=new((T * k,), I32), off=new((E + 1,), I32), cnt=new((E,), I32), r=new((T, H)),
         y=new((T, H), B16), q=new((T, H), torch.float8_e4m3fn), sf=new((T, 1)), rows=new((T * k, H), B16),
         dE=new((T * k, H), B16), dw=new((T, k)), dx=new((T, H), B16), dr=new((T, H)), dg=new((H,)))
ws = new((back.workspace_bytes(),), torch.uint8)
def calls():
    norm.run(x, r, b["r"], gamma, 1e-6, b["y"], b["q"], b["sf"])
    route.run(ids, b["row"], b["slot"], b["off"], b["cnt"])
    disp.run(b["y"], b["row"], b["slot"], b["rows"])
    grad.run(x, b["rows"], b["row"], b["slot"], w, b["dE"], b["dw"])
    disp.run_grad(b["dE"], b["row"], b["dx"])
    back.run(b["dx"], r, b["r"], gamma, 1e-6, b["dr"], b["dg"], ws)
torch.cuda.synchronize()
graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
    calls()
graph.replay()
torch.cuda.synchronize()
first = dict((n, t.clone()) for n, t in b.items())
calls()
torch.cuda.synchronize()
for n, t in b.items():
    assert torch.equal(first[n].view(torch.uint8), t.view(torch.uint8)), n
    assert t.view(torch.uint8).any(), n
print("captured first")
"""


@pytest.mark.parametrize("H,k", [(64, 2), (1024, 5), (4096, 8), (9000, 12)])
def test_the_first_calls_of_a_process_may_be_captured(H, k):
    """Plans load their kernels: in a new process nothing runs before the capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST.format(H=H, k=k)], cwd=root, capture_output=True, text=True,
                       timeout=240)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]
