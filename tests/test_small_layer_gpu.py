"""The MoE layer for a few tokens on the GPU against its plain 64-bit form."""
import pytest
import torch

import layer_ref
import moe_finalize_residual_rmsnorm_gb300 as mfr
import step_ref as ref
from test_layer_ops_gpu import B16, F32, FP8, I32, Guarded, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


def inputs(T, H, I, E, k, fp8=False, seed=0, share=0.0, skew=0.0):
    """Tensors of one call by the names of MoeLayerPlan.run."""
    i = dict(expert_ids=torch.from_numpy(layer_ref.draw_ids(T, k, E, seed=seed, nonlocal_share=share, skew=skew)).cuda(),
             topk_weights=torch.softmax(randn((T, k), seed + 1, F32), 1))
    if not fp8:
        i.update(x=randn((T, H), seed + 2, B16), w13=randn((E, 2 * I, H), seed + 3, B16, H ** -0.5),
                 w2=randn((E, H, I), seed + 4, B16, I ** -0.5))
        return i
    hb, ib = -(-H // 128), I // 128
    g = torch.Generator().manual_seed(seed + 7)

    def codes(shape, s):
        return randn(shape, s, F32, 64.0).clamp(-448, 448).to(FP8)

    def scales(shape, typical):
        return ((0.5 + torch.rand(shape, generator=g)) * (typical / 64)).cuda()
    i.update(x=codes((T, H), seed + 2), w13=codes((E, 2 * I, H), seed + 3), w2=codes((E, H, I), seed + 4),
             x_sf=scales((T, hb), 1.0), w13_sf=scales((E, 2 * ib, hb), H ** -0.5), w2_sf=scales((E, hb, ib), I ** -0.5))
    return i


def reference(i):
    return ref.moe_layer(i["x"], i["expert_ids"], i["topk_weights"], i["w13"], i["w2"], i.get("x_sf"), i.get("w13_sf"),
                         i.get("w2_sf"))


class Layer:
    def __init__(self, T, H, I, E, k, fp8=False, **kw):
        self.plan = mfr.MoeLayerPlan(T, H, I, E, k, dtype=FP8 if fp8 else B16, sentinel_skip=True, **kw)
        self.out = Guarded((T, H), B16)
        self.ws = Guarded((self.plan.workspace_bytes(),), torch.uint8, fill=0xFF)     # NaN, whatever is read before it is written

    def run(self, i, stream=None):
        self.plan.run(**i, out=self.out.t, workspace=self.ws.t, stream=stream)

    def check(self, i, what="out"):
        torch.cuda.synchronize()
        assert self.plan.get_status() == 0
        want, tol = reference(i)
        self.ws.check()
        ref.assert_within(self.out.check(), want, tol, what)


SHAPES = [  # T, H, I, E, k
    (1, 256, 128, 4, 2), (1, 64, 64, 1, 1), (1, 8, 8, 1, 1), (2, 16, 24, 3, 2), (1, 4096, 128, 8, 8), (3, 72, 1032, 5, 3),
    (8, 1024, 512, 32, 8), (16, 264, 200, 7, 4), (17, 520, 136, 9, 6), (33, 256, 264, 40, 5), (37, 2056, 712, 32, 6),
    (64, 512, 256, 8, 8), (65, 136, 72, 3, 2), (100, 384, 128, 2, 2), (128, 256, 128, 16, 8), (200, 264, 136, 1, 1),
    (512, 128, 64, 100, 8), (256, 64, 72, 1024, 16), (4096, 40, 8, 3, 1)]


@pytest.mark.parametrize("T,H,I,E,k", SHAPES)
def test_bf16(T, H, I, E, k):
    layer, i = Layer(T, H, I, E, k), inputs(T, H, I, E, k, seed=T)
    layer.run(i)
    layer.check(i)


@pytest.mark.parametrize("T,H,I,E,k", [
    (1, 128, 128, 1, 1), (1, 16, 128, 2, 1), (1, 4096, 128, 8, 8), (3, 144, 256, 5, 3), (8, 1024, 512, 32, 8),
    (16, 272, 384, 7, 4), (30, 2064, 256, 9, 6), (64, 512, 256, 8, 8), (100, 384, 128, 2, 2), (128, 256, 128, 16, 8),
    (200, 272, 128, 1, 1), (512, 128, 128, 100, 8)])
def test_e4m3(T, H, I, E, k):
    layer, i = Layer(T, H, I, E, k, fp8=True), inputs(T, H, I, E, k, fp8=True, seed=T)
    layer.run(i)
    layer.check(i)


# few units of many steps along K: of the first product, of the second, of both; 16 to 128 columns
LONG = [(1, 4104, 64, 1, 1), (5, 3088, 72, 2, 1), (3, 264, 2056, 2, 2), (20, 1808, 1000, 1, 1), (60, 2048, 704, 1, 1), (9, 1552, 136, 12, 1),
        (120, 2048, 704, 1, 1), (300, 2608, 704, 2, 1)]
LONG8 = [(1, 4112, 128, 1, 1), (5, 3088, 256, 2, 1), (3, 272, 2048, 2, 2), (20, 2064, 1536, 1, 1), (60, 1552, 1536, 1, 1),
         (120, 2048, 1408, 1, 1), (300, 2608, 1408, 2, 1)]


@pytest.mark.parametrize("T,H,I,E,k,fp8", [(*c, False) for c in LONG] + [(*c, True) for c in LONG8])
def test_units_divided_along_k(T, H, I, E, k, fp8):
    layer, i = Layer(T, H, I, E, k, fp8), inputs(T, H, I, E, k, fp8, seed=T)
    layer.run(i)
    layer.check(i)
    first = layer.out.t.clone()
    layer.plan.set_wait_limit(0)                      # each of a unit's CTAs gives up
    layer.run(i)
    torch.cuda.synchronize()
    assert layer.plan.get_status() & mfr.STATUS_TIMEOUT
    layer.plan.set_wait_limit(4_000_000_000)
    for _ in range(20):
        layer.run(i)
    torch.cuda.synchronize()
    assert layer.plan.get_status() == 0 and torch.equal(layer.out.t, first)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,E,k,share,skew", [(40, 16, 8, 0.4, 1.5), (5, 4, 2, 0.9, 0.0), (128, 4, 3, 0.2, 2.0)])
def test_experts_elsewhere_and_popular_ones(T, E, k, share, skew, fp8):
    layer = Layer(T, 272, 256, E, k, fp8)
    i = inputs(T, 272, 256, E, k, fp8, seed=3, share=share, skew=skew)
    layer.run(i)
    layer.check(i)


@pytest.mark.parametrize("fp8", [False, True])
def test_no_pair_has_an_expert_here(fp8):
    layer, i = Layer(9, 528, 128, 4, 2, fp8), inputs(9, 528, 128, 4, 2, fp8)
    i["expert_ids"].fill_(-1)
    layer.run(i)
    torch.cuda.synchronize()
    assert layer.plan.get_status() == 0
    assert (layer.out.check() == 0).all()
    i["expert_ids"][3, 1] = 2                   # and the plan's next call has one
    layer.run(i)
    layer.check(i)


@pytest.mark.parametrize("T,k", [(3, 4), (70, 8)])
def test_the_same_expert_for_every_slot(T, k):
    """More pairs of an expert than tokens: several chunks of one expert."""
    layer, i = Layer(T, 136, 72, 9, k), inputs(T, 136, 72, 9, k)
    i["expert_ids"].fill_(8)
    layer.run(i)
    layer.check(i)


def test_ids_out_of_range_add_nothing_and_are_reported():
    layer, i = Layer(6, 64, 64, 4, 2), inputs(6, 64, 64, 4, 2)
    i["expert_ids"][2, 0] = 4
    i["expert_ids"][5, 1] = 2 ** 31 - 1
    layer.run(i)
    assert layer.plan.get_status() == mfr.STATUS_BAD_INDEX
    layer.check(i)
    strict = mfr.MoeLayerPlan(6, 64, 64, 4, 2)                  # without sentinel_skip a negative id is one too
    i["expert_ids"][:] = 0
    i["expert_ids"][0, 0] = -1
    strict.run(**i, out=layer.out.t, workspace=layer.ws.t)
    assert strict.get_status() == mfr.STATUS_BAD_INDEX
    layer.check(i)
    with pytest.raises(mfr.MFRError) as e:
        mfr.MoeLayerPlan(6, 64, 64, 4, 2, debug_checks=True).run(**i, out=layer.out.t, workspace=layer.ws.t)
    assert e.value.code == 7


@pytest.mark.parametrize("fp8", [False, True])
def test_a_token_of_nan_and_infinities_leaves_the_others_alone(fp8):
    T, H, I, E, k = 20, 256, 128, 3, 2
    layer, i = Layer(T, H, I, E, k, fp8), inputs(T, H, I, E, k, fp8)
    layer.run(i)
    torch.cuda.synchronize()
    want = layer.out.t.clone()
    if fp8:
        i["x_sf"][7, 1] = float("nan")
        i["x_sf"][11, 0] = float("inf")
    else:
        i["x"][7, 5] = float("nan")
        i["x"][11, 0] = float("inf")
    layer.run(i)
    torch.cuda.synchronize()
    rest = [t for t in range(T) if t not in (7, 11)]
    assert torch.equal(layer.out.t[rest], want[rest])
    assert layer.out.t[7].isnan().all()
    assert not layer.out.t[11].isfinite().all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 8, 8), (37, 16, 4), (130, 3, 2)])
def test_repeats_bit_for_bit_and_with_fewer_tokens_beside(T, E, k, fp8):
    """The same bits in every call, whatever the workspace held."""
    H, I = 1040, 384
    layer, i = Layer(T, H, I, E, k, fp8), inputs(T, H, I, E, k, fp8)
    layer.run(i)
    torch.cuda.synchronize()
    want = layer.out.check().clone()
    for fill in (0, 0x7F, 0xFF):
        layer.ws.t.fill_(fill)
        layer.out.t.view(torch.uint8).fill_(0x33)
        layer.run(i)
        torch.cuda.synchronize()
        assert torch.equal(layer.out.check(), want)


def test_zero_tokens():
    plan = mfr.MoeLayerPlan(0, 64, 64, 4, 2)
    z = lambda *s: torch.zeros(s, dtype=B16, device="cuda")  # noqa: E731
    plan.run(z(0, 64), z(0, 2).to(I32), z(0, 2).to(F32), z(4, 128, 64), z(4, 64, 64), z(0, 64), None)
    assert plan.get_status() == 0 and plan.workspace_bytes() == 0


@pytest.mark.parametrize("pdl", [True, False])
def test_captured_replayed_and_on_another_stream(pdl):
    T, H, I, E, k = 12, 512, 264, 16, 4
    layer = Layer(T, H, I, E, k, enable_pdl=pdl)
    a, b = inputs(T, H, I, E, k, seed=1), inputs(T, H, I, E, k, seed=50)
    i = {n: t.clone() for n, t in a.items()}
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        layer.run(i)
        layer.run(i)
    for src in (a, b, a):
        for n in i:
            i[n].copy_(src[n])
        g.replay()
        layer.check(src)
    with torch.cuda.stream(s):
        layer.run(b)
    s.synchronize()
    layer.check(b)
    layer.run(a, stream=torch.cuda.current_stream())
    layer.check(a)


@pytest.mark.parametrize("pdl", [True, False])
@pytest.mark.parametrize("T,H,I,E,k,fp8", [(5, 3088, 72, 2, 1, False), (3, 264, 2056, 2, 2, False), (20, 2064, 1536, 1, 1, True)])
def test_divided_units_captured_and_beside_others(T, H, I, E, k, fp8, pdl):
    layer, other = Layer(T, H, I, E, k, fp8, enable_pdl=pdl), Layer(16, 1024, 512, 16, 4)
    i, j = inputs(T, H, I, E, k, fp8, seed=1), inputs(16, 1024, 512, 16, 4, seed=2)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        for _ in range(5):
            layer.run(i)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s):
            g.replay()
        other.run(j)
    other.check(j)
    layer.check(i)


@pytest.mark.parametrize("pdl", [True, False])
@pytest.mark.parametrize("share", [0.0, 0.5])
def test_many_pairs_an_expert_captured_with_other_tokens_each_time(share, pdl):
    T, H, I, E, k = 150, 1032, 136, 4, 2
    layer = Layer(T, H, I, E, k, enable_pdl=pdl)
    a, b = inputs(T, H, I, E, k, seed=1, share=share), inputs(T, H, I, E, k, seed=9, skew=1.5)
    i = {n: t.clone() for n, t in a.items()}
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        layer.run(i)
        layer.run(i)
    for src in (a, b, a):
        for n in i:
            i[n].copy_(src[n])
        g.replay()
        layer.check(src)


def test_two_plans_at_once():
    """Calls on two streams, each with its own workspace, sharing the SMs and tensor memory."""
    shapes = [(16, 1024, 512, 16, 4), (100, 512, 256, 8, 8)]
    layers = [Layer(*s) for s in shapes]
    ins = [inputs(*s, seed=n) for n, s in enumerate(shapes)]
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    for _ in range(10):
        for layer, i, s in zip(layers, ins, streams):
            layer.run(i, stream=s)
    for layer, i in zip(layers, ins):
        layer.check(i)


def test_layer_then_residual_norm():
    """As a decode step runs them: the layer's output added to the residual stream."""
    T, H, I, E, k = 8, 1024, 256, 16, 4
    layer, i = Layer(T, H, I, E, k), inputs(T, H, I, E, k)
    res, gamma = randn((T, H), 30, F32), (1 + 0.2 * randn((H,), 31, F32)).to(B16)
    norm = mfr.ResidualNormPlan(T, H, quant=mfr.QUANT_NONE)
    r, z = torch.zeros((T, H), device="cuda"), torch.zeros((T, H), dtype=B16, device="cuda")
    for _ in range(3):
        layer.run(i)
        norm.run(layer.out.t, res, r, gamma, 1e-6, z)
    layer.check(i)
    assert torch.equal(r, res + layer.out.t.float())


def test_the_c_side_refuses():
    lib = mfr.load_library()
    plan, i = mfr.MoeLayerPlan(4, 64, 64, 4, 2), inputs(4, 64, 64, 4, 2)
    ws = torch.zeros(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
    out = torch.zeros((4, 64), dtype=B16, device="cuda")

    def call(**kw):
        a = dict(x=i["x"].data_ptr(), x_sf=None, ids=i["expert_ids"].data_ptr(), w=i["topk_weights"].data_ptr(),
                 w13=i["w13"].data_ptr(), w13_sf=None, w2=i["w2"].data_ptr(), w2_sf=None, out=out.data_ptr(),
                 ws=ws.data_ptr(), n=ws.numel())
        a.update(kw)
        return lib.moe_small_layer_run(plan._h, *a.values(), torch.cuda.current_stream().cuda_stream)
    assert call() == 0
    for name in ("x", "ids", "w", "w13", "w2", "out", "ws"):
        assert call(**{name: None}) == 1, name
    for name in ("x", "w13", "w2", "out", "ws"):
        assert call(**{name: out.data_ptr() + 2}) == 3, name
    for name in ("ids", "w"):
        assert call(**{name: out.data_ptr() + 2}) == 3, name
    assert call(n=ws.numel() - 1) == 1
    assert call(x_sf=i["topk_weights"].data_ptr()) == 1
    assert call(out=i["x"].data_ptr()) == 1 and call(out=ws.data_ptr()) == 1 and call(ws=i["w2"].data_ptr()) == 1
    other = mfr.ResidualNormPlan(4, 64)
    assert lib.moe_small_layer_run(other._h, *[None] * 10, 0, None) == 1
    torch.cuda.synchronize()
    assert plan.get_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 128, 1, 1), (3, 4096, 256, 8, 4), (130, 1040, 384, 5, 3)])
def test_waits_that_run_out_end_and_report_it(T, H, I, E, k, fp8):
    """With a limit of nothing the first stage's wait gives up: the run ends, says so, and the
    plan's next run with the usual limit is as if nothing had been."""
    layer, i = Layer(T, H, I, E, k, fp8), inputs(T, H, I, E, k, fp8)
    layer.run(i)
    layer.check(i)
    want = layer.out.t.clone()
    for limit in (0, 100, 0, 3000):
        layer.plan.set_wait_limit(limit)
        layer.run(i)
        torch.cuda.synchronize()
        st = layer.plan.get_status()
        assert st == mfr.STATUS_TIMEOUT or (limit > 0 and st == 0 and torch.equal(layer.out.t, want))
        layer.ws.check()
        layer.out.check()
        layer.plan.set_wait_limit(4_000_000_000)
        layer.run(i)
        torch.cuda.synchronize()
        assert layer.plan.get_status() == 0 and torch.equal(layer.out.check(), want)
    with pytest.raises(mfr.MFRError):
        layer.plan.set_wait_limit(-1)
    with pytest.raises(mfr.MFRError):
        layer.plan.set_wait_limit(4_000_000_001)


def test_many_calls_without_a_wait_that_runs_out():
    for T, H, I, E, k in [(1, 2048, 1024, 8, 4), (130, 256, 128, 3, 2), (16, 520, 520, 32, 8)]:
        layer, i = Layer(T, H, I, E, k), inputs(T, H, I, E, k)
        for _ in range(50):
            layer.run(i)
        layer.check(i)
