"""RMSNorm of query and key heads with the rotation, and its gradient, on the
GPU against their plain 64-bit forms."""
import ctypes

import pytest
import torch

import moe_finalize_residual_rmsnorm_gb300 as mfr
import step_ref as ref
from test_layer_ops_gpu import B16, F32, I32, Guarded, randn

pytestmark = pytest.mark.gpu
F16 = torch.float16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


def table(most, rotary):
    a = torch.arange(most, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) / max(1, rotary))
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float().cuda()


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class Case:
    def __init__(self, T, hq, hk, D, rotary, interleaved=False, dtype=B16, most=100, packed=False, seed=0):
        self.shape, self.rotary, self.interleaved, self.dtype, self.most = (T, hq, hk, D), rotary, interleaved, dtype, most
        if packed:
            qkv = randn((T, hq + 2 * hk, D), seed, dtype, 2.0)
            self.q, self.k = qkv[:, :hq], qkv[:, hq:hq + hk]
            d = randn((T, hq + 2 * hk, D), seed + 1, dtype)
            self.d_q_out, self.d_k_out = d[:, hk:hk + hq], d[:, hk + hq:]
        else:
            self.q, self.k = randn((T, hq, D), seed, dtype, 2.0), randn((T, hk, D), seed + 2, dtype, 0.5)
            self.d_q_out, self.d_k_out = randn((T, hq, D), seed + 3, dtype), randn((T, hk, D), seed + 4, dtype)
        self.gq, self.gk = (1 + 0.3 * randn((D,), seed + 5, F32)).to(dtype), randn((D,), seed + 6, F32).to(dtype)
        self.table = table(most, rotary)
        self.pos = torch.randint(0, most, (T,), generator=torch.Generator().manual_seed(seed)).to(I32).cuda()

    def plan(self, **kw):
        T, hq, hk, D = self.shape
        return mfr.QkNormRopePlan(T, hq, hk, D, rotary_dim=self.rotary, interleaved=self.interleaved, dtype=self.dtype,
                                  max_positions=self.most, **kw)

    def run(self, plan, q_out, k_out, stream=None):
        plan.run(self.q, self.k, self.gq, self.gk, EPS, self.table, self.pos, q_out, k_out, stream)

    def run_grad(self, plan, d_q, d_k, d_gq, d_gk, ws, stream=None):
        plan.run_grad(self.d_q_out, self.d_k_out, self.q, self.k, self.gq, self.gk, EPS, self.table, self.pos, d_q, d_k, d_gq,
                      d_gk, ws, stream)

    def rounded(self, want, tol):
        return tol + ref.HALF_STEP[self.dtype] * (want.abs() + tol) + (2.0 ** -25 if self.dtype is F16 else ref.TINY)

    def want(self):
        out = []
        for x, g in ((self.q, self.gq), (self.k, self.gk)):
            w, tol = ref.qk_norm(x, g, EPS, self.table, self.pos, self.rotary, self.interleaved)
            out.append((w, self.rounded(w, tol)))
        return out

    def check(self, q_out, k_out, tokens=slice(None)):
        for name, got, (w, tol) in zip(("q", "k"), (q_out, k_out), self.want()):
            ref.assert_within(got[tokens], w[tokens], tol[tokens], name)

    def check_grad(self, d_q, d_k, d_gq, d_gk):
        for name, x, g, d, got, got_g in (("q", self.q, self.gq, self.d_q_out, d_q, d_gq), ("k", self.k, self.gk, self.d_k_out, d_k, d_gk)):
            w, tol, wg, tg = ref.qk_norm_grad(d, x, g, EPS, self.table, self.pos, self.rotary, self.interleaved)
            ref.assert_within(got, w, self.rounded(w, tol), "d_" + name)
            ref.assert_within(got_g, wg, tg + ref.TINY, "d_gamma_" + name)


SHAPES = [  # T, heads_q, heads_k, D, rotary
    (1, 1, 1, 8, 0), (1, 32, 8, 128, 128), (3, 5, 1, 16, 16), (2, 7, 3, 24, 16), (5, 3, 2, 72, 64), (9, 24, 4, 80, 32),
    (4, 8, 8, 96, 96), (17, 6, 2, 64, 64), (33, 4, 4, 128, 64), (5, 2, 1, 192, 192), (6, 3, 3, 200, 160), (3, 2, 2, 256, 256),
    (2, 3, 1, 512, 512), (2, 2, 1, 504, 32), (500, 4, 1, 128, 128), (4099, 1, 1, 64, 32), (7, 100, 9, 40, 32)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [B16, F16])
@pytest.mark.parametrize("T,hq,hk,D,rotary", SHAPES)
def test_forward(T, hq, hk, D, rotary, dtype, interleaved):
    c = Case(T, hq, hk, D, rotary, interleaved, dtype, packed=D % 16 == 0)
    plan, a, b = c.plan(), Guarded((T, hq, D), dtype), Guarded((T, hk, D), dtype)
    c.run(plan, a.t, b.t)
    torch.cuda.synchronize()
    assert plan.get_status() == 0
    c.check(a.check(), b.check())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [B16, F16])
@pytest.mark.parametrize("T,hq,hk,D,rotary", SHAPES)
def test_gradient(T, hq, hk, D, rotary, dtype, interleaved):
    c = Case(T, hq, hk, D, rotary, interleaved, dtype, packed=D % 16 == 0)
    plan = c.plan()
    outs = Guarded((T, hq, D), dtype), Guarded((T, hk, D), dtype), Guarded((D,), F32), Guarded((D,), F32)
    ws = Guarded((plan.workspace_bytes(),), torch.uint8, fill=0xFF)
    first = None
    for _ in range(2):
        c.run_grad(plan, *[o.t for o in outs], ws.t)
        torch.cuda.synchronize()
        assert plan.get_status() == 0
        ws.check()
        got = [o.check().clone() for o in outs]
        c.check_grad(*got)
        assert first is None or all(torch.equal(x, y) for x, y in zip(first, got))       # the same bits
        first = got


@pytest.mark.parametrize("T", [1, 3, 50])
def test_in_place_in_a_packed_tensor(T):
    c = Case(T, 6, 2, 64, 64, packed=True)
    want = c.want()
    before = c.q._base.clone() if c.q._base is not None else None
    c.run(c.plan(), c.q, c.k)
    torch.cuda.synchronize()
    for got, (w, tol) in zip((c.q, c.k), want):
        ref.assert_within(got, w, tol, "in place")
    assert torch.equal(c.q._base[:, 8:], before[:, 8:])           # the values are not touched
    # and the gradient onto d_q_out, d_k_out
    c = Case(T, 6, 2, 64, 64, packed=True, seed=9)
    plan = c.plan()
    d = [t.clone() for t in (c.d_q_out, c.d_k_out)]
    ws, gs = torch.zeros(plan.workspace_bytes(), dtype=torch.uint8, device="cuda"), [torch.zeros(64, device="cuda") for _ in range(2)]
    c.run_grad(plan, c.d_q_out, c.d_k_out, *gs, ws)
    torch.cuda.synchronize()
    got = c.d_q_out.clone(), c.d_k_out.clone()
    c.d_q_out, c.d_k_out = d
    c.check_grad(*got, *gs)


def test_heads_outside_tokens():
    """[heads, T, D] in memory, and tokens with a gap between."""
    T, hq, hk, D = 20, 4, 2, 64
    c = Case(T, hq, hk, D, 32)
    c.q = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.zeros((hq, T, D), dtype=B16, device="cuda").transpose(0, 1)
    wide = torch.full((T, 3 * hk, D + 8), 7.0, dtype=B16, device="cuda")
    k_out = wide[:, ::3, :D]
    c.run(c.plan(), out, k_out)
    torch.cuda.synchronize()
    c.check(out, k_out)
    assert (wide[:, 1::3] == 7).all() and (wide[:, :, D:] == 7).all()


def test_positions_out_of_range_leave_their_tokens_alone():
    c = Case(40, 5, 3, 64, 64, most=50)
    bad = [0, 7, 8, 39]
    c.pos[bad] = torch.tensor([-1, 50, 2 ** 31 - 1, -2 ** 31], dtype=I32, device="cuda")
    plan, a, b = c.plan(), Guarded((40, 5, 64), B16), Guarded((40, 3, 64), B16)
    before = a.t.clone(), b.t.clone()
    c.run(plan, a.t, b.t)
    assert plan.get_status() == mfr.STATUS_BAD_INDEX
    assert torch.equal(a.check()[bad], before[0][bad]) and torch.equal(b.check()[bad], before[1][bad])
    good = [t for t in range(40) if t not in bad]
    d = [torch.full((40, h, 64), 3.0, dtype=B16, device="cuda") for h in (5, 3)]
    g = [torch.zeros(64, device="cuda") for _ in range(2)]
    c.run_grad(plan, *d, *g, torch.zeros(plan.workspace_bytes(), dtype=torch.uint8, device="cuda"))
    assert plan.get_status() == mfr.STATUS_BAD_INDEX
    assert (d[0][bad] == 3).all() and (d[1][bad] == 3).all()
    # the others are as if those were not there
    for name in ("q", "k", "d_q_out", "d_k_out", "pos"):
        setattr(c, name, getattr(c, name)[good])
    c.check(a.t[good], b.t[good])
    c.check_grad(d[0][good], d[1][good], *g)
    with pytest.raises(mfr.MFRError):
        c2 = Case(2, 1, 1, 16, 16)
        c2.pos[0] = 100
        c2.run(c2.plan(debug_checks=True), torch.zeros_like(c2.q), torch.zeros_like(c2.k))


def test_zeros_nan_and_infinity_stay_in_their_heads():
    c = Case(6, 4, 2, 128, 64)
    c.q[1, 2] = 0
    c.q[2, 1, 5] = float("nan")
    c.q[3, 3, 100] = float("inf")
    plan, a, b = c.plan(), torch.zeros_like(c.q), torch.zeros_like(c.k)
    c.run(plan, a, b)
    torch.cuda.synchronize()
    (w, tol), _ = c.want()
    keep = torch.ones((6, 4), dtype=torch.bool)
    keep[2, 1] = keep[3, 3] = False
    ref.assert_within(a[keep.cuda()], w[keep], tol[keep], "q")
    assert (a[1, 2] == 0).all() and a[2, 1].isnan().all() and a[3, 3].isnan().any()


def test_gradient_against_differences():
    """The formula's forward in 64 bits at x + h dx, gamma + h dgamma."""
    c = Case(5, 3, 2, 48, 32, interleaved=True, dtype=F16)
    plan = c.plan()
    d = [torch.zeros_like(c.q), torch.zeros_like(c.k), torch.zeros(48, device="cuda"), torch.zeros(48, device="cuda")]
    c.run_grad(plan, *d, torch.zeros(plan.workspace_bytes(), dtype=torch.uint8, device="cuda"))
    for x, g, do, dx, dg in ((c.q, c.gq, c.d_q_out, d[0], d[2]), (c.k, c.gk, c.d_k_out, d[1], d[3])):
        for seed in range(3):
            gen = torch.Generator().manual_seed(seed)
            vx, vg = torch.randn(x.shape, generator=gen, dtype=ref.D), torch.randn(48, generator=gen, dtype=ref.D)

            def loss(h):
                return (ref.f64(do) * ref.qk_norm((ref.f64(x) + h * vx), ref.f64(g) + h * vg, EPS, c.table, c.pos, 32, True)[0]).sum()
            diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
            along = (ref.f64(dx) * vx).sum() + (ref.f64(dg) * vg).sum()
            # every element of dx is off by half a step of fp16 at most
            tol = 2.0 ** -11 * (ref.f64(dx) * vx).abs().sum() + 2.0 ** -25 * vx.abs().sum() + 1e-5 * (ref.f64(dg) * vg).abs().sum()
            assert abs(diff - along) < tol + 1e-6 * abs(diff)


@pytest.mark.parametrize("pdl", [True, False])
def test_captured_replayed_and_on_two_streams(pdl):
    c, other = Case(30, 8, 2, 128, 128), Case(30, 8, 2, 128, 128, seed=70)
    plan = c.plan(enable_pdl=pdl)
    bufs = [[torch.zeros_like(c.q), torch.zeros_like(c.k), torch.zeros_like(c.q), torch.zeros_like(c.k),
             torch.zeros(128, device="cuda"), torch.zeros(128, device="cuda")] for _ in range(2)]
    ws = [torch.zeros(plan.workspace_bytes(), dtype=torch.uint8, device="cuda") for _ in range(2)]
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        c.run(plan, *bufs[0][:2])
        c.run_grad(plan, *bufs[0][2:], ws[0])
    for seed in (0, 40):
        src = Case(30, 8, 2, 128, 128, seed=seed)
        for n in ("q", "k", "d_q_out", "d_k_out", "gq", "gk", "pos"):
            getattr(c, n).copy_(getattr(src, n))
        g.replay()
        with torch.cuda.stream(s):
            other.run(plan, *bufs[1][:2])
            other.run_grad(plan, *bufs[1][2:], ws[1])
        torch.cuda.synchronize()
        for case, b in ((c, bufs[0]), (other, bufs[1])):
            case.check(*b[:2])
            case.check_grad(*b[2:])
    assert plan.get_status() == 0


def test_zero_tokens():
    c = Case(0, 2, 1, 64, 64)
    plan = c.plan()
    c.run(plan, torch.zeros_like(c.q), torch.zeros_like(c.k))
    g = [torch.full((64,), 5.0, device="cuda") for _ in range(2)]
    c.run_grad(plan, torch.zeros_like(c.q), torch.zeros_like(c.k), *g, None)
    torch.cuda.synchronize()
    assert (g[0] == 0).all() and (g[1] == 0).all() and plan.get_status() == 0


def test_refusals():
    T, hq, hk, D = 4, 4, 2, 64
    c = Case(T, hq, hk, D, 64)
    plan, lib = c.plan(), mfr.load_library()
    big = torch.zeros(4096, dtype=B16, device="cuda")

    def heads(t, token=None, head=None, at=0):
        return ctypes.byref(_Heads(t.data_ptr() + at, t.stride(0) if token is None else token, t.stride(1) if head is None else head))

    def call(**kw):
        a = dict(q=heads(c.q), k=heads(c.k), gq=c.gq.data_ptr(), gk=c.gk.data_ptr(), eps=EPS, table=c.table.data_ptr(),
                 pos=c.pos.data_ptr(), qo=heads(qo), ko=heads(ko))
        a.update(kw)
        return lib.moe_qk_norm_rope_run(plan._h, *a.values(), torch.cuda.current_stream().cuda_stream)
    qo, ko = torch.zeros_like(c.q), torch.zeros_like(c.k)
    assert call() == 0
    for name in ("q", "k", "gq", "gk", "table", "pos", "qo", "ko"):
        assert call(**{name: None}) == 1, name
    for name, t in (("q", c.q), ("qo", qo)):
        assert call(**{name: heads(t, at=2)}) == 3 and call(**{name: heads(t, head=60)}) == 3
        assert call(**{name: heads(t, token=-256)}) == 1
    for name in ("gq", "gk", "table"):
        assert call(**{name: big.data_ptr() + 2}) == 3, name
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(qo=heads(qo, head=32)) == 1 and call(qo=heads(qo, token=0)) == 1       # its heads overlap
    assert call(ko=heads(qo, at=0)) == 1                              # q_out and k_out share bytes
    assert call(ko=heads(c.q, token=hq * D)) == 1                     # k_out lies in q
    assert call(qo=heads(c.q)) == 0                                   # in place
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="lie together"):
        plan.run(c.q.transpose(1, 2).contiguous().transpose(1, 2), c.k, c.gq, c.gk, EPS, c.table, c.pos, qo, ko)
    # tokens that span more than there are addresses
    large = mfr.QkNormRopePlan(1 << 26, hq, hk, D, max_positions=c.table.shape[0])
    far = heads(c.q, token=1 << 40)
    assert lib.moe_qk_norm_rope_run(large._h, far, far, c.gq.data_ptr(), c.gk.data_ptr(), EPS, c.table.data_ptr(), c.pos.data_ptr(),
                                    far, far, torch.cuda.current_stream().cuda_stream) == 1
