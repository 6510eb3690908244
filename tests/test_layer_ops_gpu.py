"""The operators around the finalize on the GPU against their plain 64-bit
forms (layer_ref.py)."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import moe_finalize_residual_rmsnorm_gb300 as mfr

pytestmark = pytest.mark.gpu

I32, F32, B16, FP8 = torch.int32, torch.float32, torch.bfloat16, torch.float8_e4m3fn
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


class Guarded:
    """An output buffer between two guard bands of a known byte."""

    def __init__(self, shape, dtype, fill=0x5A):
        n = int(np.prod(shape)) * dtype.itemsize
        self.raw = torch.full((n + 2 * GUARD * 4,), fill, dtype=torch.uint8, device="cuda")
        self.n, self.fill = n, fill
        self.t = self.raw[GUARD * 4:GUARD * 4 + n].view(dtype).view(shape)

    def check(self):
        assert (self.raw[:GUARD * 4] == self.fill).all() and (self.raw[GUARD * 4 + self.n:] == self.fill).all()
        return self.t


def cuda(a, dtype):
    return torch.as_tensor(np.asarray(a)).to(dtype).cuda().contiguous()


def randn(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


# ---- route -------------------------------------------------------------------------------

def run_route(ids, E, align, **kw):
    T, k = ids.shape
    plan = mfr.RoutePlan(T, k, E, align=align, **kw)
    outs = [Guarded(s, I32) for s in ((T, k), (plan.R,), (E + 1,), (E,))]
    ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
    plan.run(cuda(ids, I32), *[o.t for o in outs], ws)
    torch.cuda.synchronize()
    return plan, [o.check().cpu().numpy() for o in outs]


def check_route(ids, E, align, got):
    want = ref.route(ids, E, align)
    for g, w, what in zip(got, want, ("permuted_row_of", "slot_of_row", "expert_offsets", "expert_counts")):
        assert np.array_equal(g, w), what


@pytest.mark.parametrize("T,k,E,align", [
    (1, 1, 1, 1), (1, 8, 128, 1), (1, 16, 1024, 128), (2, 8, 8, 4), (5, 3, 7, 16), (16, 8, 128, 1), (17, 6, 33, 3),
    (128, 8, 256, 128), (333, 8, 31, 1), (1025, 8, 512, 16), (4097, 2, 1000, 1), (4000, 16, 64, 4096), (20000, 8, 256, 128)])
@pytest.mark.parametrize("share", [0.0, 0.3])
def test_route(T, k, E, align, share):
    ids = ref.draw_ids(T, k, E, seed=T + E, nonlocal_share=share, skew=1.2)
    plan, got = run_route(ids, E, align, sentinel_skip=True)
    check_route(ids, E, align, got)
    assert plan.get_status() == 0


@pytest.mark.parametrize("cluster", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("T,k,E", [(1, 1, 5), (100, 8, 128), (2000, 8, 100), (60, 16, 1024)])
def test_route_gives_the_same_for_every_cluster(cluster, T, k, E):
    ids = ref.draw_ids(T, k, E, seed=7, skew=0.5)
    plan, got = run_route(ids, E, 8, cluster_size=cluster)
    check_route(ids, E, 8, got)
    assert plan.get_status() == 0


@pytest.mark.parametrize("T,k,E,align,kw", [(32769, 8, 64, 1, {}), (40000, 8, 1024, 128, {}), (70001, 5, 3, 1, {}),
                                            (17000, 1, 16, 16, dict(cluster_size=1)), (32768, 8, 256, 128, {}),
                                            # several rounds a CTA: from 4096 pairs an SM up
                                            (90001, 7, 130, 16, {}), (262147, 8, 1023, 128, {}), (2000003, 1, 2, 1, {})])
def test_route_large(T, k, E, align, kw):
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, E, size=(T, k)).astype(np.int32)
    plan, got = run_route(ids, E, align, sentinel_skip=True, **kw)
    assert plan.workspace_bytes() > 0
    # the reference by a stable argsort: one pair at a time takes too long here
    flat = ids.reshape(-1)
    counts = np.bincount(flat[flat >= 0], minlength=E)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")[:counts.sum()]
    first = np.cumsum(counts) - counts
    row = offsets[flat[order]] + np.arange(counts.sum()) - first[flat[order]]
    row_of, slot_of = np.full(T * k, -1), np.where(np.arange(plan.R) < offsets[E], -1, -2)
    row_of[order], slot_of[row] = row, order
    for g, w in zip(got, (row_of.reshape(T, k), slot_of, offsets, counts)):
        assert np.array_equal(g, w)
    assert plan.get_status() == 0


def test_route_takes_repeats_and_one_expert_for_all():
    ids = np.zeros((300, 8), dtype=np.int32)
    plan, got = run_route(ids, 4, 1)
    check_route(ids, 4, 1, got)
    ids[:, ::2] = 3
    plan, got = run_route(ids, 4, 128)
    check_route(ids, 4, 128, got)


@pytest.mark.parametrize("sentinel,low,high,status", [(True, -1, 16, mfr.STATUS_BAD_INDEX), (True, -5, 3, 0),
                                                      (False, -1, 3, mfr.STATUS_BAD_INDEX), (True, 3, 2 ** 31 - 1, mfr.STATUS_BAD_INDEX),
                                                      (False, -2 ** 31, 2, mfr.STATUS_BAD_INDEX)])
def test_route_marks_ids_out_of_range(sentinel, low, high, status):
    ids = ref.draw_ids(20, 8, 16, seed=5)
    ids[3, 2], ids[19, 7] = low, high
    plan, got = run_route(ids, 16, 4, sentinel_skip=sentinel)
    check_route(ids, 16, 4, got)
    assert plan.get_status() == status
    assert plan.get_status() == 0


def test_route_without_pairs():
    plan, got = run_route(np.zeros((0, 8), dtype=np.int32), 16, 128)
    assert plan.R == 0 and not got[2].any() and not got[3].any()
    plan, got = run_route(np.full((3, 8), -1, dtype=np.int32), 16, 128, sentinel_skip=True)
    check_route(np.full((3, 8), -1), 16, 128, got)


# ---- maps for the row operators ---------------------------------------------------------

class Maps:
    def __init__(self, T, k, E, align=1, share=0.0, seed=0):
        self.ids = ref.draw_ids(T, k, E, seed=seed + T, nonlocal_share=share, skew=0.7)
        self.row_of, self.slot_of, self.offsets, _ = ref.route(self.ids, E, align)
        self.R = len(self.slot_of)
        self.upload()

    def upload(self):
        self.d_row, self.d_slot = cuda(self.row_of, I32), cuda(self.slot_of, I32)


# every form by slots (to 2, 4, 6, 8, 16) and by columns, few tokens of wide rows
# (a cluster a token) and plenty of tokens
ROWS = [(1, 8, 1), (1, 4096, 8), (3, 24, 16), (7, 136, 6), (33, 2056, 3), (130, 4096, 8), (20, 8192, 8), (9, 16384, 2),
        (600, 1032, 5), (2, 8200, 9), (30, 5000, 16), (1, 16384, 13), (2000, 264, 1), (2100, 1032, 8), (1900, 136, 4)]


@pytest.mark.parametrize("T,H,k", ROWS)
@pytest.mark.parametrize("align,share", [(1, 0.0), (4, 0.25), (32, 0.0)])
@pytest.mark.parametrize("dtype,sf", [(B16, 0), (F32, 0), (FP8, 4), (FP8, 5)])
def test_dispatch(T, H, k, align, share, dtype, sf):
    if H * dtype.itemsize % 16:
        pytest.skip("rows are multiples of 16 bytes")
    m = Maps(T, k, max(16, k), align, share)
    x = randn((T, H), T, F32).to(dtype)
    plan = mfr.DispatchPlan(T, H, k, m.R, dtype=dtype, sf_bytes=sf * 3, sentinel_skip=True)
    out = Guarded((m.R, H), dtype)
    scales = torch.randint(0, 256, (T, sf * 3), dtype=torch.uint8, device="cuda") if sf else None
    sf_out = Guarded((m.R, sf * 3), torch.uint8) if sf else None
    plan.run(x, m.d_row, m.d_slot, out.t, scales, sf_out.t if sf else None)
    torch.cuda.synchronize()
    for o, src in ((out, x), (sf_out, scales)):
        if o is None:
            continue
        got = o.check().view(torch.uint8).cpu().numpy().reshape(m.R, -1)
        src = src.view(torch.uint8).cpu().numpy().reshape(T, -1)
        want = np.full_like(got, 0x5A)                     # unused rows are left as they were
        want[m.slot_of == -1] = 0
        here = m.slot_of >= 0
        want[here] = src[m.slot_of[here] // k]
        assert np.array_equal(got, want)
    assert plan.get_status() == 0


@pytest.mark.parametrize("dtype", [torch.int8, torch.bool, torch.float16, torch.int32])
def test_dispatch_copies_any_type(dtype):
    T, H, k = 11, 48, 3
    m = Maps(T, k, 16, 4)
    x = torch.randint(0, 2, (T, H), device="cuda").to(dtype)
    out = Guarded((m.R, H), dtype)
    mfr.DispatchPlan(T, H, k, m.R, dtype=dtype).run(x, m.d_row, m.d_slot, out.t)
    torch.cuda.synchronize()
    here = torch.from_numpy(m.slot_of >= 0).cuda()
    assert torch.equal(out.check()[here], x[torch.from_numpy(m.slot_of[m.slot_of >= 0] // k).cuda()])


@pytest.mark.parametrize("T,H,k", ROWS)
@pytest.mark.parametrize("align,share", [(1, 0.0), (4, 0.25)])
def test_dispatch_grad(T, H, k, align, share):
    m = Maps(T, k, max(16, k), align, share)
    d = randn((m.R, H), 3, B16)
    plan = mfr.DispatchPlan(T, H, k, m.R, sentinel_skip=True)
    out = Guarded((T, H), B16)
    plan.run_grad(d, m.d_row, out.t)
    torch.cuda.synchronize()
    rows = np.where((m.row_of >= 0)[..., None], ref.f64(d)[np.maximum(m.row_of, 0)], 0.0)
    want, size = rows.sum(1), np.abs(rows).sum(1)
    ref.assert_within(ref.f64(out.check()), want, (1 + k * ref.U) * ref.BF16 * np.abs(want) + 2 * k * ref.U * size + ref.TINY, "d_x")
    assert plan.get_status() == 0


@pytest.mark.parametrize("T,H,k", ROWS)
@pytest.mark.parametrize("align,share", [(1, 0.0), (4, 0.25), (32, 0.0)])
@pytest.mark.parametrize("dtype", [B16, F32])
def test_finalize_grad(T, H, k, align, share, dtype):
    m = Maps(T, k, max(16, k), align, share)
    g, E = randn((T, H), 1, dtype), randn((m.R, H), 2, B16)
    w = randn((T, k), 3, F32)
    plan = mfr.FinalizeGradPlan(T, H, k, m.R, grad_dtype=dtype, sentinel_skip=True)
    dE, dw = Guarded((m.R, H), B16), Guarded((T, k), F32)
    plan.run(g, E, m.d_row, m.d_slot, w, dE.t, dw.t)
    torch.cuda.synchronize()
    rows, d_w, size = ref.finalize_grad(ref.f64(g), ref.f64(E), m.row_of, m.slot_of, ref.f64(w))
    got = ref.f64(dE.check())
    left = np.isnan(rows).any(1)
    assert (dE.t[torch.from_numpy(left).cuda()].view(torch.uint8) == 0x5A).all()
    # one FP32 product rounded to bf16
    ref.assert_within(got[~left], rows[~left], (ref.BF16 * (1 + ref.U) + ref.U) * np.abs(rows[~left]) + ref.TINY, "d_expert_out")
    ref.assert_within(ref.f64(dw.check()), d_w, ref.CHAIN * ref.U * size + ref.TINY, "d_topk_weights")
    assert plan.get_status() == 0


@pytest.mark.parametrize("op", ["dispatch", "finalize_grad"])
def test_maps_that_disagree(op):
    """Indexes out of range, two pairs with one row, rows whose pair points
    elsewhere: reported, never written, never read out of bounds; every
    other row and pair is as it should be."""
    T, H, k, E = 40, 264, 4, 8
    m = Maps(T, k, E, 4)
    clean_row, clean_slot = m.row_of.copy(), m.slot_of.copy()
    edits = [
        lambda r, s: r.__setitem__((0, 0), m.R),                    # beyond the rows
        lambda r, s: r.__setitem__((1, 1), -1),                     # not local, but its row says otherwise
        lambda r, s: r.__setitem__((2, 2), r[3, 3]),                # two pairs with the same row
        lambda r, s: r.__setitem__((5, 0), 2 ** 31 - 1),
        lambda r, s: s.__setitem__(int(r[6, 1]), T * k),            # a pair beyond the pairs
        lambda r, s: s.__setitem__(int(r[7, 1]), 2 ** 31 - 1),
        lambda r, s: s.__setitem__(int(r[8, 1]), -3),               # no such mark
        lambda r, s: s.__setitem__(int(r[9, 1]), -1),               # a pair's row marked as padding
    ]
    x, Eo, w = randn((T, H), 1, B16), randn((m.R, H), 2, B16), randn((T, k), 3, F32)
    for n, edit in enumerate(edits):
        m.row_of, m.slot_of = clean_row.copy(), clean_slot.copy()
        edit(m.row_of, m.slot_of)
        m.upload()
        out, dw = Guarded((m.R, H), B16), Guarded((T, k), F32)
        if op == "dispatch":
            plan = mfr.DispatchPlan(T, H, k, m.R, sentinel_skip=True)
            plan.run(x, m.d_row, m.d_slot, out.t)
        else:
            plan = mfr.FinalizeGradPlan(T, H, k, m.R, sentinel_skip=True)
            plan.run(x, Eo, m.d_row, m.d_slot, w, out.t, dw.t)
        torch.cuda.synchronize()
        assert plan.get_status() == mfr.STATUS_BAD_INDEX, n
        got = out.check().view(torch.uint8).cpu().numpy().reshape(m.R, -1)
        rows, d_w, size = ref.finalize_grad(ref.f64(x), ref.f64(Eo), m.row_of, m.slot_of,
                                            np.ones((T, k)) if op == "dispatch" else ref.f64(w))
        for r in range(m.R):
            s = m.slot_of[r]
            mine = 0 <= s < T * k and m.row_of.reshape(-1)[s] == r
            if mine or s == -1:
                ref.assert_within(ref.f64(out.t[r]), rows[r], 2 * ref.BF16 * np.abs(rows[r]) + ref.TINY, f"row {r}")
            else:
                assert (got[r] == 0x5A).all(), (n, r)
        if op == "finalize_grad":
            ref.assert_within(ref.f64(dw.check()), d_w, ref.CHAIN * ref.U * size + ref.TINY, "d_topk_weights")


def test_a_negative_row_needs_sentinel_skip():
    m = Maps(5, 4, 8, 1, share=0.5)
    x = randn((5, 64), 1, B16)
    plan = mfr.DispatchPlan(5, 64, 4, m.R)
    plan.run(x, m.d_row, m.d_slot, torch.empty((m.R, 64), dtype=B16, device="cuda"))
    assert plan.get_status() == mfr.STATUS_BAD_INDEX
    with pytest.raises(mfr.MFRError) as e:
        mfr.DispatchPlan(5, 64, 4, m.R, debug_checks=True).run(x, m.d_row, m.d_slot,
                                                              torch.empty((m.R, 64), dtype=B16, device="cuda"))
    assert e.value.name == "MFR_ERR_BAD_INDEX"


def test_no_rows_at_all():
    """Every pair non-local and R = 0: nothing to copy, gradients of 0."""
    T, H, k = 3, 64, 4
    row, slot = torch.full((T, k), -1, dtype=I32, device="cuda"), torch.empty(0, dtype=I32, device="cuda")
    none = torch.empty((0, H), dtype=B16, device="cuda")
    x, w = randn((T, H), 1, B16), randn((T, k), 1, F32)
    p = mfr.DispatchPlan(T, H, k, 0, sentinel_skip=True)
    p.run(x, row, slot, none)
    d_x = torch.ones((T, H), dtype=B16, device="cuda")
    p.run_grad(none, row, d_x)
    dw = torch.ones((T, k), device="cuda")
    q = mfr.FinalizeGradPlan(T, H, k, 0, sentinel_skip=True)
    q.run(x, none, row, slot, w, none, dw)
    torch.cuda.synchronize()
    assert not d_x.any() and not dw.any() and p.get_status() == 0 and q.get_status() == 0


def test_rows_past_32_bit_offsets():
    """Rows of a matrix of more than 2^32 bytes and 2^31 elements."""
    T, H, k = 34000, 8192, 8
    R = T * k                                    # 272000 rows, 4.5 GB
    g = torch.Generator(device="cuda").manual_seed(1)
    row = torch.randperm(R, generator=g, device="cuda").to(I32)
    slot = torch.empty(R, dtype=I32, device="cuda")
    slot[row.long()] = torch.arange(R, dtype=I32, device="cuda")
    row = row.view(T, k)
    x = torch.randn((T, H), generator=g, device="cuda").to(B16)
    out = torch.empty((R, H), dtype=B16, device="cuda")
    p = mfr.DispatchPlan(T, H, k, R)
    p.run(x, row, slot, out)
    for a in range(0, R, 16000):
        assert torch.equal(out[a:a + 16000], x[slot[a:a + 16000].long() // k])
    w = torch.randn((T, k), generator=g, device="cuda")
    dE, dw = torch.empty_like(out), torch.empty((T, k), device="cuda")
    q = mfr.FinalizeGradPlan(T, H, k, R)
    q.run(x, out, row, slot, w, dE, dw)
    for a in range(0, R, 16000):
        s = slot[a:a + 16000].long()
        assert torch.equal(dE[a:a + 16000], (w.view(-1)[s][:, None] * x[s // k].float()).to(B16))
    sq = (x.double() ** 2).sum(1)                # every row of a token is the token's own
    assert ((dw.double() - sq[:, None]).abs() <= ref.CHAIN * ref.U * sq[:, None]).all()
    assert p.get_status() == 0 and q.get_status() == 0


def test_many_unused_rows():
    """A matrix of far more rows than the tokens have: the rest is left as it was."""
    T, H, k, R = 2, 8, 3, 3000000
    row = torch.tensor([[5, R - 1, 70000], [1234567, 0, 2999998]], dtype=I32, device="cuda")
    slot = torch.full((R,), -2, dtype=I32, device="cuda")
    slot[row.view(-1).long()] = torch.arange(6, dtype=I32, device="cuda")
    slot[17], slot[R - 3] = -1, -1
    x, w = randn((T, H), 1, B16), randn((T, k), 2, F32)
    out, dE, dw = Guarded((R, H), B16), Guarded((R, H), B16), Guarded((T, k), F32)
    p, q = mfr.DispatchPlan(T, H, k, R), mfr.FinalizeGradPlan(T, H, k, R)
    p.run(x, row, slot, out.t)
    E = out.t.clone()
    q.run(x, E, row, slot, w, dE.t, dw.t)
    torch.cuda.synchronize()
    for buf, want in ((out, x[:, None, :].expand(T, k, H)), (dE, (w[..., None] * x[:, None, :].float()).to(B16))):
        t = buf.check()
        assert torch.equal(t[row.view(-1).long()], want.reshape(-1, H)) and not t[17].any() and not t[R - 3].any()
        rest = torch.ones(R, dtype=torch.bool, device="cuda")
        rest[row.view(-1).long()] = rest[17] = rest[R - 3] = False
        assert (t.view(torch.uint8)[rest] == 0x5A).all()
    sq = (ref.f64(x) ** 2).sum(1)[:, None] * np.ones((1, k))
    ref.assert_within(ref.f64(dw.check()), sq, ref.CHAIN * ref.U * sq, "d_w")
    assert p.get_status() == 0 and q.get_status() == 0


def test_norms_past_32_bit_offsets():
    """Residual norm and its gradient over more than 2^31 elements, the last
    rows and d_gamma against 64 bits."""
    T, H = 135000, 16384
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((T, H), dtype=B16, device="cuda")
    res = torch.empty((T, H), device="cuda")
    for a in range(0, T, 9000):
        x[a:a + 9000] = torch.randn((min(9000, T - a), H), generator=g, device="cuda")
        res[a:a + 9000] = torch.randn((min(9000, T - a), H), generator=g, device="cuda")
    gamma = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(B16)
    p = mfr.ResidualNormPlan(T, H, quant=mfr.QUANT_MX32)
    q, sf = torch.empty((T, H), dtype=FP8, device="cuda"), torch.empty(p.sf_shape(), dtype=torch.uint8, device="cuda")
    last = slice(T - 40, T)
    before = res[last].clone()
    p.run(x, res, res, gamma, 1e-6, None, q, sf)
    check_norm(x[last], before, gamma, 1e-6, mfr.QUANT_MX32, False, [res[last], None, q[last], sf[last]])
    del q
    n = mfr.ResidualNormGradPlan(T, H)
    d_in, d_x, d_g = torch.empty_like(res), torch.empty_like(x), torch.empty(H, device="cuda")
    n.run(x, None, res, gamma, 1e-6, d_in, d_g, torch.empty(n.workspace_bytes(), dtype=torch.uint8, device="cuda"), d_x)
    want, size, _, _ = ref.residual_norm_grad(ref.f64(x[last]), None, ref.f64(res[last]), ref.f64(gamma), 1e-6)
    ref.assert_within(ref.f64(d_in[last]), want, ref.GRAD_REL * size + ref.TINY, "d_residual_in")
    assert torch.equal(d_x[last], d_in[last].to(B16))
    dg, dg_size = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
    for a in range(0, T, 9000):
        r = res[a:a + 9000].double()
        term = x[a:a + 9000].double() * r * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6)
        dg += term.sum(0)
        dg_size += term.abs().sum(0)
    chain = T / 152 + 1 + 152 * 8 / 8 + 8
    ref.assert_within(ref.f64(d_g), dg.cpu().numpy(), ((chain + 4) * ref.U + ref.Y_REL) * dg_size.cpu().numpy(), "d_gamma")
    assert p.get_status() == 0 and n.get_status() == 0


# ---- residual norm ------------------------------------------------------------------------

NORMS = [(1, 8), (1, 4096), (60, 12288), (50, 12296), (45, 9000), (2, 24), (5, 136), (3, 1000), (7, 2056), (130, 4096), (33, 8192), (17, 8200), (9, 16384),
         (300, 264), (257, 64)]


def norm_inputs(T, H, seed=0):
    return (randn((T, H), seed + 1, B16), randn((T, H), seed + 2, F32, 2.0),
            (1 + 0.3 * randn((H,), seed + 3, F32)).to(B16))


def run_norm(x, res, gamma, eps, quant, tiled=False, bf16=True, inplace=False):
    T, H = x.shape
    plan = mfr.ResidualNormPlan(T, H, quant=quant, sf_layout=mfr.SF_TILED_128x4 if tiled else mfr.SF_ROW_MAJOR)
    res_out = Guarded((T, H), F32)
    if inplace:
        res_out.t.copy_(res)
        res = res_out.t
    out = Guarded((T, H), B16) if bf16 or quant == mfr.QUANT_NONE else None
    q = sf = None
    if quant != mfr.QUANT_NONE:
        q = Guarded((T, H), FP8)
        sf = Guarded(plan.sf_shape(), torch.uint8 if quant == mfr.QUANT_MX32 else F32)
        assert sf.n == plan._lib.moe_residual_rmsnorm_sf_bytes(plan._h)
    plan.run(x, res, res_out.t, gamma, eps, out.t if out else None, q.t if q else None, sf.t if sf else None)
    torch.cuda.synchronize()
    return [o.check() if o else None for o in (res_out, out, q, sf)]


def untile(sf, T, S):
    t, b = np.arange(T)[:, None], np.arange(S)[None, :]
    return sf[(t // 128 * -(-S // 4) + b // 4) * 512 + t % 32 * 16 + t // 32 % 4 * 4 + b % 4]


def check_norm(x, res, gamma, eps, quant, tiled, got):
    T, H = x.shape
    r, y, _ = ref.residual_norm(ref.f64(x), res.cpu().numpy(), ref.f64(gamma), eps)
    res_out, out, q, sf = got
    assert np.array_equal(res_out.cpu().numpy().view(np.uint32), r.view(np.uint32))       # one FP32 addition
    if out is not None:
        ref.assert_within(ref.f64(out), y, (ref.BF16 + 2 * ref.Y_REL) * np.abs(y) + ref.TINY, "out")
    if q is None:
        return
    size = {mfr.QUANT_TOKEN: H, mfr.QUANT_GROUP128: 128, mfr.QUANT_MX32: 32}[quant]
    amax = ref.group_amax(y, size)
    if quant == mfr.QUANT_MX32:
        S = -(-H // 32)
        raw = sf.cpu().numpy()
        if tiled:
            used = np.zeros(raw.size, dtype=bool)
            used[untile(np.arange(raw.size), T, S)] = True
            assert (raw[~used] == 0x5A).all()              # padding bytes are not written
            raw = untile(raw, T, S)
        scale = 2.0 ** (raw.astype(np.float64) - 127)
        assert (amax * (1 - ref.Y_REL) <= 448 * scale).all() and (amax * (1 + ref.Y_REL) > 224 * scale).all()
    else:
        scale = ref.f64(sf)
        ref.assert_within(scale, amax / 448, (ref.Y_REL + 2 * ref.U) * amax / 448, "scale")
    full = np.repeat(scale, size, axis=1)[:, :H]
    # E4M3 rounds a value to half a step: 2^-4 of it, or 2^-10 of the scale below the normals; y / scale
    # carries Y_REL, the scale's error and two more roundings
    v = np.abs(y) / full
    tol = np.maximum(ref.E4M3 * v, 2.0 ** -10) + (2 * ref.Y_REL + 4 * ref.U) * v * 1.07
    ref.assert_within(ref.f64(q), y / full, tol, "out_q")


QUANTS = [(mfr.QUANT_NONE, False), (mfr.QUANT_TOKEN, False), (mfr.QUANT_GROUP128, False), (mfr.QUANT_MX32, False),
          (mfr.QUANT_MX32, True)]


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("quant,tiled", QUANTS)
def test_residual_norm(T, H, quant, tiled):
    x, res, gamma = norm_inputs(T, H)
    for bf16, inplace, eps in ((True, False, 1e-6), (False, True, 1e-5)):
        check_norm(x, res, gamma, eps, quant, tiled, run_norm(x, res, gamma, eps, quant, tiled, bf16, inplace))


@pytest.mark.parametrize("quant,tiled", QUANTS[1:])
def test_residual_norm_extreme_rows(quant, tiled):
    """Rows of zeros, tiny and huge values, one value far above the rest, and
    groups below the floor of the scales."""
    T, H = 8, 520
    x, res, gamma = norm_inputs(T, H, 9)
    x[0], res[0] = 0, 0                                    # zeros: scale at its floor, codes 0
    x[1], res[1] = 0, res[1] * 1e-30                       # eps rules the root
    x[2], res[2] = 0, res[2] * 1e15
    res[3, 100] = 1e6
    gamma[128:256] = 0                                     # a group of zeros in every row
    x[4], res[4] = 0, 0
    res[4, 7] = 1.0
    check_norm(x, res, gamma, 1e-6, quant, tiled, run_norm(x, res, gamma, 1e-6, quant, tiled))


@pytest.mark.parametrize("quant,tiled", QUANTS[1:])
def test_residual_norm_nan_and_inf_stay_in_their_rows(quant, tiled):
    T, H = 6, 264
    x, res, gamma = norm_inputs(T, H, 11)
    clean = run_norm(x, res, gamma, 1e-6, quant, tiled)
    x[1, 5] = float("nan")
    res[3, 200] = float("inf")
    got = run_norm(x, res, gamma, 1e-6, quant, tiled)
    q = got[2].view(torch.uint8).cpu().numpy()
    assert (q[1] == 0x7F).all() or ((q[1] & 0x7F) == 0x7F).all()
    assert (q[3, 200] & 0x7F) == 0x7F and (np.delete(q[3], 200) & 0x7F == 0).all()      # x * 0 and inf * 0
    keep = [0, 2, 4, 5]
    assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[1][keep], clean[1][keep])
    assert np.array_equal(q[keep], clean[2].view(torch.uint8).cpu().numpy()[keep])
    if not tiled:
        assert torch.equal(got[3][keep], clean[3][keep])


@pytest.mark.parametrize("quant", [mfr.QUANT_GROUP128, mfr.QUANT_MX32, mfr.QUANT_TOKEN])
def test_residual_norm_infinite_values_saturate(quant):
    """An infinite gamma gives infinite y: amax is taken as FLT_MAX, the codes saturate."""
    x, res, gamma = norm_inputs(2, 256, 3)
    gamma[3] = float("inf")
    got = run_norm(x, res, gamma, 1e-6, quant)
    assert (got[2].float()[:, 3].abs() == 448).all()
    assert torch.isinf(got[1][:, 3]).all()
    assert not torch.isnan(got[2].float()).any()


@pytest.mark.parametrize("m", [1.75, 1.7578125, 1.0, 1.9921875])
def test_residual_norm_mx_scale_at_its_border(m):
    """448 = 1.75 * 2^8: a group whose largest magnitude is exactly 1.75 * 2^n
    needs no larger scale, the next bf16 value does.  y is exact here: one
    column of value sqrt(H) a row (inv = 1) times gamma, eps = 0."""
    H = 64
    res = torch.zeros((1, H), device="cuda")
    res[0, 10] = 8.0                                       # mean of squares = 1
    gamma = torch.full((H,), m / 8 * 16, dtype=B16, device="cuda")
    got = run_norm(torch.zeros((1, H), dtype=B16, device="cuda"), res, gamma, 0.0, mfr.QUANT_MX32)
    y = 8.0 * float(gamma[0])
    assert abs(float(got[1][0, 10]) - y) <= ref.BF16 * y
    sf = int(got[3][0, 0]) - 127
    assert sf == 4 - 8 + (1 if m > 1.75 else 0)            # y = m * 2^4
    assert int(got[3][0, 1]) == 127 - 100 - 8              # a group of zeros: the floor 2^-100


# ---- its gradient ----------------------------------------------------------------------------

def run_norm_grad(d_out, d_res, r, gamma, eps, d_x=True, inplace=False):
    T, H = r.shape
    plan = mfr.ResidualNormGradPlan(T, H)
    d_in, dx, dg = Guarded((T, H), F32), Guarded((T, H), B16) if d_x else None, Guarded((H,), F32)
    ws = Guarded((plan.workspace_bytes(),), torch.uint8)
    if inplace:
        d_in.t.copy_(d_res)
        d_res = d_in.t
    plan.run(d_out, d_res, r, gamma, eps, d_in.t, dg.t, ws.t, dx.t if d_x else None)
    torch.cuda.synchronize()
    ws.check()
    return d_in.check(), dx.check() if d_x else None, dg.check()


@pytest.mark.parametrize("T,H", NORMS + [(1500, 128), (3000, 8), (700, 4104)])
@pytest.mark.parametrize("kind", ["plain", "inplace", "no_residual_gradient"])
def test_residual_norm_grad(T, H, kind):
    d_out, r, gamma = norm_inputs(T, H, 20)
    d_res = None if kind == "no_residual_gradient" else randn((T, H), 5, F32)
    eps = 1e-5
    d_in, d_x, d_gamma = run_norm_grad(d_out, d_res, r, gamma, eps, d_x=kind != "inplace", inplace=kind == "inplace")
    want, size, dg, dg_size = ref.residual_norm_grad(ref.f64(d_out), None if d_res is None else ref.f64(d_res), ref.f64(r),
                                                     ref.f64(gamma), eps)
    ref.assert_within(ref.f64(d_in), want, ref.GRAD_REL * size + ref.TINY, "d_residual_in")
    if d_x is not None:
        assert torch.equal(d_x, d_in.to(B16))              # the FP32 result rounded once
    # over the tokens: a CTA adds at most ceil(T / 152) + 1 terms, then come its partial sums and 8 warps
    chain = T / 152 + 1 + 152 * 8 / 8 + 8
    ref.assert_within(ref.f64(d_gamma), dg, (chain + 4) * ref.U * dg_size + ref.Y_REL * dg_size + ref.TINY, "d_gamma")


def test_residual_norm_grad_without_tokens():
    z = torch.empty((0, 64), device="cuda")
    dg = torch.ones(64, device="cuda")
    p = mfr.ResidualNormGradPlan(0, 64)
    assert p.workspace_bytes() == 0
    p.run(z.to(B16), z, z, torch.ones(64, dtype=B16, device="cuda"), 1e-6, z.clone(), dg, None)
    torch.cuda.synchronize()
    assert not dg.any()


def test_residual_norm_grad_at_large_and_small_rows():
    """Rows whose inv^3 would leave the FP32 range."""
    T, H = 4, 256
    d_out, r, gamma = norm_inputs(T, H, 30)
    r[0] *= 1e15
    r[1] *= 1e-12
    d_res = torch.zeros((T, H), device="cuda")
    eps = 0.0
    d_in, _, d_gamma = run_norm_grad(d_out, d_res, r, gamma, eps)
    want, size, dg, dg_size = ref.residual_norm_grad(ref.f64(d_out), None, ref.f64(r), ref.f64(gamma), eps)
    ref.assert_within(ref.f64(d_in), want, ref.GRAD_REL * size + ref.TINY, "d_residual_in")
    ref.assert_within(ref.f64(d_gamma), dg, (16 * ref.U + ref.Y_REL) * dg_size, "d_gamma")


# ---- refusals of the C side (checked before any launch) ------------------------------------------

def test_c_calls_refuse_bad_pointers():
    lib = mfr.load_library()
    T, H, k, R = 4, 64, 4, 16
    buf = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    at = [buf.data_ptr() + 65536 * i for i in range(12)]
    INVALID, MISALIGNED = 1, 3
    route, disp = mfr.RoutePlan(T, k, 8), mfr.DispatchPlan(T, H, k, R)
    big = mfr.RoutePlan(40000, 8, 8)
    fgrad, norm, ngrad = mfr.FinalizeGradPlan(T, H, k, R), mfr.ResidualNormPlan(T, H), mfr.ResidualNormGradPlan(T, H)
    need = ngrad.workspace_bytes()
    calls = {
        "moe_route_run": (route, [at[0], at[1], at[2], at[3], at[4], None, 0, None], range(5)),
        "moe_dispatch_run": (disp, [at[0], None, at[1], at[2], at[3], None, None], (0, 2, 3, 4)),
        "moe_dispatch_grad_run": (disp, [at[0], at[1], at[2], None], range(3)),
        "moe_finalize_grad_run": (fgrad, [at[0], at[1], at[2], at[3], at[4], at[5], at[6], None], range(7)),
        "moe_residual_rmsnorm_run": (norm, [at[0], at[1], at[2], at[3], 1e-6, None, at[4], at[5], None], (0, 1, 2, 3, 6, 7)),
        "moe_residual_rmsnorm_grad_run": (ngrad, [at[0], at[1], at[2], at[3], 1e-6, at[4], None, at[5], at[6], need, None],
                                          (0, 2, 3, 5, 7, 8)),
    }
    for name, (plan, args, pointers) in calls.items():
        fn = getattr(lib, name)
        for i in pointers:
            for value, code in ((None, INVALID), (args[i] + 2, MISALIGNED)):
                bad = list(args)
                bad[i] = value
                assert fn(plan._h, *bad) == code, (name, i, value)
        others = [p for p in (route, disp, fgrad, norm, ngrad) if p is not plan]
        for other in others:
            assert fn(other._h, *args) == INVALID
        assert fn(plan._h, *args) == 0, name
    # outputs that meet an input or one another
    assert lib.moe_dispatch_run(disp._h, at[0], None, at[1], at[2], at[0], None, None) == INVALID
    assert lib.moe_route_run(route._h, at[0], at[1], at[1], at[3], at[4], None, 0, None) == INVALID
    assert lib.moe_finalize_grad_run(fgrad._h, at[0], at[1], at[2], at[3], at[4], at[1], at[6], None) == INVALID
    assert lib.moe_residual_rmsnorm_run(norm._h, at[0], at[1], at[1] + 16, at[3], 1e-6, None, at[4], at[5], None) == INVALID
    assert lib.moe_residual_rmsnorm_run(norm._h, at[0], at[1], at[2], at[3], -1.0, None, at[4], at[5], None) == INVALID
    assert lib.moe_residual_rmsnorm_run(norm._h, at[0], at[1], at[2], at[3], float("nan"), None, at[4], at[5], None) == INVALID
    g = calls["moe_residual_rmsnorm_grad_run"][1]
    assert lib.moe_residual_rmsnorm_grad_run(ngrad._h, *g[:9], need - 1, None) == INVALID
    assert lib.moe_route_run(big._h, at[0], at[1], at[2], at[3], at[4], None, 0, None) == INVALID
    fp8 = mfr.DispatchPlan(T, H, k, R, dtype=FP8, sf_bytes=4)
    assert lib.moe_dispatch_grad_run(fp8._h, at[0], at[1], at[2], None) == INVALID
    assert lib.moe_dispatch_run(fp8._h, at[0], None, at[1], at[2], at[3], at[4], None) == INVALID
    torch.cuda.synchronize()
