"""The bounds of exact_layer.py on the CPU: what the layer does with h is within
them, and mistakes with h are not."""
import pytest
import torch

import exact_layer as el
from step_ref import assert_within

B16 = torch.bfloat16


def parts(h):
    high = h.float().to(B16).double()
    return high, (h - high).float().to(B16).double()


def codes(h):
    g = h.view(h.shape[0], -1, 128)
    sf = g.abs().amax(-1, keepdim=True).clamp(min=el.AMAX_FLOOR) / 448
    return el.e4m3(g / sf), sf


def dropped(h, n):
    """h without its columns 128 .. 128 + n - 1 (as far as there are)."""
    h = h.clone()
    h[:, 128:128 + n] = 0
    return h


SHAPES = [(10, 264, 200, 1, 1), (20, 1808, 1000, 1, 1), (6, 264, 2056, 2, 2)]
SHAPES8 = [(20, 2064, 1536, 1, 1), (12, 272, 384, 4, 2), (6, 272, 2048, 2, 2)]


def shifted(low):
    return low.roll(1, 0)


BF16 = {
    "both parts": lambda h: sum(parts(h)),
    "no lower part": lambda h: parts(h)[0],
    "lower part subtracted": lambda h: parts(h)[0] - parts(h)[1],
    "the neighbouring pair's lower part": lambda h: parts(h)[0] + shifted(parts(h)[1]),
    "lower parts of the next 64 columns": lambda h: parts(h)[0] + parts(h)[1].roll(64, 1),
    "no lower part in 64 columns": lambda h: parts(h)[0] + dropped(parts(h)[1], 64),
}


@pytest.mark.parametrize("what", list(BF16))
@pytest.mark.parametrize("shape", SHAPES)
def test_bf16(shape, what):
    i = el.inputs_bf16(*shape)
    want, tol = el.layer(i)
    got = el.emulated(i, BF16[what])
    if what == "both parts":
        assert_within(got, want, tol, what)
    else:
        with pytest.raises(AssertionError):
            assert_within(got, want, tol, what)


def scaled(h, change):
    q, sf = codes(h)
    return (q * change(sf)).view(h.shape)


E4M3 = {
    "the rule": lambda h: scaled(h, lambda sf: sf),
    "not quantised": lambda h: h,
    "a group dropped": lambda h: dropped(scaled(h, lambda sf: sf), 128),
    "32 columns dropped": lambda h: dropped(scaled(h, lambda sf: sf), 32),
    "a column dropped": lambda h: dropped(scaled(h, lambda sf: sf), 1),
    "the next group's scales": lambda h: scaled(h, lambda sf: sf.roll(1, 1)),
    "the next pair's scales": lambda h: scaled(h, lambda sf: sf.roll(1, 0)),
}


@pytest.mark.parametrize("what", list(E4M3))
@pytest.mark.parametrize("shape", SHAPES8)
def test_e4m3(shape, what):
    i = el.inputs_e4m3(*shape)
    want, tol = el.layer(i)
    got = el.emulated(i, E4M3[what])
    if what == "the rule":
        assert_within(got, want, tol, what)
    else:
        with pytest.raises(AssertionError):
            assert_within(got, want, tol, what)


@pytest.mark.parametrize("fp8,shape", [(False, s) for s in SHAPES] + [(True, s) for s in SHAPES8])
def test_first_products_are_exact(fp8, shape):
    """Forwards, backwards and in 64 bits: the same numbers."""
    i = (el.inputs_e4m3 if fp8 else el.inputs_bf16)(*shape)
    x, a = i["x"].double(), i["w13"][0].double()
    if fp8:
        x = x * i["x_sf"].double().repeat_interleave(128, 1)[:, :x.shape[1]]
        a = a * el.spread(i["w13_sf"][0].double(), *a.shape)
    exact = x @ a.t()
    p = (x[:, None, :200] * a[None, :40, :200]).float()
    assert torch.equal(p.double(), x[:, None, :200] * a[None, :40, :200])
    total, back = torch.zeros(p.shape[:2]), torch.zeros(p.shape[:2])
    for n in range(p.shape[2]):
        total += p[:, :, n]
        back += p[:, :, -1 - n]
    assert torch.equal(total, back) and torch.equal(total.double(), x[:, :200] @ a[:40, :200].t())
    # whole multiples of the smallest factors' product, below 2^24 of them in all
    unit = x[x != 0].abs().min() * a[a != 0].abs().min()
    assert (x.abs() @ a.abs().t()).max() / unit < 2 ** 24 and torch.equal((exact / unit).round(), exact / unit)
