"""The README's example of the operators around the finalize holds for every
width that they take, not only for multiples of 128."""
import os
import re

import pytest
import torch

import moe_finalize_residual_rmsnorm_gb300 as mfr

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def norm_plan(T, H, quant):
    p = mfr.ResidualNormPlan.__new__(mfr.ResidualNormPlan)      # shapes only: no device
    p._h, p.T, p.H, p.quant, p.sf_layout = None, T, H, quant, mfr.SF_ROW_MAJOR
    return p


@pytest.mark.parametrize("H", [8, 128, 2056, 4096, 4104, 8200, 16384])
def test_the_dispatch_takes_the_scales_that_the_norm_writes(H):
    text = open(README).read()
    sf_bytes = re.search(r"DispatchPlan\(.*sf_bytes=(.+)\)\n", text).group(1)
    quant = re.search(r"ResidualNormPlan\(T, H, quant=mfr\.(\w+)\)", text).group(1)
    shape = norm_plan(4, H, getattr(mfr, quant)).sf_shape()
    assert eval(sf_bytes, {"H": H}) == shape[1] * torch.float32.itemsize
