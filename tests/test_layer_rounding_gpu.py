"""What the MoE layer for a few tokens holds of h, on inputs whose first products are
exact: every column, both of its bf16 parts, every E4M3 group and scale."""
import pytest
import torch

import exact_layer as el
import moe_finalize_residual_rmsnorm_gb300 as mfr
import step_ref as ref
from test_small_layer_gpu import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


# 16, 32, 64 and 128 columns; units divided along K in the first product, the second, both, none
SHAPES = [(10, 264, 200, 1, 1), (10, 1552, 704, 1, 1), (20, 1808, 1000, 1, 1), (60, 2048, 704, 1, 1), (120, 2048, 704, 1, 1),
          (300, 2608, 704, 2, 1), (3, 264, 2056, 2, 2), (37, 520, 264, 24, 4), (100, 1040, 264, 8, 4), (150, 520, 264, 12, 8),
          (128, 264, 136, 3, 2), (200, 264, 136, 1, 1)]
SHAPES8 = [(1, 272, 256, 1, 1), (20, 2064, 1536, 1, 1), (60, 1552, 1536, 1, 1), (120, 2048, 1408, 1, 1), (300, 2608, 1408, 2, 1),
           (3, 272, 2048, 2, 2), (16, 272, 384, 7, 4), (100, 384, 256, 2, 2), (37, 528, 256, 24, 4)]


@pytest.mark.parametrize("T,H,I,E,k,fp8", [(*s, False) for s in SHAPES] + [(*s, True) for s in SHAPES8])
def test_every_column_of_h_counts(T, H, I, E, k, fp8):
    i = (el.inputs_e4m3 if fp8 else el.inputs_bf16)(T, H, I, E, k, seed=T)
    layer = Layer(T, H, I, E, k, fp8)
    layer.run({n: t.cuda() for n, t in i.items()})
    torch.cuda.synchronize()
    assert layer.plan.get_status() == 0
    want, tol = el.layer(i)
    ref.assert_within(layer.out.check(), want, tol, "out")
