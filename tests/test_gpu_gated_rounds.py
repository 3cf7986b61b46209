"""Gated products of decode batches over wide stacks of long rows, which take several
rounds of workgroups or of activations: every number of row groups of the dispatch."""
import pytest
import torch

import gated_ref as gr
import operators_ref as ref
from gated_ref import BF16, F32, Packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from ternary_weight_linear_bitlinear_amd import bitlinear
    return bitlinear


@pytest.mark.parametrize("layout,M,F,K", [
    ("base3", 16, 6500, 5300), ("base3", 9, 8192, 8192), ("base3", 40, 8192, 5136), ("base3", 13, 8193, 5200),
    ("base3", 16, 12300, 5201), ("2bit", 16, 6500, 4112), ("2bit", 11, 8200, 8192), ("2bit", 47, 12290, 4100),
    ("1bit", 16, 6500, 8200), ("1bit", 33, 8200, 8320)])
def test_forward(bl, layout, M, F, K):
    p = Packed(bl, M, [F, F], K, layout, seed=M + F)
    r = bl.bitlinear_forward_gated(p.xq, p.scale, p.packed, p.gammas, F, K, layout, act="silu", out_dtype=F32, z=True)
    z, tol = p.z()
    ref.close(r.z, z, tol, "z")
    ref.close(r.y, gr.gated(z, "silu"), gr.gated_tol(z, tol, "silu"), "y")
    low = bl.bitlinear_forward_gated(p.xq, p.scale, p.packed, p.gammas, F, K, layout, act="silu", out_dtype=BF16).y
    assert torch.equal(low, r.y.to(BF16))
