"""Input gradients over stacks in problems of large tiles, with gammas at the ends of
fp32's range (u = 2^-24)."""
import pytest
import torch

import operators_ref as ref
from gated_ref import TYPES, U, Packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from ternary_weight_linear_bitlinear_amd import bitlinear
    return bitlinear


def check_input(bl, p, grad_y, nonzero):
    got = bl.bitlinear_backward_input_segmented(grad_y, p.packed, p.gammas, p.segs, p.K, p.layout)
    v = grad_y.cpu().double() * p.row_gamma
    want, terms = v @ p.codes.double(), v.abs() @ p.codes.double().abs()
    # each segment's end and the last gamma: a ratio, its product, another
    n = max(4, sum(p.segs)) + 3 * nonzero + 3 * len(p.segs) + 6
    ref.close(got, want, n * U * terms, "grad_x")


@pytest.mark.parametrize("gammas,scale", [([1e32], 1.0), ([1e-44], 1e30), ([1e32, 1e-30], 1.0), ([-1e-30, 1e31], 1e-3),
                                          ([3e38, 1e-38], 1e-5), ([1e-44, 2e-44], 1e30)])
@pytest.mark.parametrize("gy", ["f32", "bf16"])
def test_input_gammas(bl, gammas, scale, gy):
    """Gammas at the ends of the range over equal codes: the sums of 600 equal signs, and
    what gamma makes of them, are inside fp32's."""
    M, K, segs = 4100, 4112, [600 // len(gammas)] * len(gammas)
    p = Packed(bl, 0, segs, K, seed=1, gammas=gammas)
    p.packed[:] = bl.bitlinear_pack_weights(torch.ones(600, K, device="cuda"))[0]
    p.codes = torch.ones(600, K, dtype=torch.int8)
    grad_y = ((1 + torch.rand(M, 600, generator=p.gen, device="cuda")) * scale).to(TYPES[gy])
    check_input(bl, p, grad_y, 600)
