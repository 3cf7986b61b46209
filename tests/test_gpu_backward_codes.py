"""Weight gradients from INT8 codes and input gradients over stacks, against 64-bit
products. Every product term is exact in fp32 (grad_w's factor after the two
roundings that define it), so a sum of n terms is off by at most n u times the sum
of their absolute values, in any order."""
import pytest
import torch

import operators_ref as ref
from gated_ref import BF16, F32, TYPES, U, Packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from ternary_weight_linear_bitlinear_amd import bitlinear
    return bitlinear


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 8, 16), (5, 3, 7), (32, 256, 256), (33, 264, 272), (100, 1003, 2001),
                                   (64, 130, 15), (250, 257, 300), (1000, 72, 80), (77, 4100, 4112), (4096, 64, 48)])
@pytest.mark.parametrize("gy,gw", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_weight(bl, M, N, K, gy, gw):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    grad_y = (torch.randn(M, N, generator=g, device="cuda") * 1e-3).to(TYPES[gy])
    xq, scale = bl.bitlinear_quant_acts(torch.randn(M, K, generator=g, device="cuda") * 5)
    got = bl.bitlinear_backward_weight_codes(grad_y, xq, scale, TYPES[gw])
    v = grad_y.cpu().double() * (scale.cpu().double() / 127)[:, None]
    want, terms = v.t() @ xq.cpu().double(), v.abs().t() @ xq.cpu().double().abs()
    # three pieces a term of one sign; or two, which leave out less than 2^-15
    rel = (3 * M + 4) * U if gw == "f32" else 2.0 ** -15 + (2 * M + 4) * U
    ref.close(got, want, rel * terms, "grad_w")


def test_weight_pieces_carry_every_bit(bl):
    """One token: each output is one product, to the roundings of the scale's quotient
    and of its product with grad_y (and none of the sum of its pieces, beyond one)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    for e in (-60, -10, 0, 20):
        grad_y = torch.randn(1, 40, generator=g, device="cuda") * 2.0 ** e
        xq = torch.arange(-127, 128, device="cuda", dtype=torch.int8)[None].contiguous()
        scale = torch.tensor([3.14159], device="cuda")
        got = bl.bitlinear_backward_weight_codes(grad_y, xq, scale)
        want = grad_y.cpu().double().t() * (scale.cpu().double() / 127) * xq.cpu().double()
        ref.close(got, want, 6 * U * want.abs(), "grad_w")


STACKS = [([256, 256], 256, 256), ([8], 5, 16), ([1], 1, 1), ([3, 5, 1, 9, 2, 40, 7, 33], 20, 77), ([1003, 500, 500], 200, 3000),
          ([72, 200], 130, 264), ([64, 64, 64], 257, 300), ([700, 704], 1000, 520), ([512, 512], 64, 4112)]


@pytest.mark.parametrize("segs,M,K", STACKS)
@pytest.mark.parametrize("layout", ["2bit", "base3", "1bit"])
@pytest.mark.parametrize("gy", ["f32", "bf16"])
def test_input(bl, segs, M, K, layout, gy):
    p = Packed(bl, 0, segs, K, layout, seed=M)
    check_input(bl, p, p.rand(M, sum(segs), dtype=TYPES[gy], scale=1e-3), F32 if M % 2 else BF16)


def check_input(bl, p, grad_y, gx):
    got = bl.bitlinear_backward_input_segmented(grad_y, p.packed, p.gammas, p.segs, p.K, p.layout, gx)
    v = grad_y.cpu().double() * p.row_gamma
    want, terms = v @ p.codes.double(), v.abs() @ p.codes.double().abs()
    # rescaling: a ratio and its product where a segment ends, gamma's at the end
    n = (3 if grad_y.dtype is F32 else 1) * sum(p.segs) + 3 * len(p.segs) + 2
    ref.close(got, want, n * U * terms, "grad_x")


@pytest.mark.parametrize("gammas", [[0.0, 1.0, 2.0], [2.0, 0.0, 0.5], [0.0, 0.0, 0.0], [1e30, 1e-30, 1.0], [1.0, 1.0, 1.0],
                                    [-0.5, 0.25, -2.0], [3e-39, 1e-3, 1e-42]])
def test_input_gammas(bl, gammas):
    """Segments in any order of gamma, zeros and the widest range among them."""
    p = Packed(bl, 0, [100, 72, 40], 96, seed=3, gammas=gammas)
    grad_y = p.rand(50, 212, dtype=BF16)
    got = bl.bitlinear_backward_input_segmented(grad_y, p.packed, p.gammas, p.segs, 96)
    v = grad_y.cpu().double() * p.row_gamma
    want, terms = v @ p.codes.double(), v.abs() @ p.codes.double().abs()
    # (a sum whose factor sinks below fp32's least normal value is lost, beside the others' 2^-126 / u)
    ref.close(got, want, (212 + 11) * U * terms + 2.0 ** -120, "grad_x")


def test_input_of_one_segment_is_the_plain_call(bl):
    p = Packed(bl, 0, [264], 528, seed=9)
    grad_y = p.rand(70, 264, dtype=BF16, scale=1e-3)
    got = bl.bitlinear_backward_input_segmented(grad_y, p.packed, p.gammas, 264, 528)
    plain = bl.bitlinear_backward_input(grad_y, p.packed, p.gammas, 528)
    ref.close(got, plain.cpu().double(), 2 * 266 * U * (grad_y.cpu().double().abs() @ p.codes.double().abs()) *
              float(p.gammas[0]), "grad_x")


def test_empty(bl):
    p = Packed(bl, 0, [24, 8], 64)
    assert bl.bitlinear_backward_input_segmented(torch.empty(0, 32, device="cuda"), p.packed, p.gammas, [24, 8],
                                                 64).shape == (0, 64)
    for dtype in (F32, BF16):
        w = bl.bitlinear_backward_weight_codes(torch.empty(0, 24, device="cuda"),
                                               torch.empty(0, 64, dtype=torch.int8, device="cuda"),
                                               torch.empty(0, device="cuda"), dtype)
        assert w.shape == (24, 64) and w.dtype is dtype and not w.any()
