"""Weight gradients from INT8 codes and input gradients over stacks, against 64-bit
products. A term's factor is exact, or rounded twice by definition (grad_w's), and
enters in up to three pieces that leave out at most 2^-22 = 4 u of it (fp16 pieces of
a large problem; below fp16's normal range 2^-39 of the row's largest factor). Each
piece's product is exact in fp32, so a sum over n factors is off by at most 3 n u times
the sum of the terms' absolute values, in any order, besides the factors' own 6 u."""
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


# (problems of both tile sizes, and of both with several workgroups a tile)
@pytest.mark.parametrize("M,N,K", [(512, 2048, 2064), (4096, 1024, 1040), (512, 4096, 4112), (130, 3000, 3001), (2048, 300, 520), (4096, 1030, 1000), (1, 1, 1), (1, 8, 16), (5, 3, 7), (32, 256, 256), (33, 264, 272), (100, 1003, 2001),
                                   (64, 130, 15), (300, 5, 70000), (250, 257, 300), (1000, 72, 80), (77, 4100, 4112), (4096, 64, 48)])
@pytest.mark.parametrize("gy,gw", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_weight(bl, M, N, K, gy, gw):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    grad_y = (torch.randn(M, N, generator=g, device="cuda") * 1e-3).to(TYPES[gy])
    xq, scale = bl.bitlinear_quant_acts(torch.randn(M, K, generator=g, device="cuda") * 5)
    got = bl.bitlinear_backward_weight_codes(grad_y, xq, scale, TYPES[gw])
    v = grad_y.cpu().double() * (scale.cpu().double() / 127)[:, None]
    want, terms = v.t() @ xq.cpu().double(), v.abs().t() @ xq.cpu().double().abs()
    # grad_w in bf16: two bf16 pieces, cut off at eight bits each, leave out less than 2^-15;
    # one of fp16 is rounded, half a step of 2^-10
    rel = (3 * M + 6) * U if gw == "f32" else 2.0 ** -11 + (2 * M + 4) * U
    least = 2.0 ** -39 * v.abs().amax(0)[:, None] * xq.cpu().double().abs().sum(0)
    ref.close(got, want, rel * terms + least, "grad_w")


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


def test_weight_of_wide_range(bl):
    """Columns of any magnitude beside each other, zeros and single large tokens among
    them, in a problem of large tiles: each is scaled by its own power of two."""
    M, N, K = 300, 4096, 4096
    assert bl.bitlinear_backward_weight_codes_workspace_bytes(M, N, K) > 0
    g = torch.Generator(device="cuda").manual_seed(8)
    grad_y = torch.randn(M, N, generator=g, device="cuda") * torch.logspace(-34, 30, N, device="cuda")
    grad_y[:, ::7] = 0
    grad_y[17, 1::5] *= 1000.0
    xq, scale = bl.bitlinear_quant_acts(torch.randn(M, K, generator=g, device="cuda"))
    got = bl.bitlinear_backward_weight_codes(grad_y, xq, scale).cpu()
    v = grad_y.cpu().double() * (scale.cpu().double() / 127)[:, None]
    want, terms = v.t() @ xq.cpu().double(), v.abs().t() @ xq.cpu().double().abs()
    least = 2.0 ** -39 * v.abs().amax(0)[:, None] * xq.cpu().double().abs().sum(0)
    # (and what fp32 holds at all: products below 2^-126 lose bits)
    ref.close(got, want, (3 * M + 6) * U * terms + least + M * 2.0 ** -126, "grad_w")
    assert not got[::7].any()


STACKS = [([5], 65, 200), ([3, 6], 129, 64), ([256, 256], 256, 256), ([8], 5, 16), ([1], 1, 1), ([3, 5, 1, 9, 2, 40, 7, 33], 20, 77), ([1003, 500, 500], 200, 3000),
          ([72, 200], 130, 264), ([64, 64, 64], 257, 300), ([700, 704], 1000, 520), ([512, 512], 64, 4112),
          ([2000, 1000], 2100, 2056), ([600], 4100, 4112), ([301, 300], 4100, 4112), ([2000, 2001], 1100, 1500), ([4096], 512, 2050), ([4100, 4097], 300, 1500)]


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
    n = (3 if grad_y.dtype is F32 else 1) * sum(p.segs) + 3 * len(p.segs) + 6
    least = 2.0 ** -39 * grad_y.cpu().double().abs().amax(1)[:, None] * (
        p.row_gamma[:, None] * p.codes.double().abs()).sum(0) if grad_y.dtype is F32 else 0.0
    ref.close(got, want, n * U * terms + least, "grad_x")


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


@pytest.mark.parametrize("gy", ["f32", "bf16"])
def test_input_of_a_gamma_that_is_no_number(bl, gy):
    """Every segment keeps its place: the call ends, with NaN everywhere, and the next one is right."""
    nan = float("nan")
    for gammas in ([nan, 1.0, 2.0], [1.0, nan, nan], [nan] * 3, [float("inf"), nan, 0.0]):
        p = Packed(bl, 0, [100, 72, 41], 96, seed=3, gammas=gammas)
        grad_y = p.rand(50, 213, dtype=TYPES[gy])
        got = bl.bitlinear_backward_input_segmented(grad_y, p.packed, p.gammas, p.segs, 96)
        assert bool(got.isnan().all())
    check_input(bl, Packed(bl, 0, [100, 72, 41], 96, seed=3), grad_y, F32)


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


def test_gradients_are_the_derivatives(bl):
    """Against differences of the 64-bit loss sum(grad_y * y), y = (xq scale / 127) (gamma
    codes)^T: it is linear in the weights and in the input, so a difference of any step is the
    derivative. Its error is what the gradients' own bounds make of the direction."""
    M, K, segs = 60, 150, [70, 41]
    p = Packed(bl, M, segs, K, seed=12)
    gy = p.rand(M, sum(segs), scale=1e-2)
    x = p.xq.cpu().double() * (p.scale.cpu().double() / 127)[:, None]
    W, g64 = p.codes.double() * p.row_gamma[:, None], gy.cpu().double()
    loss = lambda x, W: (g64 * (x @ W.t())).sum()  # noqa: E731
    gw = bl.bitlinear_backward_weight_codes(gy, p.xq, p.scale).cpu().double()
    gx = bl.bitlinear_backward_input_segmented(gy, p.packed, p.gammas, segs, K).cpu().double()
    r = torch.Generator().manual_seed(3)
    for _ in range(4):
        D, E = torch.randn(W.shape, generator=r, dtype=torch.float64), torch.randn(x.shape, generator=r, dtype=torch.float64)
        dw, dx = (loss(x, W + D) - loss(x, W - D)) / 2, (loss(x + E, W) - loss(x - E, W)) / 2
        tw = (D.abs() * ((3 * M + 7) * U * (g64.abs().t() @ x.abs()))).sum()
        tx = (E.abs() * ((3 * sum(segs) + 12) * U * (g64.abs() @ W.abs()))).sum()
        assert (gw * D).sum().sub(dw).abs() <= tw + 1e-12 and (gx * E).sum().sub(dx).abs() <= tx + 1e-12
