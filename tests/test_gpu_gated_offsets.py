"""Tensors of more than 2^31 elements: the last rows of a large call are those of a call
on them alone, bit for bit, or the 64-bit definition's."""
import pytest
import torch

import gated_ref as gr
import operators_ref as ref
from gated_ref import BF16, F32, U, Packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from ternary_weight_linear_bitlinear_amd import bitlinear
    yield bitlinear
    torch.cuda.empty_cache()


def test_forward(bl):
    M, F, K, tail = 60000, 37000, 64, 300
    p = Packed(bl, M, [F, F], K, seed=1)
    y = bl.bitlinear_forward_gated(p.xq, p.scale, p.packed, p.gammas, F, K, out_dtype=BF16).y
    assert y.numel() > 2 ** 31
    last = bl.bitlinear_forward_gated(p.xq[-tail:].contiguous(), p.scale[-tail:].contiguous(), p.packed, p.gammas, F, K,
                                      out_dtype=BF16).y
    same = torch.equal(y[-tail:], last)
    assert same


@pytest.mark.parametrize("K", [36001, 36000])
def test_checkpoint_and_backward(bl, K):
    M, tail = 60000, 64
    z = torch.empty(M, K, dtype=BF16, device="cuda").normal_()
    kept = bl.bitlinear_checkpoint(z)
    back = bl.bitlinear_checkpoint_restore(kept, BF16)
    assert kept.codes.numel() > 2 ** 31
    codes, scale = gr.quantised(z[-tail:])
    same = [torch.equal(kept.codes[-tail:].cpu(), codes), torch.equal(kept.scale[-tail:].cpu(), scale),
            torch.equal(back[-tail:].cpu(), gr.restored(codes, scale).to(BF16))]
    assert all(same)
    del back
    gy = torch.empty(M // 2, K, dtype=BF16, device="cuda").normal_()
    pair = bl.Checkpoint(kept.codes, kept.scale)  # rows 2m and 2m + 1 of M / 2 tokens
    part = bl.Checkpoint(kept.codes[-tail:], kept.scale[-tail:])
    for whole, end in ((z.view(M // 2, 2 * K), z.view(M // 2, 2 * K)[-tail // 2:]), (pair, part)):
        if isinstance(end, bl.Checkpoint):
            end = bl.Checkpoint(end.codes.clone(), end.scale.clone())
        else:
            end = end.clone()
        g = bl.bitlinear_gated_backward(gy, whole, grad_bias=None).grad_z
        last = bl.bitlinear_gated_backward(gy[-tail // 2:].clone(), end, grad_bias=None).grad_z
        same = torch.equal(g[-tail // 2:], last)
        assert same


def test_weight(bl):
    M, N, K, tail = 8, 48008, 45008, 5
    gy = torch.empty(M, N, device="cuda").normal_()
    xq, scale = bl.bitlinear_quant_acts(torch.empty(M, K, device="cuda").normal_())
    gw = bl.bitlinear_backward_weight_codes(gy, xq, scale)
    assert gw.numel() > 2 ** 31
    v = gy.cpu().double()[:, -tail:] * (scale.cpu().double() / 127)[:, None]
    want, terms = v.t() @ xq.cpu().double(), v.abs().t() @ xq.cpu().double().abs()
    least = 2.0 ** -39 * v.abs().amax(0)[:, None] * xq.cpu().double().abs().sum(0)
    ref.close(gw[-tail:], want, (3 * M + 6) * U * terms + least, "grad_w")


@pytest.mark.parametrize("segs", [[5000, 3200], [5001, 3200]])
def test_input(bl, segs):
    M, K, tail = 270000, 64, 40
    p = Packed(bl, 0, segs, K, seed=4)
    gy = torch.empty(M, sum(segs), dtype=BF16, device="cuda").normal_()
    assert gy.numel() > 2 ** 31
    gx = bl.bitlinear_backward_input_segmented(gy, p.packed, p.gammas, segs, K)
    v = gy[-tail:].cpu().double() * p.row_gamma
    ref.close(gx[-tail:], v @ p.codes.double(), (sum(segs) + 12) * U * (v.abs() @ p.codes.double().abs()), "grad_x")
    assert gx.dtype is F32
