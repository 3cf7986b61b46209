"""Activations kept in 8 bits: codes, scales and restored values bit for bit against
the definition in fp32, over widths that groups and vectors do not divide."""
import pytest
import torch

import gated_ref as gr
from gated_ref import BF16, F32, TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from ternary_weight_linear_bitlinear_amd import bitlinear
    return bitlinear


def check(bl, x, out=F32):
    kept = bl.bitlinear_checkpoint(x)
    codes, scale = gr.quantised(x)
    assert torch.equal(kept.scale.cpu(), scale)
    assert torch.equal(kept.codes.cpu(), codes)
    y = bl.bitlinear_checkpoint_restore(kept, out)
    assert y.dtype is out and torch.equal(y.cpu(), gr.restored(codes, scale).to(out))
    return kept


@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (300, 5), (1, 8), (5, 9), (17, 63), (4, 64), (4, 65), (2, 127),
                                 (333, 5001), (64, 2048), (9, 2056), (1000, 72), (31, 11008), (2, 70001), (1, 600001),
                                 (5000, 66), (70000, 8)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_bit_for_bit(bl, M, K, x):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    v = torch.randn(M, K, generator=g, device="cuda") * torch.rand(M, 1, generator=g, device="cuda") * 30
    check(bl, v.to(TYPES[x]), F32 if (M + K) % 2 else BF16)


def test_ties_zeros_and_small_values(bl):
    x = torch.zeros(4, 192, device="cuda")
    x[0, :64] = torch.arange(64, device="cuda") - 31.5  # scale 32.5 in the middle group's place
    x[0, 64:128] = (torch.arange(64, device="cuda") + 0.5) / 127 * 64
    x[0, 64] = 64.0                                     # quotients at half codes
    x[1, 3], x[1, 100] = 1e-7, -1e-9                    # below the least scale
    x[2] = 1e30
    check(bl, x)
    check(bl, x.bfloat16(), BF16)


def test_buffers_are_filled_and_nothing_else(bl):
    M, K = 13, 1001
    big = torch.full((M * K + 64,), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((M * gr.groups_of(K) + 16,), -1.0, device="cuda")
    x = torch.randn(M, K, device="cuda")
    kept = bl.Checkpoint(big[:M * K].view(M, K), scale[:M * gr.groups_of(K)].view(M, -1))
    assert bl.bitlinear_checkpoint(x, kept) is kept
    assert bool((big[M * K:] == 77).all()) and bool((scale[M * gr.groups_of(K):] == -1).all())
    codes, s = gr.quantised(x)
    assert torch.equal(kept.codes.cpu(), codes) and torch.equal(kept.scale.cpu(), s)


def test_empty(bl):
    kept = bl.bitlinear_checkpoint(torch.empty(0, 70, device="cuda"))
    assert kept.scale.shape == (0, 2) and bl.bitlinear_checkpoint_restore(kept).shape == (0, 70)


def test_the_largest_values(bl):
    """Up to the largest finite values of both types: 128 scale / 127 is past fp32's range.
    (127 fl(scale / 127) itself is, by its definition, where the quotient was rounded up from
    the last value, (2 - 2^-23) 2^127: codes of 127 in such a group alone may be infinite.)"""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = (torch.rand(5, 200, generator=g, device="cuda") * 2 - 1) * 3.4e38
    x[0, 3], x[1, 70] = torch.finfo(F32).max, -torch.finfo(F32).max
    codes, scale = gr.quantised(x)
    y = bl.bitlinear_checkpoint_restore(bl.Checkpoint(codes.cuda(), scale.cuda()))
    same = torch.equal(y.cpu(), gr.restored(codes, scale))
    last = (scale == torch.finfo(F32).max).repeat_interleave(64, 1)[:, :200] & (codes.abs() == 127)
    inside = bool((y.cpu().isfinite() | last).all())
    assert same and inside
    z = torch.full((2, 128), torch.finfo(BF16).max, device="cuda")
    z[1] = -z[1]
    kept = bl.Checkpoint(*(t.cuda() for t in gr.quantised(z)))
    y = bl.bitlinear_gated_backward(torch.full((1, 128), 2.0 ** -20, device="cuda"), kept, "relu").grad_z
    want = gr.restored(*gr.quantised(z))
    same = [torch.equal(y.cpu()[0, 128:], want[0] * 2.0 ** -20), torch.equal(y.cpu()[0, :128], want[1] * 2.0 ** -20)]
    assert all(same)
