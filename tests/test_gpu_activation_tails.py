"""Relative accuracy of the smooth activations and their slopes where they decay
(z < -3), down to the end of fp32's normal range, in the decode and the tiled
kernels and in the epilogue's backward pass.

u = 2^-24; the hardware's exp2 and reciprocal are off by one unit in the last
place, 2 u. An exponent v formed with relative error k u makes k v u of relative
error in exp(-v):
  silu       z / (1 + e), e = exp2(-log2(e) z): the constant and a product, 2 |z|; exp2 2,
             the sum 1, the reciprocal 2, the product 1.
  gelu       z erfc(-z / sqrt 2) / 2 = z poly(t) g / 2: g's exponent, a constant and two
             products, 3 z^2 / 2, and exp2 2; the polynomial 8 (4.5e-7), t's 3 times the
             polynomial's slope (at most 2.7), three products.
  gelu_tanh  v = 1.596 |z| (1 + 0.0447 z^2): constants of 3 and 5, z^2, the fused sum and
             the product: 8 v; exp2, sum, reciprocal, product as in silu.
A slope is two terms of the value's error whose difference is at least 1 / 1.5 (silu),
1 / 1.3 (gelu), 1 / 1.25 (gelu_tanh) of their sum for z < -3, and a few products more."""
import math

import pytest
import torch

import operators_ref as ref
from test_gpu_epilogue import bl  # noqa: F401

pytestmark = pytest.mark.gpu

C = 2 * math.sqrt(2 / math.pi)
# the first z, the value's and the slope's relative bounds in u
TAILS = {"silu": (-86.0, lambda z: 2 * z.abs() + 8, lambda z: 2 * z.abs() + 12),
         "gelu": (-12.9, lambda z: 1.5 * z * z + 24, lambda z: 1.3 * (1.5 * z * z + 24)),
         "gelu_tanh": (-9.9, lambda z: 8 * C * z.abs() * (1 + 0.044715 * z * z) + 8,
                       lambda z: 10 * C * z.abs() * (1 + 0.044715 * z * z) + 20)}


def check(got, want, rel, what):
    got = got.cpu().double()
    lim = rel * ref.U * want.abs()
    assert torch.all(lim < want.abs() / 2), "a tail cut off at 0 would be beyond the bound"
    err = (got - want).abs()
    worst = float((err / lim).max())
    print(f"[case] {what}: {worst:.2f} of the bound", flush=True)
    assert worst <= 1, (what, worst)


@pytest.mark.parametrize("act", list(TAILS))
def test_tails(bl, act):
    first, value, slope = TAILS[act]
    N, K = 4096, 64
    z = torch.linspace(first, -3.0, N)
    z64 = z.double().expand(1, N)
    packed = torch.zeros((N, bl.bitlinear_packed_row_bytes(K)), dtype=torch.uint8, device="cuda")
    gammas = torch.ones(1, device="cuda")
    for M in (1, 16, 300):  # products of zeros: z is the bias
        xq = torch.zeros((M, K), dtype=torch.int8, device="cuda")
        y = bl.bitlinear_forward_epilogue(xq, torch.ones(M, device="cuda"), packed, gammas, N, K, bias=z.cuda(), act=act)
        check(y[M - 1:], ref.act64(z64, act), value(z64), f"{act} M={M}")
    for M in (1, 200):
        r = bl.bitlinear_epilogue_backward(torch.ones(M, N, device="cuda"), z.cuda().expand(M, N).contiguous(), act)
        check(r.grad_z[M - 1:], ref.slope64(z64, act), slope(z64) + 1, f"{act} slope M={M}")
