"""Gated feed-forward products and their backward pass against the 64-bit
definitions (gated_ref.py) over the batch sizes and shapes at which the dispatch
changes kernels, with every output and activation."""
import pytest
import torch

import gated_ref as gr
import operators_ref as ref
from gated_ref import BF16, F32, TYPES, Packed

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "relu2", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from ternary_weight_linear_bitlinear_amd import bitlinear
    return bitlinear


def check_kept(kept, z, tol):
    """Codes of z in fp32: a code is off by half a step of its scale, the scale by z's
    own error at the group's maximum; quotient, product and the value's two roundings
    are 6 u of it."""
    top = torch.stack([z[:, i:i + 64].abs().amax(1) for i in range(0, z.shape[1], 64)], 1)
    tt = torch.stack([tol[:, i:i + 64].amax(1) for i in range(0, z.shape[1], 64)], 1)
    ref.close(kept.scale, top.clamp(min=1e-6), tt, "kept scale")
    s = (top + tt).clamp(min=1e-6).repeat_interleave(64, 1)[:, :z.shape[1]]
    err = (gr.restored(kept.codes, kept.scale).double() - z).abs()
    assert bool((err <= s / 254 + tol + 6 * ref.U * s).all())


# (given, M, F, K, layout): fused decode (one token, streamed tiles, two and four row
# groups, several rounds), decode batches of one and several chunks with one to three
# row groups, each tiled kernel with its ends, ragged and short rows
SHAPES = [
    ("x", 1, 2048, 4096, "2bit"), ("x", 1, 5504, 4096, "base3"), ("x", 1, 8200, 512, "1bit"), ("x", 1, 100, 9000, "2bit"),
    ("x", 1, 1, 1, "2bit"), ("x", 2, 17, 33, "base3"), ("x", 4, 4200, 1024, "2bit"), ("x", 3, 8200, 256, "1bit"),
    ("x", 4, 16400, 128, "base3"), ("x", 2, 1000, 777, "1bit"),
    ("codes", 1, 4096, 4096, "2bit"), ("codes", 3, 8200, 256, "base3"), ("codes", 16, 2000, 4096, "base3"),
    ("codes", 16, 5504, 1024, "2bit"), ("codes", 13, 10000, 520, "2bit"), ("codes", 9, 7, 100, "1bit"),
    ("codes", 40, 2048, 2048, "2bit"), ("codes", 47, 33, 100, "base3"), ("codes", 33, 10000, 256, "1bit"),
    ("codes", 200, 1003, 3000, "1bit"), ("codes", 200, 1000, 3000, "base3"), ("codes", 130, 1024, 2001, "2bit"),
    ("codes", 256, 4096, 1024, "2bit"), ("codes", 512, 5504, 512, "base3"), ("codes", 500, 4096, 512, "2bit"),
    ("codes", 300, 2048, 8192, "2bit"), ("codes", 700, 64, 8320, "base3"), ("codes", 1024, 8192, 256, "1bit"),
    ("codes", 2048, 5504, 256, "2bit"), ("codes", 2000, 5510, 320, "2bit"), ("codes", 2048, 5504, 320, "base3"),
    ("codes", 17, 3, 20, "2bit"), ("codes", 300, 1, 5, "base3"),
]


@pytest.mark.parametrize("given,M,F,K,layout", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_forward(bl, given, M, F, K, layout, out):
    i = SHAPES.index((given, M, F, K, layout)) + (out == "bf16")
    act = ACTS[i % 6]
    p = Packed(bl, M, [F, F], K, layout, seed=i, x_dtype=F32 if i % 3 == 0 else BF16)
    bias = None if i % 4 == 0 else p.rand(2 * F, dtype=F32 if i % 4 == 1 else BF16, scale=0.3)
    more = {"bias": bias, "act": act, "out_dtype": TYPES[out]}
    run = (lambda **kw: bl.bitlinear_linear_gated(p.x, p.packed, p.gammas, F, layout, **more, **kw)) if given == "x" \
        else (lambda **kw: bl.bitlinear_forward_gated(p.xq, p.scale, p.packed, p.gammas, F, K, layout, **more, **kw))
    r = run(z=True)
    z, tol = p.z(bias)
    ref.close(r.z, z, tol, "z")
    ref.close(r.y, gr.gated(z, act), gr.gated_tol(z, tol, act), "y")
    plain = run()
    assert plain.z is None and plain.kept is None and torch.equal(plain.y, r.y)
    if given == "codes":
        k = run(kept=True, z=True)
        check_kept(k.kept, z.view(2 * M, F), tol.view(2 * M, F))
        # sums are exact and what follows them is the same on every path
        assert torch.equal(k.y, r.y) and torch.equal(k.z, r.z)
        if out == "f32":
            same = bl.bitlinear_checkpoint(k.z.view(2 * M, F))
            assert torch.equal(k.kept.codes, same.codes) and torch.equal(k.kept.scale, same.scale)


BACK = [(1, 1), (1, 8), (5, 7), (128, 64), (100, 1003), (129, 72), (33, 5000), (700, 256), (1100, 1027), (2048, 130),
        (600, 11008), (257, 15)]


@pytest.mark.parametrize("M,F", BACK)
@pytest.mark.parametrize("z_type", ["f32", "bf16", "8bit"])
def test_backward(bl, M, F, z_type):
    i = BACK.index((M, F)) + {"f32": 0, "bf16": 1, "8bit": 2}[z_type]
    act, gy, gz = ACTS[i % 6], [F32, BF16][i % 2], [F32, BF16][i // 2 % 2]
    g = torch.Generator(device="cuda").manual_seed(i)
    z = torch.randn(M, 2 * F, generator=g, device="cuda") * 3
    grad_y = torch.randn(M, F, generator=g, device="cuda").to(gy)
    if z_type == "8bit":
        given = bl.bitlinear_checkpoint(z.view(2 * M, F))
        z64 = gr.restored(*given).double().view(M, 2 * F)
    else:
        given = z.to(TYPES[z_type])
        z64 = given.cpu().double()
    r = bl.bitlinear_gated_backward(grad_y, given, act, out_dtype=gz)
    want, tol = gr.gated_back(grad_y.cpu().double(), z64, act), gr.gated_back_tol(grad_y.cpu().double(), z64, act)
    assert r.grad_z.dtype is gz
    ref.close(r.grad_z, want, tol, "grad_z")
    ref.close(r.grad_bias, want.sum(0), gr.column_tol(want, tol), "grad_bias")
    only = bl.bitlinear_gated_backward(grad_y, given, act, grad_z=None)
    assert only.grad_z is None and torch.equal(only.grad_bias, r.grad_bias)
    assert bl.bitlinear_gated_backward(grad_y, given, act, out_dtype=gz, grad_bias=None).grad_z.equal(r.grad_z)


@pytest.mark.parametrize("act", ACTS)
def test_backward_is_the_derivative(bl, act):
    """Against differences of the 64-bit forward: central, step h, error h^2 / 6 times
    the third derivative (at most 8 times the values here) and 2^-50 / h of rounding."""
    g = torch.Generator(device="cuda").manual_seed(4)
    z = (torch.randn(6, 2 * 70, generator=g, device="cuda") * 2).double()
    z[z.abs() < 0.05] = 0.05  # away from relu's corner
    z = z.float()
    grad_y = torch.randn(6, 70, generator=g, device="cuda")
    got = bl.bitlinear_gated_backward(grad_y, z, act).grad_z.cpu().double()
    z64, gy, h = z.cpu().double(), grad_y.cpu().double(), 1e-4
    tol = gr.gated_back_tol(gy, z64, act)
    for half in range(2):
        d = torch.zeros_like(z64)
        d[:, half * 70:(half + 1) * 70] = h
        want = gy * (gr.gated(z64 + d, act) - gr.gated(z64 - d, act)) / (2 * h)
        lim = tol[:, half * 70:(half + 1) * 70] + 8 * h * h * (1 + z64.abs().max()) * gy.abs() + 1e-9
        assert bool(((got[:, half * 70:(half + 1) * 70] - want).abs() <= lim).all()), half


def test_extreme_preactivations(bl):
    """Far tails: act(z) z_1 and its slopes stay finite where the exponentials do not."""
    vals = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 80.0, -80.0, 300.0, -300.0, 1e4, -1e4], device="cuda")
    z = torch.cat([vals, torch.ones_like(vals)])[None].contiguous()
    gy = torch.ones(1, 10, device="cuda")
    for act in ACTS:
        r = bl.bitlinear_gated_backward(gy, z, act)
        want = gr.gated_back(gy.cpu().double(), z.cpu().double(), act)
        # (1e-30)^2 = 1e-60 lies below fp32's least normal value, 2^-126: whatever a value
        # there is rounded to, it is off by less than 2^-126
        tol = gr.gated_back_tol(gy.cpu().double(), z.cpu().double(), act) + 2.0 ** -126
        ref.close(r.grad_z, want, tol, act)


def test_empty(bl):
    p = Packed(bl, 0, [24, 24], 64)
    xq, scale = torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    assert bl.bitlinear_forward_gated(xq, scale, p.packed, p.gammas, 24, 64, kept=True).y.shape == (0, 24)
    r = bl.bitlinear_gated_backward(torch.empty(0, 24, device="cuda"), torch.empty(0, 48, device="cuda"))
    assert r.grad_z.shape == (0, 48) and not r.grad_bias.any()
