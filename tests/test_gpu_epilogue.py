"""Products with bias, activation and residual in the epilogue, and that
epilogue's backward pass, against the 64-bit definitions (operators_ref.py) on
the exact INT32 sums, over the batch sizes and shapes at which the product
dispatch changes kernels."""
import pytest
import torch

import operators_ref as ref
from parity_util import guarded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}
ACTS = ["none", "relu", "relu2", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from ternary_weight_linear_bitlinear_amd import bitlinear
    return bitlinear


class Problem:
    """Codes, stacked packed weights of one or more segments, and the exact sums."""

    def __init__(self, bl, M, N, K, layout="2bit", segs=None, seed=0, x_dtype=BF16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.bl, self.M, self.N, self.K, self.layout = bl, M, N, K, layout
        self.segs = list(segs) if segs else [N]
        assert sum(self.segs) == N
        scheme = "binary" if layout == "1bit" else "ternary"
        rb = bl.bitlinear_packed_row_bytes(K, layout)
        self.packed = torch.empty((N, rb), dtype=torch.uint8, device="cuda")
        self.gammas = torch.empty(len(self.segs) + 3, dtype=F32, device="cuda")
        at = 0
        for i, n in enumerate(self.segs):
            W = torch.randn(n, K, generator=g, device="cuda") * 0.02 * (i + 1)
            p, gm = bl.bitlinear_pack_weights(W, layout, scheme)
            self.packed[at:at + n], self.gammas[i] = p, gm[0]
            at += n
        self.x = torch.randn(M, K, generator=g, device="cuda").to(x_dtype)
        self.xq, self.scale = bl.bitlinear_quant_acts(self.x)
        _, acc = bl.bitlinear_forward_segmented(self.xq, self.scale, self.packed, self.gammas, self.segs, K, layout,
                                                acc=True)
        gamma = torch.cat([self.gammas[i].cpu().double().expand(n) for i, n in enumerate(self.segs)])
        self.prod = acc.cpu().double() * gamma * (self.scale.cpu().double()[:, None] / 127)
        self.gen = g

    def rand(self, *shape, dtype=F32, scale=1.0):
        return (torch.randn(*shape, generator=self.gen, device="cuda") * scale).to(dtype)

    def check(self, y, z=None, bias=None, act="none", residual=None, scale=1.0):
        """z: the factor gamma scale / 127 takes three roundings, its product with
        the (exact) sum one, the bias addition one. y: act's slope (at most 1.13, or
        2 |z| for relu2) times that, act's own error, one rounding for the sum."""
        u = ref.U
        z64, z_tol = self.prod, 5 * u * self.prod.abs()
        if bias is not None:
            z64 = z64 + bias.cpu().double()
            z_tol = z_tol + u * (z64.abs() + z_tol)
        a_tol, _ = ref.act_tol(z64, act)
        y64 = ref.act64(z64, act)
        y_tol = (2 * z64.abs() + 1.0 if act == "relu2" else 1.13) * z_tol + a_tol
        if residual is not None:
            y64 = y64 + scale * residual.cpu().double()
            y_tol = y_tol + u * (y64.abs() + (scale * residual.cpu().double()).abs())
        if z is not None:
            ref.close(z, z64, z_tol, "z")
        ref.close(y, y64, y_tol, "y")


# the dispatch's branches: fused and separate decode (one token, streamed tiles,
# two and four row groups), 16-token chunks, each tiled kernel with its ends
SHAPES = [
    ("codes", 1, 4096, 4096, "2bit"), ("codes", 3, 1000, 777, "2bit"), ("codes", 4, 16400, 256, "1bit"),
    ("codes", 16, 4096, 11008, "base3"), ("codes", 16, 12288, 4096, "2bit"), ("codes", 13, 20000, 520, "2bit"),
    ("codes", 40, 4096, 4096, "2bit"), ("codes", 47, 33, 100, "base3"), ("codes", 33, 20000, 256, "1bit"),
    ("codes", 200, 2000, 3000, "2bit"), ("codes", 200, 2000, 3000, "base3"), ("codes", 200, 2001, 3001, "1bit"),
    ("codes", 256, 4096, 11008, "2bit"), ("codes", 512, 4096, 4096, "1bit"), ("codes", 512, 4096, 4096, "base3"),
    ("codes", 512, 12288, 4096, "2bit"), ("codes", 500, 12288, 512, "2bit"), ("codes", 700, 4100, 4096, "base3"),
    ("codes", 2048, 11008, 256, "2bit"), ("codes", 2048, 11008, 256, "1bit"), ("codes", 2048, 11008, 320, "base3"),
    ("codes", 2000, 11008, 128, "2bit"), ("codes", 1000, 11009, 130, "2bit"), ("codes", 4096, 4096, 256, "2bit"),
    ("codes", 4000, 4352, 384, "1bit"), ("codes", 300, 1000, 515, "2bit"), ("codes", 1100, 1003, 8200, "2bit"),
    ("x", 1, 4096, 4096, "2bit"), ("x", 1, 11008, 4096, "base3"), ("x", 1, 4096, 11008, "1bit"),
    ("x", 1, 33000, 520, "2bit"), ("x", 2, 16390, 512, "2bit"), ("x", 4, 33000, 512, "base3"),
    ("x", 3, 12000, 4096, "2bit"), ("x", 4, 1001, 1003, "base3"), ("x", 2, 5, 7, "1bit")]


def run(p, kind, **kw):
    if kind == "codes":
        return p.bl.bitlinear_forward_epilogue(p.xq, p.scale, p.packed, p.gammas, p.segs, p.K, p.layout, **kw)
    return p.bl.bitlinear_linear_epilogue(p.x, p.packed, p.gammas, p.segs, p.layout, **kw)


@pytest.mark.parametrize("kind,M,N,K,layout", SHAPES)
def test_everything_on(bl, kind, M, N, K, layout):
    """bias, gelu, a scaled residual and z, in both output types, one matrix and
    three stacked ones."""
    print(f"[case] epilogue {kind} M={M} N={N} K={K} {layout}", flush=True)
    for segs in (None, (N // 3 + 1, 1, N - N // 3 - 2)):
        if segs and min(segs) < 1:
            continue
        p = Problem(bl, M, N, K, layout, segs, seed=M + N)
        for out, b in ((F32, BF16), (BF16, F32)):
            bias, res = p.rand(N, dtype=b, scale=0.3), p.rand(M, N, dtype=out)
            y, gy = guarded((M, N), out)
            z, gz = guarded((M, N), out)
            got = run(p, kind, bias=bias, act="gelu", residual=res, residual_scale=0.75, y=y, z=z)
            assert got[0] is y and got[1] is z
            gy.check("y", all_written=False)
            gz.check("z", all_written=False)
            p.check(y, z, bias, "gelu", res, 0.75)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind,M,N,K", [("codes", 5, 260, 520), ("codes", 300, 1000, 520), ("x", 2, 260, 520),
                                        ("codes", 512, 12288, 128)])
@pytest.mark.parametrize("out", list(TYPES))
def test_activations(bl, act, kind, M, N, K, out):
    p = Problem(bl, M, N, K, seed=7)
    bias = p.rand(N, scale=4.0)
    y, z = run(p, kind, bias=bias, act=act, out_dtype=TYPES[out], z=True)
    p.check(y, z, bias, act)


@pytest.mark.parametrize("kind,M,N,K,layout", SHAPES)
def test_nothing_on_is_the_plain_product(bl, kind, M, N, K, layout):
    """Without bias, activation and residual the outputs are those of the plain
    product, bit for bit."""
    for out in (F32, BF16):
        p = Problem(bl, M, N, K, layout, seed=K)
        y = run(p, kind, out_dtype=out)
        if kind == "codes":
            want = bl.bitlinear_forward(p.xq, p.scale, p.packed, p.gammas, N, K, layout, out_dtype=out)
        else:
            want = bl.bitlinear_linear(p.x, p.packed, p.gammas, N, layout, out_dtype=out)
        assert torch.equal(y, want), out


@pytest.mark.parametrize("M,N,K", [(1, 512, 512), (16, 4096, 512), (100, 1000, 520), (512, 12288, 256),
                                   (2048, 11008, 128), (300, 1003, 515)])
@pytest.mark.parametrize("out", list(TYPES))
def test_residual_in_place(bl, M, N, K, out):
    p = Problem(bl, M, N, K, seed=5)
    bias, res = p.rand(N), p.rand(M, N, dtype=TYPES[out])
    want = run(p, "codes", bias=bias, residual=res)
    assert want.dtype == TYPES[out]
    y = res.clone()
    got = run(p, "codes", bias=bias, residual=y, y=y)
    assert got is y and torch.equal(y, want)


def test_linear_epilogue_picks_by_batch(bl):
    for M in (1, 4, 5, 70):
        p = Problem(bl, M, 300, 520, seed=M)
        bias = p.rand(300)
        y = bl.linear_epilogue(p.x, p.packed, p.gammas, 300, bias=bias, act="silu", out_dtype=BF16)
        p.check(y, None, bias, "silu")


def test_activation_tails(bl):
    """Each activation over z from -40 to 40 (and far beyond), through a bias on a
    product of zeros."""
    N = 20000
    p = Problem(bl, 2, N, 64, seed=1)
    xq = torch.zeros_like(p.xq)
    z = torch.cat([torch.linspace(-40, 40, N - 6), torch.tensor([-1e4, 1e4, -1e15, 1e15, 0.0, -0.0])]).cuda()
    p.prod = torch.zeros(2, N, dtype=torch.float64)
    for act in ACTS:
        keep = z.abs() <= (1e8 if act == "relu2" else 1e30)
        b = torch.where(keep, z, torch.zeros_like(z))
        y = bl.bitlinear_forward_epilogue(xq, p.scale, p.packed, p.gammas, N, 64, bias=b, act=act)
        p.check(y, None, b, act)
        g = torch.ones(2, N, device="cuda")
        r = bl.bitlinear_epilogue_backward(g, b.expand(2, N).contiguous(), act)
        z64 = b.cpu().double().expand(2, N)
        want = ref.slope64(z64, act)
        ref.close(r.grad_z, want, ref.act_tol(z64.clamp(-100, 100), act)[1] + 2 * ref.U * want.abs(), act)


# ---- backward of the epilogue -----------------------------------------------------
def check_backward(bl, M, N, act, gy, zt, gz, seed, **kw):
    g = torch.Generator().manual_seed(seed)
    grad_y = torch.randn(M, N, generator=g).to(TYPES[gy])
    z = (2 * torch.randn(M, N, generator=g)).to(TYPES[zt])
    r = bl.bitlinear_epilogue_backward(grad_y.cuda(), z.cuda(), act, residual_scale=0.625, out_dtype=TYPES[gz],
                                       grad_residual=True, **kw)
    assert r.grad_z.dtype == TYPES[gz] and r.grad_residual.dtype == TYPES[gy] and r.grad_bias.dtype == F32
    g64, z64 = grad_y.double(), z.double()
    want = g64 * ref.slope64(z64, act)
    tol = g64.abs() * ref.act_tol(z64, act)[1] + 2 * ref.U * want.abs()
    ref.close(r.grad_z, want, tol, "grad_z")
    # chunks of at most 512 terms in fp32, added in 64 bits
    ref.close(r.grad_bias, want.sum(0), (tol + (min(M, 512) + 4) * ref.U * want.abs()).sum(0), "grad_bias")
    ref.close(r.grad_residual, 0.625 * g64, ref.U * g64.abs(), "grad_residual")
    return r


@pytest.mark.parametrize("M,N", [(1, 1), (1, 4096), (2, 3), (5, 8), (16, 255), (17, 1000), (64, 1003), (513, 4096),
                                 (1030, 264), (2048, 11008), (5000, 24)])
@pytest.mark.parametrize("act", ACTS)
def test_backward_shapes(bl, M, N, act):
    print(f"[case] epilogue backward M={M} N={N} {act}", flush=True)
    check_backward(bl, M, N, act, "f32", "bf16", "bf16", M + N)


@pytest.mark.parametrize("gy,zt,gz", [(a, b, c) for a in TYPES for b in TYPES for c in TYPES])
@pytest.mark.parametrize("N", [1000, 1001])
def test_backward_types(bl, gy, zt, gz, N):
    check_backward(bl, 90, N, "gelu_tanh", gy, zt, gz, 3)


def test_backward_parts(bl):
    """Each output alone, none without its buffer, and z left out for a plain sum."""
    g = torch.Generator(device="cuda").manual_seed(2)
    gy = torch.randn(300, 1000, generator=g, device="cuda")
    z = torch.randn(300, 1000, generator=g, device="cuda")
    full = bl.bitlinear_epilogue_backward(gy, z, "silu", 0.5, grad_residual=True)
    a = bl.bitlinear_epilogue_backward(gy, z, "silu", grad_z=None)
    assert a.grad_z is None and a.grad_residual is None and torch.equal(a.grad_bias, full.grad_bias)
    b = bl.bitlinear_epilogue_backward(gy, z, "silu", grad_bias=None)
    assert b.grad_bias is None and torch.equal(b.grad_z, full.grad_z)
    c = bl.bitlinear_epilogue_backward(gy, None, residual_scale=0.5, grad_z=None, grad_bias=None, grad_residual=True)
    assert torch.equal(c.grad_residual, full.grad_residual) and torch.equal(c.grad_residual, 0.5 * gy)
    d = bl.bitlinear_epilogue_backward(gy, None, grad_z=None)
    assert (d.grad_bias.double() - gy.double().sum(0)).abs().max() <= 304 * ref.U * gy.double().abs().sum(0).max()
    need = bl.bitlinear_epilogue_backward_workspace_bytes(300, 1000)
    ws, wg = guarded((need,), torch.uint8)
    gz, zg = guarded((300, 1000), BF16)
    gb, bg = guarded((1000,), F32)
    e = bl.bitlinear_epilogue_backward(gy, z, "silu", workspace=ws, grad_z=gz, grad_bias=gb)
    assert torch.equal(e.grad_bias, full.grad_bias) and torch.equal(gz, full.grad_z.to(BF16))
    for guard in (wg, zg, bg):
        guard.check("output", all_written=False)


def test_backward_empty(bl):
    e = torch.empty((0, 40), device="cuda")
    b = torch.full((40,), 3.0, device="cuda")
    bl.bitlinear_epilogue_backward(e, e, "relu", grad_bias=b)
    assert torch.all(b == 0)
    r = bl.bitlinear_epilogue_backward(torch.empty((5, 0), device="cuda"), None)
    assert r.grad_z.shape == (5, 0)


def test_backward_against_differences(bl):
    """grad_z against the central difference of the 64-bit activation (step 1e-6)."""
    g = torch.Generator().manual_seed(4)
    z = 2 * torch.randn(64, 100, generator=g)
    gy = torch.randn(64, 100, generator=g)
    for act in ACTS:
        r = bl.bitlinear_epilogue_backward(gy.cuda(), z.cuda(), act)
        h = 1e-6
        slope = (ref.act64(z.double() + h, act) - ref.act64(z.double() - h, act)) / (2 * h)
        smooth = z.abs() > 2 * h  # (relu's corner)
        err = (r.grad_z.cpu().double() - gy.double() * slope).abs()
        assert (err[smooth] <= 1e-5 * (1 + z.abs().double())[smooth] * gy.abs().double()[smooth]).all(), act


def test_offsets_past_32_bits(bl):
    """Output rows that begin past element 2^31, forward and back."""
    M, N, K = 270000, 8192, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    p = Problem(bl, 64, N, K, seed=3)
    xq = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    scale = torch.ones(M, device="cuda")
    rows = torch.tensor([0, 262143, 262144, 262145, M - 1], device="cuda")
    xq[rows] = p.xq[:5]
    res = torch.full((M, N), 0.5, dtype=BF16, device="cuda")
    res[rows] = torch.randn(5, N, generator=g, device="cuda").to(BF16)
    bias = p.rand(N)
    more = dict(bias=bias, act="gelu", out_dtype=BF16)
    y, z = bl.bitlinear_forward_epilogue(xq, scale, p.packed, p.gammas, N, K, residual=res, z=True, **more)
    # the same rows among other ones, through the same tiled kernels
    few = torch.zeros((512, K), dtype=torch.int8, device="cuda")
    few[:5] = p.xq[:5]
    some = torch.full((512, N), 0.5, dtype=BF16, device="cuda")
    some[:5] = res[rows]
    y2, z2 = bl.bitlinear_forward_epilogue(few, scale[:512], p.packed, p.gammas, N, K, residual=some, z=True, **more)
    assert torch.equal(y[rows], y2[:5]) and torch.equal(z[rows], z2[:5])
    del y
    r = bl.bitlinear_epilogue_backward(res, z, "gelu", grad_bias=None)
    r2 = bl.bitlinear_epilogue_backward(res[rows], z[rows], "gelu", grad_bias=None)
    assert torch.equal(r.grad_z[rows], r2.grad_z)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (1, 1003, 520), (1, 33000, 520), (2, 16390, 512), (4, 33000, 512),
                                   (3, 12000, 4096), (3, 12001, 512), (4, 1001, 1003), (2, 5, 7)])
@pytest.mark.parametrize("out", list(TYPES))
def test_fused_residual_in_place(bl, M, N, K, out):
    """residual == y in the fused products: one token and several, two and four row
    groups, streamed tiles (12000 rows and more of 16-byte K), widths that four does not divide."""
    print(f"[case] fused in place M={M} N={N} K={K} {out}", flush=True)
    p = Problem(bl, M, N, K, seed=6)
    bias, res = p.rand(N), p.rand(M, N, dtype=TYPES[out])
    want = run(p, "x", bias=bias, act="silu", residual=res, residual_scale=0.5)
    p.check(want, None, bias, "silu", res, 0.5)
    y, guard = guarded((M, N), TYPES[out])
    for _ in range(3):
        y.copy_(res)
        got = run(p, "x", bias=bias, act="silu", residual=y, residual_scale=0.5, y=y)
        assert got is y and torch.equal(y, want)
    guard.check("y", all_written=False)
