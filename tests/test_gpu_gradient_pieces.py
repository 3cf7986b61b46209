"""Weight gradients from INT8 codes and input gradients over stacks in problems of large
tiles, with values of any magnitude beside each other and gammas at the ends of fp32's
range.

A factor (grad_y, or grad_w's product with the token's scale) enters in pieces that hold it
to within max(4, P) u of its own magnitude, P factors being summed (u = 2^-24; grad_w in
bf16: to within 2^-11). The bounds count that, three roundings for each term that is not
zero, and no other value of the row: a single large one whose code is zero is nothing to
an output."""
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


def check_input(bl, p, grad_y, nonzero):
    got = bl.bitlinear_backward_input_segmented(grad_y, p.packed, p.gammas, p.segs, p.K, p.layout)
    v = grad_y.cpu().double() * p.row_gamma
    want, terms = v @ p.codes.double(), v.abs() @ p.codes.double().abs()
    # each segment's end and the last gamma: a ratio, its product, another
    n = max(4, sum(p.segs)) + 3 * nonzero + 3 * len(p.segs) + 6
    ref.close(got, want, n * U * terms, "grad_x")


def check_weight(bl, grad_y, xq, scale, out, nonzero):
    got = bl.bitlinear_backward_weight_codes(grad_y, xq, scale, out)
    v = grad_y.cpu().double() * (scale.cpu().double() / 127)[:, None]
    want, terms = v.t() @ xq.cpu().double(), v.abs().t() @ xq.cpu().double().abs()
    n = max(4, grad_y.shape[0]) + 3 * nonzero + 6
    rel = n * U if out is F32 else 2.0 ** -11 + (3 * nonzero + 6) * U
    ref.close(got, want, rel * terms, "grad_w")


# (large tiles: rows in whole pieces, rows at any element, shared by three workgroups)
STACKS = [([200, 400], 4100, 4112), ([301, 300], 4100, 4112), ([2000, 1000], 2100, 2056)]


@pytest.mark.parametrize("segs,M,K", STACKS)
@pytest.mark.parametrize("layout", ["2bit", "base3"])
@pytest.mark.parametrize("below", [0, 12, 20, 24, 30, 40, 90])
def test_input_beside_a_large_value(bl, segs, M, K, layout, below):
    """Nine values a row: eight of them 2^-below of the ninth, whose code is zero for a
    third of the outputs."""
    N = sum(segs)
    p = Packed(bl, 0, segs, K, layout, seed=below)
    grad_y = torch.zeros(M, N, device="cuda")
    at = torch.rand(M, N, generator=p.gen, device="cuda").topk(9, 1).indices
    v = p.rand(M, 9) + p.rand(M, 9).sign()
    v[:, 1:] *= 2.0 ** -below
    grad_y.scatter_(1, at, v)
    check_input(bl, p, grad_y, 9)


@pytest.mark.parametrize("segs,M,K", STACKS)
def test_input_one_value_a_row(bl, segs, M, K):
    """Each output is one product, to the roundings of its factors' last bits."""
    N = sum(segs)
    p = Packed(bl, 0, segs, K, seed=3, gammas=[0.013, 0.021])
    grad_y = torch.zeros(M, N, device="cuda")
    grad_y.scatter_(1, torch.randint(0, N, (M, 1), generator=p.gen, device="cuda"), p.rand(M, 1))
    got = bl.bitlinear_backward_input_segmented(grad_y, p.packed, p.gammas, segs, K)
    want = (grad_y.cpu().double() * p.row_gamma) @ p.codes.double()
    # pieces 4 u; a ratio, its product and gamma's
    ref.close(got, want, 8 * U * want.abs(), "grad_x")


@pytest.mark.parametrize("segs,M,K", STACKS)
def test_input_of_mixed_rows(bl, segs, M, K):
    """Rows of Gaussian values, zeros, one dominant value, and 60 powers of two, side by
    side in every tile."""
    N = sum(segs)
    p = Packed(bl, 0, segs, K, "2bit", seed=5)
    grad_y = p.rand(M, N)
    grad_y[1::5] = 0
    grad_y[2::5, 7] *= 1e8
    grad_y[3::5] *= torch.logspace(-9, 9, N, device="cuda")
    check_input(bl, p, grad_y, N)


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


WEIGHTS = [(512, 4096, 4112), (4096, 1024, 1040), (130, 3000, 3001)]


@pytest.mark.parametrize("M,N,K", WEIGHTS)
@pytest.mark.parametrize("gy", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("below", [0, 12, 20, 24, 30, 40, 90])
def test_weight_beside_a_large_value(bl, M, N, K, gy, out, below):
    """The same along the tokens: nine gradients a column, the largest token's codes zero
    for half of the outputs."""
    g = torch.Generator(device="cuda").manual_seed(below + M)
    at = torch.rand(N, M, generator=g, device="cuda").topk(9, 1).indices
    v = torch.randn(N, 9, generator=g, device="cuda")
    v = v + v.sign()
    v[:, 1:] *= 2.0 ** -below
    grad_y = torch.zeros(N, M, device="cuda").scatter_(1, at, v).t().contiguous().to(TYPES[gy])
    xq = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    xq[torch.rand(M, K, generator=g, device="cuda") < 0.5] = 0
    scale = 1 + torch.rand(M, generator=g, device="cuda")
    check_weight(bl, grad_y, xq, scale, TYPES[out], 9)


@pytest.mark.parametrize("M,N,K", WEIGHTS)
def test_weight_one_token_a_column(bl, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    grad_y = torch.zeros(M, N, device="cuda")
    grad_y.scatter_(0, torch.randint(0, M, (1, N), generator=g, device="cuda"),
                    torch.randn(1, N, generator=g, device="cuda"))
    xq, scale = bl.bitlinear_quant_acts(torch.randn(M, K, generator=g, device="cuda"))
    got = bl.bitlinear_backward_weight_codes(grad_y, xq, scale)
    v = grad_y.cpu().double() * (scale.cpu().double() / 127)[:, None]
    want = v.t() @ xq.cpu().double()
    # pieces 4 u; the quotient of the scale, its product with grad_y, the sum of the pieces
    ref.close(got, want, 8 * U * want.abs(), "grad_w")


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_weight_of_mixed_columns(bl, out):
    M, N, K = 512, 4096, 4112
    g = torch.Generator(device="cuda").manual_seed(9)
    grad_y = torch.randn(M, N, generator=g, device="cuda")
    grad_y[:, 1::5] = 0
    grad_y[7, 2::5] *= 1e10
    grad_y[:, 3::5] *= torch.logspace(-9, 9, M, device="cuda")[:, None]
    xq = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    xq[7, ::2] = 0
    xq[M // 3:, 5::7] = 0
    scale = 1 + torch.rand(M, generator=g, device="cuda")
    check_weight(bl, grad_y, xq, scale, TYPES[out], M)


def test_bf16_gradients_are_one_piece(bl):
    """Gradients stored in bf16 enter as they are, whatever stands beside them."""
    p = Packed(bl, 0, [200, 400], 4112, seed=2)
    grad_y = torch.zeros(4100, 600, device="cuda")
    at = torch.rand(4100, 600, generator=p.gen, device="cuda").topk(9, 1).indices
    v = p.rand(4100, 9)
    v[:, 1:] *= 2.0 ** -60
    check_input(bl, p, grad_y.scatter_(1, at, v).to(BF16), 9)


def test_a_graph_follows_the_values(bl):
    """Which pieces a tile takes is found from the values at every replay: a graph captured
    with values of one range gives, for others, what the eager calls give."""
    M, K, segs = 1024, 2048, [2048, 2048]
    p = Packed(bl, 0, segs, K, seed=4)
    xq, scale = bl.bitlinear_quant_acts(p.rand(M, K))
    gy = p.rand(M, sum(segs))
    spread = torch.logspace(-14, 0, sum(segs), device="cuda")[None] * torch.logspace(-14, 0, M, device="cuda")[:, None]
    ws = torch.empty(max(bl.bitlinear_backward_weight_codes_workspace_bytes(M, sum(segs), K),
                         bl.bitlinear_backward_input_segmented_workspace_bytes(M, sum(segs), K)),
                     dtype=torch.uint8, device="cuda")
    gw, gx = torch.empty(sum(segs), K, device="cuda"), torch.empty(M, K, device="cuda")

    def run():
        bl.bitlinear_backward_weight_codes(gy, xq, scale, grad_w=gw, workspace=ws)
        bl.bitlinear_backward_input_segmented(gy, p.packed, p.gammas, segs, K, grad_x=gx, workspace=ws)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for rep in range(6):
        g = p.rand(M, sum(segs))
        if rep % 3 == 1:
            g = g * spread
        elif rep % 3 == 2:  # half of the rows' tiles, half of the columns'
            g[:M // 2, :segs[0]] = (g * spread)[:M // 2, :segs[0]]
        gy.copy_(g)
        run()
        want = gw.clone(), gx.clone()
        gw.zero_()
        gx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gw, want[0]) and torch.equal(gx, want[1]), rep
    v = gy.cpu().double() * p.row_gamma
    ref.close(gx, v @ p.codes.double(), (4 * sum(segs) + 12) * U * (v.abs() @ p.codes.double().abs()), "grad_x")
