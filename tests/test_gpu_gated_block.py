"""A gated feed-forward sublayer forward and back with activations kept in 8 bits:
the operators run together, against 64-bit definitions, captured in a graph and
replayed, on two streams at once and on a given stream."""
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


class Block:
    """n = rms(h); y = h + down(act(gate(n)) up(n)), each product on INT8 codes."""

    def __init__(self, bl, M, K, F, layout="2bit", act="silu", seed=0):
        self.bl, self.M, self.K, self.F, self.layout, self.act = bl, M, K, F, layout, act
        self.up, self.down = Packed(bl, 0, [F, F], K, layout, seed), Packed(bl, 0, [K], F, layout, seed + 1)
        p = self.up
        self.h, self.gy, self.bias = p.rand(M, K), p.rand(M, K, scale=0.1), p.rand(2 * F, scale=0.1)
        self.norm = bl.Norm("rms", 1 + p.rand(K, scale=0.1))

    def forward(self):
        bl, u = self.bl, self.up
        a = bl.bitlinear_block_norm(self.h, pre=self.norm, quant=True, stats=True)
        g = bl.bitlinear_forward_gated(a.xq, a.scale, u.packed, u.gammas, self.F, self.K, self.layout, bias=self.bias,
                                       act=self.act, kept=True)
        uq, us = bl.bitlinear_quant_acts(g.y)
        y = bl.bitlinear_forward_epilogue(uq, us, self.down.packed, self.down.gammas, self.K, self.F, self.layout,
                                          residual=self.h)
        return {"xq": a.xq, "scale": a.scale, "stats": a.stats, "u": g.y, "codes": g.kept.codes, "code_scale": g.kept.scale,
                "uq": uq, "us": us, "y": y}

    def backward(self, f):
        bl, u, d = self.bl, self.up, self.down
        gu = bl.bitlinear_backward_input_segmented(self.gy, d.packed, d.gammas, self.K, self.F, self.layout)
        gw2 = bl.bitlinear_backward_weight_codes(self.gy, f["uq"], f["us"])
        g = bl.bitlinear_gated_backward(gu, bl.Checkpoint(f["codes"], f["code_scale"]), self.act)
        gn = bl.bitlinear_backward_input_segmented(g.grad_z, u.packed, u.gammas, [self.F, self.F], self.K, self.layout)
        gw1 = bl.bitlinear_backward_weight_codes(g.grad_z, f["xq"], f["scale"])
        n = bl.bitlinear_block_norm_backward(self.gy, gn, self.h, None, f["stats"], pre=self.norm)
        return {"gu": gu, "gw2": gw2, "grad_z": g.grad_z, "grad_bias": g.grad_bias, "gn": gn, "gw1": gw1,
                "grad_h": n.grad_h, "grad_norm": n.grad_pre_weight}

    def both(self):
        f = self.forward()
        return {**f, **self.backward(f)}


@pytest.mark.parametrize("M,K,F,layout,act", [(1, 128, 264, "2bit", "silu"), (16, 520, 1027, "base3", "relu2"),
                                              (300, 264, 520, "1bit", "gelu"), (2048, 256, 384, "2bit", "gelu_tanh")])
def test_block_forward_and_back(bl, M, K, F, layout, act):
    b = Block(bl, M, K, F, layout, act, seed=M)
    r = b.both()
    d = lambda t: t.detach().cpu().double()  # noqa: E731
    # from the codes that the block itself made: no code can fall on the other side
    W1, W2 = b.up.codes.double() * b.up.row_gamma[:, None], b.down.codes.double() * b.down.row_gamma[:, None]
    x64 = d(r["xq"]) * (d(r["scale"])[:, None] / 127)
    prod = x64 @ W1.t()
    z, tol = prod + d(b.bias), ref.U * (5 * prod.abs() + (prod + d(b.bias)).abs() * 1.01)
    ref.close(r["u"], gr.gated(z, act), gr.gated_tol(z, tol, act), "u")
    kept = gr.restored(r["codes"], r["code_scale"]).double().view(M, 2 * F)
    top = r["code_scale"].cpu().double().repeat_interleave(64, 1)[:, :F].reshape(M, 2 * F)
    assert bool(((kept - z).abs() <= top / 254 + tol + 6 * ref.U * top).all())
    u64 = d(r["uq"]) * (d(r["us"])[:, None] / 127)
    down = u64 @ W2.t()
    ref.close(r["y"], down + d(b.h), ref.U * (8 * down.abs() + 2 * d(b.h).abs() + (down + d(b.h)).abs()), "y")
    # back: the exact gradients with identity quantisers, at the kept pre-activations
    gy = d(b.gy)
    gu = gy @ W2
    gz = gr.gated_back(gu, kept, act)
    gn = gz @ W1
    h = d(b.h).requires_grad_(True)
    w = d(b.norm.weight).requires_grad_(True)
    ref.norm64(h, {"kind": "rms", "weight": w, "bias": None, "eps": 1e-5}).backward(gn)
    want = {"gu": gu, "gw2": gy.t() @ u64, "grad_z": gz, "grad_bias": gz.sum(0), "gn": gn, "gw1": gz.t() @ x64,
            "grad_h": gy + h.grad, "grad_norm": w.grad}
    for k, v in want.items():
        # fp32 chains over sums of up to 2F terms and three operators: a few hundred roundings of
        # 2^-24 relative to the norm, and fp16 pieces' 2^-22
        err = (d(r[k]) - v).norm() / v.norm()
        assert err <= 2 ** -15, (k, float(err))


def test_kept_activations_cost_little_accuracy(bl):
    """Gradients from kept pre-activations against those from exact ones: a kept value
    is off by at most 1/254 of its group's largest, and the two differ by what that
    makes of the definition, no more."""
    g = torch.Generator(device="cuda").manual_seed(1)
    z, gy = torch.randn(64, 2 * 512, generator=g, device="cuda"), torch.randn(64, 512, generator=g, device="cuda")
    kept = bl.bitlinear_checkpoint(z.view(128, 512))
    off = (gr.restored(*kept) - z.cpu().view(128, 512)).abs()
    assert bool((off <= kept.scale.cpu().repeat_interleave(64, 1) / 253.9).all())
    a, b = (bl.bitlinear_gated_backward(gy, t).grad_z.cpu().double() for t in (z, kept))
    want = gr.gated_back(gy.cpu().double(), gr.restored(*kept).double().view(64, -1), "silu")
    assert (b - want).norm() <= 2 ** -20 * want.norm()
    assert (a - b).norm() <= 2 ** -6 * a.norm()


def test_block_in_a_graph(bl):
    """Captured once, replayed on new inputs with eager work between: every replay
    equals the eager call, bit for bit."""
    b = Block(bl, 200, 512, 1032, seed=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.both()
    for rep in range(4):
        for i, t in enumerate((b.h, b.gy, b.bias)):
            t.copy_(torch.randn(t.shape, generator=torch.Generator(device="cuda").manual_seed(10 * rep + i), device="cuda"))
        want = {k: v.clone() for k, v in b.both().items()}
        for v in out.values():
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in want.items():
            assert torch.equal(out[k], v), (rep, k)
    del graph


def test_large_gradients_in_a_graph(bl):
    """The products that leave partial sums and largest values in a workspace, one
    workspace for both calls: replays equal the eager calls."""
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    M, K = 2048, 2048
    p = Packed(bl, 0, [4096, 4096], K, seed=3)
    gy, gy2, xq, scale = r(M, 2048), r(M, 8192), torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    bl.bitlinear_quant_acts(r(M, K), xq, scale)
    need = (bl.bitlinear_backward_weight_codes_workspace_bytes(M, 2048, K),
            bl.bitlinear_backward_input_segmented_workspace_bytes(M, 8192, K))
    assert need[0] > 8 * 2048 * K and need[1] > 8 * M * K  # partial sums, and largest values behind them
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    gw, gx = torch.empty(2048, K, device="cuda"), torch.empty(M, K, device="cuda")

    def run():
        bl.bitlinear_backward_weight_codes(gy, xq, scale, grad_w=gw, workspace=ws)
        bl.bitlinear_backward_input_segmented(gy2, p.packed, p.gammas, p.segs, K, grad_x=gx, workspace=ws)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for rep in range(4):
        gy.copy_(r(M, 2048) * 10.0 ** rep)
        gy2.copy_(r(M, 8192) * 10.0 ** -rep)
        run()
        want = gw.clone(), gx.clone()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gw, want[0]) and torch.equal(gx, want[1]), rep
    del graph


def test_two_streams_at_once(bl):
    jobs = [Block(bl, 300, 520, 1032, seed=i) for i in (1, 7)]
    want = [b.both() for b in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        got = []
        for b, st in zip(jobs, streams):
            with torch.cuda.stream(st):
                got.append(b.both())
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for k, v in w.items():
                assert torch.equal(g[k], v), k


def test_outputs_belong_to_the_given_stream(bl):
    """With `stream`, outputs and workspaces come from that stream's memory: results stay
    right while the current stream keeps freeing and refilling tensors of the same
    sizes."""
    M, N, K = 256, 1024, 1024
    p = Packed(bl, M, [512, 512], K, seed=4, x_dtype=F32)
    gy = p.rand(M, N)
    st = torch.cuda.Stream()

    def calls(**kw):
        f = bl.bitlinear_forward_gated(p.xq, p.scale, p.packed, p.gammas, 512, K, z=True, kept=True, **kw)
        l = bl.bitlinear_linear_gated(p.x[:3], p.packed, p.gammas, 512, **kw)
        q = bl.linear_gated(p.x, p.packed, p.gammas, 512, **kw)
        return [f.y, f.z, *f.kept, l.y, q.y, *bl.bitlinear_gated_backward(gy[:, :512].contiguous(), p.z_in, **kw),
                bl.bitlinear_checkpoint_restore(bl.bitlinear_checkpoint(gy, **kw), **kw),
                bl.bitlinear_backward_weight_codes(gy, p.xq, p.scale, **kw),
                bl.bitlinear_backward_input_segmented(gy, p.packed, p.gammas, p.segs, K, **kw)]

    p.z_in = p.rand(M, N)
    want = calls()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append(calls(stream=st))
        for n in {t.numel() * t.element_size() for t in want}:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for r in got:
        for i, (a, b) in enumerate(zip(r, want)):
            assert torch.equal(a, b), i


def test_linear_gated_picks_the_same_result(bl):
    """From unquantised x: one fused launch, or quantise then multiply, or with a
    checkpoint: the same bits."""
    for M in (1, 4, 5, 40):
        p = Packed(bl, M, [130, 130], 96, seed=M, x_dtype=BF16)
        want = bl.bitlinear_forward_gated(p.xq, p.scale, p.packed, p.gammas, 130, 96, act="gelu", z=True, out_dtype=BF16)
        for kw in ({}, {"kept": True}):
            got = bl.linear_gated(p.x, p.packed, p.gammas, 130, act="gelu", z=True, out_dtype=BF16, **kw)
            assert torch.equal(got.y, want.y) and torch.equal(got.z, want.z) and (got.kept is None) == (not kw)


def test_rows_behind_the_last_token_stay(bl):
    """Outputs are written for M tokens and nothing behind them, in every operator."""
    M, F, K = 37, 100, 96
    p = Packed(bl, M, [F, F], K, seed=6)
    gy = p.rand(M, F)

    def roomy(rows, cols, dtype):
        big = torch.full((rows * cols + 256,), 77, dtype=dtype, device="cuda")
        return big, big[:rows * cols].view(rows, cols)

    bufs = {n: roomy(*a) for n, a in {"y": (M, F, BF16), "z": (M, 2 * F, BF16), "codes": (2 * M, F, torch.int8),
                                      "cs": (2 * M, gr.groups_of(F), F32), "gz": (M, 2 * F, F32), "x": (2 * M, F, F32),
                                      "gx": (M, K, BF16), "gw": (2 * F, K, F32)}.items()}
    v = {n: b[1] for n, b in bufs.items()}
    kept = bl.Checkpoint(v["codes"], v["cs"])
    bl.bitlinear_forward_gated(p.xq, p.scale, p.packed, p.gammas, F, K, y=v["y"], z=v["z"], kept=kept)
    bl.bitlinear_gated_backward(gy, kept, grad_z=v["gz"])
    bl.bitlinear_checkpoint_restore(kept, y=v["x"])
    bl.bitlinear_backward_input_segmented(v["gz"], p.packed, p.gammas, [F, F], K, grad_x=v["gx"])
    bl.bitlinear_backward_weight_codes(v["gz"], p.xq, p.scale, grad_w=v["gw"])
    torch.cuda.synchronize()
    for n, (big, view) in bufs.items():
        assert bool((big[view.numel():] == 77).all()), n
        assert bool((view != 77).any()), n
