"""bitlinear_block_norm and its backward pass against the 64-bit definitions
(operators_ref.py), at the widths where the kernels change (rows held in
registers, longer rows, widths that no vector divides), over types, norms,
gates and layouts of the call."""
import pytest
import torch

import operators_ref as ref
from parity_util import guarded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from ternary_weight_linear_bitlinear_amd import bitlinear
    return bitlinear


def rand(g, *shape, scale=1.0, shift=0.0, dtype=F32):
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


class Case:
    """Inputs on the CPU (as stored), the same on the GPU, and in 64 bits."""

    def __init__(self, bl, M, K, h="f32", x="f32", p="f32", pre="rms", post="rms", gate="channel",
                 bias=False, weight=True, scale=1.0, block=True, seed=0, shift=0.3):
        g = torch.Generator().manual_seed(1000 + seed)
        self.M, self.K, self.scale, self.bl = M, K, scale, bl
        P = TYPES[p]
        self.h = rand(g, M, K, scale=1.5, shift=-0.2, dtype=TYPES[h])
        self.block = rand(g, M, K, scale=0.7, shift=shift, dtype=TYPES[x]) if block else None

        def norm(kind):
            if kind == "none":
                return None
            return {"kind": kind, "weight": rand(g, K, scale=0.2, shift=1.0, dtype=P) if weight else None,
                    "bias": rand(g, K, scale=0.2, dtype=P) if bias else None, "eps": 1e-5}

        self.pre = norm(pre)
        self.post = norm(post) if block else None
        self.gate = None
        if block and gate == "channel":
            self.gate = rand(g, K, scale=0.2, shift=0.6, dtype=P)
        elif block and gate == "token":
            self.gate = torch.sigmoid(rand(g, M, K)).to(TYPES[x])
        self.X = TYPES[x]
        # outer gradients
        self.G = rand(g, M, K, dtype=TYPES[h])
        self.Gn = rand(g, M, K)

    def dev(self, t):
        return None if t is None else t.cuda()

    def norm(self, p):
        return None if p is None else self.bl.Norm(p["kind"], self.dev(p["weight"]), self.dev(p["bias"]), p["eps"])

    def call(self, **kw):
        return self.bl.bitlinear_block_norm(self.dev(self.h), self.dev(self.block), pre=self.norm(self.pre),
                                            post=self.norm(self.post), gate=self.dev(self.gate),
                                            residual_scale=self.scale,
                                            **({} if self.block is not None else {"out_dtype": self.X}), **kw)

    def f64(self):
        d = lambda t: None if t is None else t.double()  # noqa: E731
        n = lambda p: None if p is None else dict(p, weight=d(p["weight"]), bias=d(p["bias"]))  # noqa: E731
        return d(self.h), d(self.block), n(self.pre), n(self.post), d(self.gate), self.scale


def check_forward(c, r):
    args = c.f64()
    h, n = ref.block64(*args)
    th, tn = ref.block_tols(*args)
    if c.block is not None:
        ref.close(r.h_out, h, th, "h_out")
    if c.pre is not None and r.n is not None:
        ref.close(r.n, n, tn, "n")
    return h, n


WIDTHS = [1, 3, 8, 63, 64, 65, 257, 520, 1000, 2048, 4095, 4096, 5001, 8192, 8200, 11008, 16384, 16391, 20000,
          32768, 33000, 70001]


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_forward_widths(bl, K, kind):
    print(f"[case] block norm K={K} {kind}", flush=True)
    c = Case(bl, 3, K, pre=kind, post=kind, bias=kind == "layer", seed=K)
    check_forward(c, c.call())


@pytest.mark.parametrize("h,x,p", [(h, x, p) for h in TYPES for x in TYPES for p in TYPES])
@pytest.mark.parametrize("M,K", [(1, 4096), (5, 1001), (40, 1536)])
def test_forward_types(bl, h, x, p, M, K):
    c = Case(bl, M, K, h, x, p, scale=1.25, seed=M)
    r = c.call()
    assert r.h_out.dtype == TYPES[h] and r.n.dtype == TYPES[x]
    check_forward(c, r)


@pytest.mark.parametrize("pre,post,gate,bias,weight", [
    ("rms", "none", "none", False, True), ("layer", "none", "channel", True, True),
    ("none", "rms", "token", False, True), ("rms", "layer", "token", True, True),
    ("layer", "rms", "none", True, True), ("none", "none", "channel", False, True),
    ("rms", "rms", "channel", True, False), ("layer", "layer", "token", False, False)])
@pytest.mark.parametrize("K", [777, 4096, 33000])
def test_forward_forms(bl, pre, post, gate, bias, weight, K):
    c = Case(bl, 4, K, "f32", "bf16", "f32", pre, post, gate, bias, weight, scale=0.5, seed=K + 1)
    check_forward(c, c.call())


@pytest.mark.parametrize("K", [5, 4096, 9001, 40000])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_forward_without_block(bl, K, kind):
    """norm_pre alone: h is not written and comes back as h_out."""
    c = Case(bl, 6, K, "f32", "bf16", pre=kind, bias=kind == "layer", block=False, seed=K)
    r = c.call()
    assert r.n.dtype == BF16
    check_forward(c, r)


@pytest.mark.parametrize("K", [1, 9, 520, 4096, 5001, 11008, 33000])
@pytest.mark.parametrize("pre,bias", [("rms", False), ("rms", True), ("layer", True)])
def test_codes_are_those_of_the_quantiser(bl, K, pre, bias):
    """xq and scale equal bitlinear_quant_acts of the fp32 n bit for bit, whatever
    type n is stored in, with or without n."""
    c = Case(bl, 7, K, "f32", "f32", pre=pre, bias=bias, seed=K + 3)
    r = c.call(quant=True)
    xq, scale = bl.bitlinear_quant_acts(r.n)
    assert torch.equal(r.xq, xq) and torch.equal(r.scale, scale)
    alone = c.call(quant=True, normed=False)
    assert alone.n is None and torch.equal(alone.xq, xq) and torch.equal(alone.scale, scale)
    b16 = Case(bl, 7, K, "f32", "bf16", pre=pre, bias=bias, seed=K + 3)
    wide = Case(bl, 7, K, "f32", "f32", pre=pre, bias=bias, seed=K + 3)
    wide.block = b16.block.float()
    a, b = b16.call(quant=True), wide.call(quant=True)
    assert torch.equal(a.xq, b.xq) and torch.equal(a.scale, b.scale)


def test_codes_of_a_zero_row(bl):
    c = Case(bl, 3, 4096, gate="none", seed=2)
    c.h[1] = 0
    c.block[1] = 0
    r = c.call(quant=True)
    assert torch.all(r.n[1] == 0) and torch.all(r.xq[1] == 0)
    assert r.scale[1].item() == torch.tensor(1e-6, dtype=F32).item()
    check_forward(c, r)


@pytest.mark.parametrize("K", [512, 4096, 40000])
def test_layer_norm_far_from_zero(bl, K):
    """The variance is that of centred values: a mean 1000 times the deviation
    loses no more than fp32's own spacing there (the bound's x_tol term)."""
    c = Case(bl, 4, K, pre="layer", post="layer", gate="none", bias=True, seed=9, shift=700.0)
    check_forward(c, c.call())


def test_in_place_and_guards(bl):
    for K in (1000, 1003, 4096, 33000):
        c = Case(bl, 5, K, "f32", "bf16", gate="token", seed=K)
        want = c.call(quant=True, stats=True)
        h = c.h.cuda()
        out = {k: guarded(s, t) for k, s, t in (("n", (5, K), BF16), ("xq", (5, K), torch.int8), ("scale", (5,), F32),
                                                ("stats", (5, 4), F32))}
        got = bl.bitlinear_block_norm(h, c.block.cuda(), pre=c.norm(c.pre), post=c.norm(c.post), gate=c.gate.cuda(),
                                      h_out=h, **{k: t for k, (t, _) in out.items()})
        assert got.h_out is h and torch.equal(h, want.h_out)
        for k, (t, guard) in out.items():
            assert torch.equal(t, getattr(want, k)), k
            guard.check(k, all_written=False)
        t, guard = guarded((5, K), F32)
        c.call(h_out=t)
        assert torch.equal(t, want.h_out)
        guard.check("h_out", all_written=False)


def test_offsets_past_32_bits(bl):
    """Rows that begin past element 2^31 and 2^32 equal the same rows alone."""
    M, K = 1050000, 4096
    h = torch.empty((M, K), dtype=BF16, device="cuda").fill_(0.5)
    b = torch.empty((M, K), dtype=BF16, device="cuda").fill_(-0.25)
    rows = [0, 524287, 524288, 524289, 1048575, 1048576, M - 1]
    g = torch.Generator(device="cuda").manual_seed(5)
    for r in rows:
        h[r] = torch.randn(K, generator=g, device="cuda").to(BF16)
        b[r] = torch.randn(K, generator=g, device="cuda").to(BF16)
    w = torch.rand(K, generator=g, device="cuda") + 0.5
    norm = bl.Norm("rms", w)
    big = bl.bitlinear_block_norm(h, b, pre=norm, post=norm, quant=True, stats=True)
    at = torch.tensor(rows, device="cuda")
    one = bl.bitlinear_block_norm(h[at], b[at], pre=norm, post=norm, quant=True, stats=True)
    for k in ("h_out", "n", "xq", "scale", "stats"):
        assert torch.equal(getattr(big, k)[at], getattr(one, k)), k
    del big
    gn = torch.full((M, K), 0.125, dtype=BF16, device="cuda")
    st = bl.bitlinear_block_norm(h, b, pre=norm, post=norm, normed=False, quant=True, stats=True).stats
    back = bl.bitlinear_block_norm_backward(None, gn, h, b, st, pre=norm, post=norm, params=False)
    some = bl.bitlinear_block_norm_backward(None, gn[at], h[at], b[at], st[at], pre=norm, post=norm, params=False)
    for k in ("grad_h", "grad_block"):
        assert torch.equal(getattr(back, k)[at], getattr(some, k)), k


def test_empty_batch(bl):
    w = torch.ones(64, device="cuda")
    e = torch.empty((0, 64), device="cuda")
    r = bl.bitlinear_block_norm(e, e, pre=bl.Norm("layer", w, w), post=bl.Norm("rms", w), gate=w, quant=True,
                                stats=True)
    assert r.n.shape == (0, 64) and r.scale.shape == (0,)
    out = {k: torch.full((64,), 7.0, device="cuda") for k in
           ("grad_gate", "grad_post_weight", "grad_pre_weight", "grad_pre_bias")}
    bl.bitlinear_block_norm_backward(e, e, e, e, r.stats, pre=bl.Norm("layer", w, w), post=bl.Norm("rms", w), gate=w,
                                     **out)
    for k, v in out.items():
        assert torch.all(v == 0), k


# ---- backward -------------------------------------------------------------------
def backward64(c):
    """Gradients by autograd in 64 bits at the stored h_out, and bounds of the
    fp32 errors: each row sum has `sums` u, and the terms of d, grad_block and
    the columns are counted as they are formed."""
    h, b, pre, post, gate, scale = c.f64()
    sums = 64
    out64 = c.stored.double()
    leaves = {}

    def leaf(name, t):
        if t is not None:
            leaves[name] = t.requires_grad_(True)

    x = out64.clone().requires_grad_(True)
    if pre is not None:
        leaf("grad_pre_weight", pre["weight"])
        leaf("grad_pre_bias", pre["bias"])
        ref.norm64(x, pre).backward(c.Gn.double())
        d = x.grad + c.G.double()
    else:
        d = c.G.double()
    want = {"grad_h": d if b is None else scale * d}
    if b is not None:
        b.requires_grad_(True)
        leaf("grad_gate", gate)
        if post is not None:
            leaf("grad_post_weight", post["weight"])
            leaf("grad_post_bias", post["bias"])
        p = ref.norm64(b, post)
        (p if gate is None else gate * p).backward(d)
        want["grad_block"] = b.grad
    want.update({k: v.grad for k, v in leaves.items()})

    # bounds
    det = lambda t: t.detach() if torch.is_tensor(t) else t  # noqa: E731
    tol, Gn, G = {}, c.Gn.double(), c.G.double()

    def through(v, v_tol, x, p):
        """J^T v of a norm: |rs| (|w v| + mean |w v| + |x^| mean |w v x^|), each sum with sums u, each
        product with 4 u, x^ itself off by 4 u (1 + |mu| rs) from the stored statistics."""
        if p is None:
            return v_tol
        mean, r = (t.detach() for t in ref.stats64(det(x), p["kind"], p["eps"]))
        w = det(p["weight"]).abs() if p["weight"] is not None else 1.0
        hat = ((det(x) - mean) * r).abs()
        hat_tol = 4 * ref.U * (hat + (mean * r).abs() + (det(x) * r).abs())
        wv, wt = w * v.abs(), w * v_tol + 2 * ref.U * w * v.abs()
        m1 = wv.mean(1, keepdim=True) * (p["kind"] == "layer")
        m2 = (wv * hat).mean(1, keepdim=True)
        t1 = wt.mean(1, keepdim=True) + sums * ref.U * m1
        t2 = (wt * hat + wv * hat_tol).mean(1, keepdim=True) + sums * ref.U * m2
        return r * (wt + t1 + hat * t2 + hat_tol * m2 + 6 * ref.U * (wv + m1 + hat * m2))

    d_tol = through(Gn, torch.zeros_like(Gn), out64, pre) if pre is not None else torch.zeros_like(G)
    d_tol = d_tol + 2 * ref.U * (d.abs() + G.abs())
    tol["grad_h"] = abs(scale) * d_tol + ref.U * want["grad_h"].abs()
    # columns: a chunk of at most 512 rows in fp32, the rest in 64 bits; M + 8 covers it
    col = lambda terms, t_tol: (t_tol + (min(c.M, 512) + 8) * ref.U * terms.abs()).sum(0)  # noqa: E731

    def hats(x, p):
        if p is None:
            return det(x), 0 * det(x)
        mean, r = (t.detach() for t in ref.stats64(det(x), p["kind"], p["eps"]))
        hat = (det(x) - mean) * r
        return hat, 4 * ref.U * (hat.abs() + (mean * r).abs() + (det(x) * r).abs())

    if pre is not None:
        hat, ht = hats(out64, pre)
        tol["grad_pre_weight"] = col(Gn * hat, Gn.abs() * ht)
        tol["grad_pre_bias"] = col(Gn, 0 * Gn)
    if b is not None:
        g = det(gate) if gate is not None else torch.ones(1, dtype=torch.float64)
        v, v_tol = d * g, d_tol * g.abs() + 2 * ref.U * (d * g).abs()
        tol["grad_block"] = through(v, v_tol, b, post)
        hat, ht = hats(b, post)
        tol["grad_post_weight"] = col(v * hat, v_tol * hat.abs() + v.abs() * ht) * (1 + 4 * ref.U)
        tol["grad_post_bias"] = col(v, v_tol)
        w = det(post["weight"]) if post is not None and post["weight"] is not None else 1.0
        bias = det(post["bias"]) if post is not None and post["bias"] is not None else 0.0
        if gate is not None and gate.dim() == 2:
            p = hat * w + bias
            tol["grad_gate"] = d_tol * p.abs() + d.abs() * ht * abs(w) + 8 * ref.U * d.abs() * (hat.abs() * abs(w) + abs(bias))
        elif gate is not None:
            tol["grad_gate"] = col(d * hat, d_tol * hat.abs() + d.abs() * ht) * abs(w) + col(d, d_tol) * abs(bias)
    return want, tol


def run_backward(c, Gn_dtype=F32, grad_out=True, **kw):
    c.Gn = c.Gn.to(Gn_dtype)
    fwd = c.call(stats=True)
    c.stored = fwd.h_out.cpu()
    # statistics of the stored rows, so that the definition is exactly that of h_out
    st = fwd.stats.clone()
    if c.pre is not None:
        mean, r = ref.stats64(c.stored.double(), c.pre["kind"], c.pre["eps"])
        st[:, 2], st[:, 3] = mean[:, 0].float().cuda(), r[:, 0].float().cuda()
    if c.post is not None:
        mean, r = ref.stats64(c.block.double(), c.post["kind"], c.post["eps"])
        # the forward call's own statistics: its fp32 sums
        assert (fwd.stats[:, 1].cpu().double() / r[:, 0] - 1).abs().max() < 128 * ref.U
    if not grad_out:
        c.G = torch.zeros_like(c.G)
    return bl_backward(c, st, grad_out, **kw)


def bl_backward(c, st, grad_out=True, **kw):
    return c.bl.bitlinear_block_norm_backward(
        c.G.cuda() if grad_out else None, c.Gn.cuda() if c.pre is not None else None, c.stored.cuda(),
        c.dev(c.block), st, pre=c.norm(c.pre), post=c.norm(c.post), gate=c.dev(c.gate), residual_scale=c.scale, **kw)


def check_backward(c, r):
    want, tol = backward64(c)
    for k, v in want.items():
        ref.close(getattr(r, k), v, tol[k], k)
    for k, v in r._asdict().items():
        assert (v is not None) == (k in want), k


@pytest.mark.parametrize("K", [1, 3, 8, 65, 520, 1000, 2048, 4096, 5001, 8192, 8200, 11008, 16384, 16391, 33000])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_backward_widths(bl, K, kind):
    print(f"[case] block norm backward K={K} {kind}", flush=True)
    c = Case(bl, 9, K, pre=kind, post=kind, bias=kind == "layer", seed=K)
    check_backward(c, run_backward(c))


@pytest.mark.parametrize("M", [1, 2, 17, 255, 600, 1500])
@pytest.mark.parametrize("gate", ["channel", "token", "none"])
def test_backward_rows(bl, M, gate):
    c = Case(bl, M, 264, "f32", "bf16", gate=gate, scale=0.75, seed=M)
    check_backward(c, run_backward(c))


@pytest.mark.parametrize("h,x,p,gn", [(h, x, p, g) for h in TYPES for x in TYPES for p in TYPES for g in TYPES])
def test_backward_types(bl, h, x, p, gn):
    c = Case(bl, 21, 1032, h, x, p, pre="layer", post="layer", gate="token", bias=True, scale=1.5, seed=4)
    check_backward(c, run_backward(c, TYPES[gn]))


@pytest.mark.parametrize("pre,post,gate,bias,weight,block", [
    ("rms", "none", "none", False, True, True), ("layer", "none", "channel", True, True, True),
    ("none", "rms", "token", False, True, True), ("rms", "layer", "channel", True, True, True),
    ("layer", "rms", "none", True, True, True), ("none", "none", "channel", False, True, True),
    ("none", "none", "token", False, True, True), ("rms", "rms", "channel", True, False, True),
    ("rms", "none", "none", False, True, False), ("layer", "none", "none", True, True, False)])
@pytest.mark.parametrize("K", [777, 4096, 33000])
def test_backward_forms(bl, pre, post, gate, bias, weight, block, K):
    c = Case(bl, 6, K, "f32", "bf16", "f32", pre, post, gate, bias, weight, scale=0.5, block=block, seed=K + 1)
    check_backward(c, run_backward(c, BF16))


def test_backward_without_outer_gradient(bl):
    c = Case(bl, 12, 1000, seed=3)
    check_backward(c, run_backward(c, grad_out=False))


def test_backward_writes_only_its_outputs(bl):
    for K in (1000, 1001, 4096, 20000):
        c = Case(bl, 20, K, "f32", "bf16", pre="layer", post="layer", bias=True, seed=K)
        r = run_backward(c)
        st = c.call(stats=True).stats
        want = bl_backward(c, st)
        out = {k: guarded(v.shape, v.dtype) for k, v in r._asdict().items() if v is not None}
        need = bl.bitlinear_block_norm_backward_workspace_bytes(20, K)
        ws, wg = guarded((need,), torch.uint8)
        got = bl_backward(c, st, workspace=ws, **{k: t for k, (t, _) in out.items()})
        wg.check("workspace", all_written=False)
        for k, (t, guard) in out.items():
            assert getattr(got, k) is t and torch.equal(t, getattr(want, k)), k
            guard.check(k, all_written=False)


def test_backward_leaves_out_what_is_not_asked_for(bl):
    c = Case(bl, 20, 1000, "f32", "bf16", seed=6)
    full = run_backward(c)
    st = c.call(stats=True).stats
    full, bare = bl_backward(c, st), bl_backward(c, st, params=False)
    assert bare.grad_gate is None and bare.grad_pre_weight is None and bare.grad_post_weight is None
    assert torch.equal(bare.grad_h, full.grad_h) and torch.equal(bare.grad_block, full.grad_block)
    only = torch.empty(1000, device="cuda")
    part = bl_backward(c, st, params=False, grad_gate=only)
    assert part.grad_gate is only and torch.equal(only, full.grad_gate)


def test_backward_is_the_same_each_time(bl):
    c = Case(bl, 700, 1024, "f32", "bf16", seed=8)
    a = run_backward(c)
    st = c.call(stats=True).stats
    a, b = bl_backward(c, st), bl_backward(c, st)
    for k in a._fields:
        if getattr(a, k) is not None:
            assert torch.equal(getattr(a, k), getattr(b, k)), k


def test_gradient_against_differences(bl):
    """sum(G h') + sum(Gn n) along a random direction of every input at once: the
    kernels' gradients times the direction against the central difference of the
    64-bit definition (step 1e-5: truncation and rounding below 1e-8 relative),
    within the gradients' own fp32 error, under 1e-5 of the sum of absolute terms."""
    c = Case(bl, 8, 200, pre="layer", post="rms", gate="channel", bias=True, scale=0.8, seed=11)
    r = run_backward(c)
    h, b, pre, post, gate, scale = c.f64()
    # the same point: h such that the stored h_out is h' exactly
    h = (c.stored.double() - gate * ref.norm64(b, post)) / scale
    g = torch.Generator().manual_seed(3)
    d = lambda t: torch.randn(t.shape, generator=g, dtype=torch.float64)  # noqa: E731
    dirs = {"grad_h": d(h), "grad_block": d(b), "grad_gate": d(gate), "grad_pre_weight": d(gate),
            "grad_pre_bias": d(gate), "grad_post_weight": d(gate), "grad_post_bias": d(gate)}

    def loss(t):
        q = lambda p, s: dict(p, weight=p["weight"] + t * dirs[f"grad_{s}_weight"], bias=p["bias"] + t * dirs[f"grad_{s}_bias"])  # noqa: E731
        o, n = ref.block64(h + t * dirs["grad_h"], b + t * dirs["grad_block"], q(pre, "pre"), q(post, "post"),
                           gate + t * dirs["grad_gate"], scale)
        return (c.G.double() * o).sum() + (c.Gn.double() * n).sum()

    step = 1e-5
    slope = (loss(step) - loss(-step)) / (2 * step)
    terms = torch.cat([(getattr(r, k).cpu().double() * v).reshape(-1) for k, v in dirs.items()])
    assert abs(terms.sum() - slope) <= 1e-5 * terms.abs().sum()


@pytest.mark.parametrize("K", [64, 1000, 2048, 4096, 5001, 8192, 11008])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_do_not_depend_on_the_batch(bl, K, kind):
    """A token's outputs, codes and statistics are the same bits alone, in a small
    batch and in one that takes the many-row launch shape."""
    c = Case(bl, 1024, K, "bf16", "bf16", pre=kind, post=kind, bias=kind == "layer", seed=K)
    big = c.call(quant=True, stats=True)
    for rows in (slice(0, 1), slice(5, 12), slice(0, 511)):
        part = Case.__new__(Case)
        part.__dict__.update(c.__dict__)
        part.h, part.block = c.h[rows], c.block[rows]
        r = part.call(quant=True, stats=True)
        for k in ("h_out", "n", "xq", "scale", "stats"):
            assert torch.equal(getattr(r, k), getattr(big, k)[rows]), (k, rows)


def test_more_rows_than_one_grid(bl):
    """2^26 + 5 rows of 8 (more than 2^32 threads at one workgroup per row), and
    2^24 rows of 4 backward: the rows around the launches' ends equal the same rows alone."""
    M, K = (1 << 26) + 5, 8
    h = torch.full((M, K), 0.5, dtype=BF16, device="cuda")
    rows = torch.tensor([0, (1 << 21) - 1, 1 << 21, (1 << 26) - 1, 1 << 26, M - 1], device="cuda")
    h[rows] = torch.randn(len(rows), K, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF16)
    w = torch.linspace(0.5, 1.5, K, device="cuda")
    big = bl.bitlinear_block_norm(h, pre=bl.Norm("rms", w)).n
    assert torch.equal(big[rows], bl.bitlinear_block_norm(h[rows], pre=bl.Norm("rms", w)).n)
    assert torch.equal(big[1000], bl.bitlinear_block_norm(h[1000:1001], pre=bl.Norm("rms", w)).n[0])
    del big, h
    M, K = 1 << 24, 4
    h = torch.full((M, K), 0.5, device="cuda")
    rows = torch.tensor([0, (1 << 21) - 1, 1 << 21, M - 1], device="cuda")
    h[rows] = torch.randn(len(rows), K, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    norm = bl.Norm("rms", w[:K].contiguous())
    st = bl.bitlinear_block_norm(h, pre=norm, stats=True).stats
    big = bl.bitlinear_block_norm_backward(h, h, h, None, st, pre=norm).grad_h
    assert torch.equal(big[rows], bl.bitlinear_block_norm_backward(h[rows], h[rows], h[rows], None, st[rows],
                                                                   pre=norm).grad_h)


@pytest.mark.parametrize("K", [4104, 6000, 6001, 8185])
@pytest.mark.parametrize("kind,gate", [("layer", "token"), ("layer", "channel"), ("rms", "token")])
def test_backward_two_chunks(bl, K, kind, gate):
    """Rows of two chunks per thread, whose parameters lie in LDS."""
    c = Case(bl, 7, K, "f32", "bf16", pre=kind, post=kind, gate=gate, bias=kind == "layer", scale=0.5, seed=K)
    check_backward(c, run_backward(c, BF16))
