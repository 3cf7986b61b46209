"""The statistics that bitlinear_block_norm writes for its backward pass, against
64 bits, and the two passes in a chain with the forward pass's own statistics."""
import pytest
import torch

import operators_ref as ref
from test_gpu_block_norm import BF16, F32, Case, backward64, bl, bl_backward  # noqa: F401

pytestmark = pytest.mark.gpu

SUMS = 64  # additions that follow one another in a row's sum, as the other bounds count them


def stat_tols(x, x_tol, p):
    """Errors of a row's mean and (relative) 1 / deviation for an x off by x_tol:
    the mean's sum has SUMS u, the variance SUMS u and the centred values' own error
    (root mean square over the deviation, at most r times it)."""
    mean, r = ref.stats64(x, p["kind"], p["eps"])
    top = x.abs().amax(1, keepdim=True)
    mu_tol = (SUMS + 2) * ref.U * top + x_tol if p["kind"] == "layer" else torch.zeros_like(top)
    return mean, r, mu_tol, (SUMS + 6) * ref.U + 2 * r * (x_tol + mu_tol + ref.U * top)


def check_stats(c, st):
    h, b, pre, post, gate, scale = c.f64()
    out, _ = ref.block64(h, b, pre, post, gate, scale)
    out_tol = ref.block_tols(h, b, None, post, gate, scale)[0].amax(1, keepdim=True)
    for at, x, x_tol, p in ((0, b, 0.0, post), (2, out, out_tol, pre)):
        mean, rstd = st[:, at:at + 1], st[:, at + 1:at + 2]
        if p is None:
            assert torch.all(mean == 0) and torch.all(rstd == 1), at
            continue
        mean64, r64, mu_tol, rs_rel = stat_tols(x, x_tol, p)
        if p["kind"] == "rms":
            assert torch.all(mean == 0), at
        ref.close(mean, mean64, mu_tol, f"mean {at}")
        ref.close(rstd, r64, r64 * rs_rel, f"1 / deviation {at}")


@pytest.mark.parametrize("M,K", [(3, 5), (3, 8), (3, 520), (3, 1001), (3, 4096), (3, 5001), (600, 2048), (520, 5001),
                                 (3, 11008), (3, 16391), (3, 32768), (3, 33000)])
@pytest.mark.parametrize("pre,post", [("layer", "layer"), ("rms", "rms"), ("layer", "rms"), ("rms", "none"),
                                      ("none", "layer"), ("layer", "none")])
def test_stats(bl, M, K, pre, post):
    print(f"[case] block norm statistics M={M} K={K} {pre} {post}", flush=True)
    c = Case(bl, M, K, "f32", "bf16", pre=pre, post=post, gate="token", bias="layer" in (pre, post), scale=0.75,
             seed=M + K, shift=1.5)
    check_stats(c, c.call(stats=True).stats)


@pytest.mark.parametrize("K", [7, 4096, 5001, 33000])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_stats_without_block(bl, K, kind):
    c = Case(bl, 5, K, "bf16", "bf16", pre=kind, block=False, seed=K)
    check_stats(c, c.call(stats=True).stats)
    check_stats(c, c.call(stats=True, normed=False, quant=True).stats)


@pytest.mark.parametrize("M,K", [(9, 5), (9, 520), (9, 4096), (9, 5001), (600, 2048), (9, 8192), (9, 11008), (4, 33000)])
@pytest.mark.parametrize("kind,gate", [("layer", "channel"), ("layer", "token"), ("rms", "channel")])
def test_forward_and_back(bl, M, K, kind, gate):
    """The backward pass from the forward pass's own h_out and statistics. What their
    errors add to the gradients' bounds, to first order: x^ is off by e = r dm + |x^| dr
    for a mean off by dm and an r off by dr relative; J^T v = r (w v - mean(w v) - x^ mean(w v x^))
    by dr times its terms, r |x^| mean(|w v| e) and r e mean(|w v x^|); and d's error goes on
    into the block's side."""
    print(f"[case] block norm forward and back M={M} K={K} {kind} {gate}", flush=True)
    c = Case(bl, M, K, "f32", "bf16", pre=kind, post=kind, gate=gate, bias=kind == "layer", scale=0.75, seed=K)
    fwd = c.call(stats=True)
    c.stored = fwd.h_out.cpu()
    got = bl_backward(c, fwd.stats)
    want, tol = backward64(c)
    h, b, pre, post, gate64, scale = c.f64()
    x = c.stored.double()
    out_tol = (ref.block_tols(h, b, None, post, gate64, scale)[0] + ref.U * x.abs()).amax(1, keepdim=True)

    def side(x, x_tol, p, v, v_more):
        """(x^, its error, what the statistics and v's error add to J^T v)"""
        mean, r, dm, dr = stat_tols(x, x_tol, p)
        hat = ((x - mean) * r).abs()
        e = r * dm + hat * dr
        wv, wm = p["weight"].abs() * v.abs(), p["weight"].abs() * v_more
        layer = p["kind"] == "layer"
        m1, m2 = wv.mean(1, keepdim=True) * layer, (wv * hat).mean(1, keepdim=True)
        through = wm + wm.mean(1, keepdim=True) * layer + hat * (wm * hat).mean(1, keepdim=True)
        more = r * (dr * (wv + m1 + hat * m2) + hat * (wv * e).mean(1, keepdim=True) + e * m2 + through)
        return hat, e, more

    Gn, d = c.Gn.double(), (want["grad_h"] / scale).detach()
    _, e, d_more = side(x, out_tol, pre, Gn, torch.zeros_like(Gn))
    tol["grad_h"] = tol["grad_h"] + abs(scale) * d_more
    tol["grad_pre_weight"] = tol["grad_pre_weight"] + (Gn.abs() * e).sum(0)
    hat, e, b_more = side(b, 0.0, post, d * gate64, d_more * gate64.abs())
    tol["grad_block"] = tol["grad_block"] + b_more
    g, w = gate64.abs(), post["weight"].abs()
    tol["grad_post_weight"] = tol["grad_post_weight"] + (g * (d_more * hat + d.abs() * e)).sum(0)
    bias = post["bias"].abs() if post["bias"] is not None else 0.0
    gate_more = (d_more * hat + d.abs() * e) * w + d_more * bias
    tol["grad_gate"] = tol["grad_gate"] + (gate_more if gate == "token" else gate_more.sum(0))
    if kind == "layer":
        tol["grad_post_bias"] = tol["grad_post_bias"] + (g * d_more).sum(0)
    for k, v in want.items():
        ref.close(getattr(got, k), v, tol[k].detach(), k)
