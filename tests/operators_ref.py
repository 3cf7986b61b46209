"""Plain 64-bit implementations of the operators around the product, on CPU
tensors, and the tolerances that go with them.

u = 2^-24 is fp32's half step, half_step(dtype) a type's own (bf16 2^-8...):
an output stored in a type may be off by half_step * |value| on top of the
fp32 error, which each function below bounds from the number of roundings."""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, tol, what):
    """|got - want| <= tol elementwise, plus the half step of got's own type."""
    got64, want = got.detach().cpu().double(), want.double()
    assert got64.shape == want.shape, (what, got64.shape, want.shape)
    assert torch.isfinite(got64).all(), f"{what}: not finite"
    tol = tol * torch.ones_like(want)
    lim = tol + half_step(got.dtype) * (want.abs() + tol)
    err = (got64 - want).abs()
    bad = err > lim
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float((err / lim.clamp(min=1e-300)).max()):.2f} times it, first at "
                           f"{bad.nonzero()[0].tolist()}")


# ---- activations -------------------------------------------------------------
def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "relu2":
        return z.clamp(min=0) ** 2
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "relu2":
        return 2 * z.clamp(min=0)
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def act_tol(z, act):
    """fp32 error of act(z) and act'(z) for an exact z.

    exp(-v) is one exp2 of a product rounded to fp32: relative error |v| u from
    the product, 3 u from the constant's, exp2's and the reciprocal's rounding;
    v is |z| (silu), z^2 / 2 (gelu), at most 1.6 |z| (1 + 0.045 z^2) (gelu_tanh,
    itself 4 u off). Times p (1 - p) or the Gauss tail, (|v| + 4) exp(-v / 2) stays
    below 4, so 16 u (1 + |z|) covers each, and the fit of erfc adds 4.3e-7 < 8 u
    relative. A derivative sums two such terms, times z: 64 u (1 + |z|)."""
    if act in ("none", "relu"):
        return 0.0 * z.abs(), 0.0 * z.abs()
    if act == "relu2":
        return U * z * z, U * z.abs()
    return 32 * U * (1 + z.abs()), 64 * U * (1 + z.abs())


# ---- norms --------------------------------------------------------------------
def stats64(x, kind, eps):
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros(x.shape[0], 1, dtype=torch.float64)
    if kind == "none":
        return mean, torch.ones_like(mean)
    return mean, ((x - mean) ** 2).mean(1, keepdim=True).add(eps).rsqrt()


def norm64(x, p):
    if p is None:
        return x
    mean, r = stats64(x, p["kind"], p["eps"])
    y = (x - mean) * r
    if p["weight"] is not None:
        y = y * p["weight"]
    return y + p["bias"] if p["bias"] is not None else y


def norm_tol(x, x_tol, p, sums):
    """Error of norm(x) in fp32 for an x that is itself off by x_tol (a row
    maximum): the mean and the variance are sums of K terms over which at most
    `sums` additions follow one another (sums u relative to the sum of absolute
    values); the mean's error counts like x's. x^ = (x - mu) rs is then off by
    rs (x_tol + mu's) and, through rs, by |x^| times the same relative error."""
    if p is None:
        return x_tol * torch.ones_like(x)
    mean, r = stats64(x, p["kind"], p["eps"])
    w = p["weight"].abs() if p["weight"] is not None else 1.0
    b = p["bias"].abs() if p["bias"] is not None else 0.0
    top = x.abs().amax(1, keepdim=True)
    mu_tol = (sums + 2) * U * top + x_tol if p["kind"] == "layer" else 0.0
    hat = (x - mean).abs() * r
    # the variance: sums u relative, and the centred values' own error twice
    rs_rel = (sums + 6) * U + 2 * r * (x_tol + mu_tol)
    return w * (r * (x_tol + mu_tol + 2 * U * top) + hat * (rs_rel + 4 * U)) + 2 * U * b


def block64(h, block, pre, post, gate, scale):
    if block is not None:
        p = norm64(block, post)
        h = scale * h + (p if gate is None else gate * p)
    return h, (norm64(h, pre) if pre is not None else None)


def block_tols(h, block, pre, post, gate, scale, sums=64):
    """fp32 error bounds of block64's two outputs (before their own rounding)."""
    if block is None:
        return torch.zeros_like(h), norm_tol(h, 0.0, pre, sums)
    p = norm64(block, post)
    tol = norm_tol(block, 0.0, post, sums)
    if gate is not None:
        tol, p = gate.abs() * tol + 2 * U * (gate * p).abs(), gate * p
    tol = tol + 2 * U * ((scale * h).abs() + p.abs())
    out = scale * h + p
    return tol, None if pre is None else norm_tol(out, tol.amax(1, keepdim=True), pre, sums)
