"""How far a kept value is from what it was kept of, by the definition that the kernels
follow bit for bit (gated_ref.quantised and restored; no GPU needed).

With u = 2^-24: x / s and its product with 127 are rounded, so what is rounded to a code is
off by at most 127 (2 u + u^2), and the code by that and a half; s / 127 and its product with
the code are rounded, at most s (2 u + u^2). In all s / 254 + (4 u + 2 u^2) s, which is less
than s / 254 + 2^-21 s."""
import torch

import gated_ref as gr


def errors(x):
    codes, scale = gr.quantised(x)
    s = scale.double().repeat_interleave(64, 1)[:, :x.shape[1]]
    return (gr.restored(codes, scale).double() - x.double()).abs(), s


def test_bound():
    g = torch.Generator().manual_seed(0)
    for power in (-30, -3, 0, 40, 120):
        x = torch.rand(20000, 64, generator=g) * 2.0 ** power * torch.rand(20000, 1, generator=g)
        err, s = errors(x)
        assert bool((err <= s / 254 + 2.0 ** -21 * s).all())


def test_half_a_code_alone_is_not_the_bound():
    """A quotient just past a half code that rounds down to it."""
    x = torch.tensor([[float.fromhex("0x1.0f783cp+0"), float.fromhex("0x1.019358p+0")]])
    err, s = errors(x)
    assert float(err[0, 1]) > float(s[0, 1]) / 254
    assert bool((err <= s / 254 + 2.0 ** -21 * s).all())


def test_ties():
    """Values at every half code of many scales, and their neighbours."""
    g = torch.Generator().manual_seed(1)
    s = (1 + torch.rand(4000, 1, generator=g))
    at = ((torch.arange(63) * 2 + 1.5) / 127)[None] * s
    for x in (at, torch.nextafter(at, 2 * at), torch.nextafter(at, 0 * at)):
        err, sc = errors(torch.cat([s, x], 1))
        assert bool((sc == s).all()) and bool((err <= sc / 254 + 2.0 ** -21 * sc).all())
