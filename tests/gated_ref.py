"""Plain 64-bit implementations of the gated feed-forward block's operators on CPU
tensors, their fp32 error bounds, and the packed problems that the tests share."""
import torch

import operators_ref as ref

U = ref.U
F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}
GROUP = 64


def groups_of(K):
    return -(-K // GROUP)


def quantised(x):
    """Codes and scales of a checkpoint of fp32 values: the quotient, its product with
    127 and the rounding (half to even) are fp32 by definition."""
    x = x.detach().cpu().float()
    codes = torch.zeros(x.shape, dtype=torch.int8)
    scale = torch.zeros(x.shape[0], groups_of(x.shape[1]))
    for g in range(scale.shape[1]):
        part = x[:, g * GROUP:(g + 1) * GROUP]
        s = part.abs().amax(1).clamp(min=1e-6)
        codes[:, g * GROUP:(g + 1) * GROUP] = (part / s[:, None] * 127).round().clamp(-127, 127).to(torch.int8)
        scale[:, g] = s
    return codes, scale


def restored(codes, scale):
    """What kept codes stand for: an fp32 product with the fp32 quotient scale / 127."""
    f = (scale.detach().cpu() / 127).repeat_interleave(GROUP, 1)[:, :codes.shape[1]]
    return codes.detach().cpu().float() * f


def gated(z, act):
    F = z.shape[1] // 2
    return ref.act64(z[:, :F], act) * z[:, F:]


def gated_tol(z, z_tol, act):
    """Error of act(z_0) z_1 in fp32 for a z that is off by z_tol: act's slope is at
    most 1.13 (2 |z| for relu2, over the interval), its own error act_tol's; the
    product's rounding is one more."""
    F = z.shape[1] // 2
    g, u, tg, tu = z[:, :F], z[:, F:], z_tol[:, :F], z_tol[:, F:]
    a = ref.act64(g, act)
    ta = (2 * (g.abs() + tg) if act == "relu2" else 1.13) * tg + ref.act_tol(g, act)[0]
    err = ta * (u.abs() + tu) + a.abs() * tu
    return err + U * ((a * u).abs() + err)


def gated_back(grad_y, z, act):
    F = z.shape[1] // 2
    return torch.cat([grad_y * z[:, F:] * ref.slope64(z[:, :F], act), grad_y * ref.act64(z[:, :F], act)], 1)


def gated_back_tol(grad_y, z, act):
    """Error of both in fp32 for exact operands: the value's and the slope's own
    (act_tol), and a rounding for each product, two and one."""
    F = z.shape[1] // 2
    ta, ts = ref.act_tol(z[:, :F], act)
    g, u = grad_y.abs(), z[:, F:].abs()
    want = gated_back(grad_y, z, act).abs()
    err = torch.cat([g * u * ts, g * ta], 1)
    return err + 2 * U * (want + err)


def column_tol(terms, tol):
    """Error of fp32 sums of terms (each off by tol) down the columns: at most 512 / 8
    additions in a thread's run and 32 threads' sums follow one another; the runs are
    added in fp64 and rounded once."""
    return tol.sum(0) + 98 * U * (terms.abs() + tol).sum(0)


class Packed:
    """A stack of packed matrices on the GPU, their codes and gammas on the CPU, and
    quantised tokens."""

    def __init__(self, bl, M, segs, K, layout="2bit", seed=0, x_dtype=BF16, gammas=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.bl, self.M, self.K, self.layout, self.segs, self.gen = bl, M, K, layout, list(segs), g
        N = sum(segs)
        scheme = "binary" if layout == "1bit" else "ternary"
        self.packed = torch.empty((N, bl.bitlinear_packed_row_bytes(K, layout)), dtype=torch.uint8, device="cuda")
        self.gammas = torch.empty(len(segs), dtype=F32, device="cuda")
        codes, at = [], 0
        for i, n in enumerate(segs):
            W = torch.randn(n, K, generator=g, device="cuda") * 0.02 * (i + 1)
            p, gm = bl.bitlinear_pack_weights(W, layout, scheme)
            self.packed[at:at + n], self.gammas[i] = p, gm[0]
            # (the quantiser's decision in fp32, as its own tests pin it)
            W64 = W.double()
            codes.append(torch.where(W64 > W64.mean().float(), 1, -1) if scheme == "binary" else
                         (W / (gm[0] + 1e-5)).round().clamp(-1, 1))
            at += n
        self.codes = torch.cat(codes).to(torch.int8).cpu()
        if gammas is not None:
            self.gammas.copy_(torch.tensor(gammas))
        self.row_gamma = torch.cat([self.gammas[i].cpu().double().expand(n) for i, n in enumerate(segs)])
        if M:
            self.x = torch.randn(M, K, generator=g, device="cuda").to(x_dtype)
            self.xq, self.scale = bl.bitlinear_quant_acts(self.x)

    def rand(self, *shape, dtype=F32, scale=1.0):
        return (torch.randn(*shape, generator=self.gen, device="cuda") * scale).to(dtype)

    def z(self, bias=None):
        """The pre-activations and their fp32 error: the factor gamma scale / 127 takes
        two roundings (three as one matrix), its product with the exact sum one, the
        bias one."""
        acc = self.xq.cpu().double() @ self.codes.double().t()
        z = acc * self.row_gamma * (self.scale.cpu().double()[:, None] / 127)
        tol = 5 * U * z.abs()
        if bias is not None:
            z = z + bias.cpu().double()
            tol = tol + U * (z.abs() + tol)
        return z, tol
