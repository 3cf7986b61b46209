"""Column sums of the block norm's backward pass where a workgroup takes several
rows: rows added up in registers, the parameters fetched again for later rows, the
next row's loads in flight, and runs of up to 512 rows, for every form of the
kernels (one and two chunks per thread, whole and ragged widths, other rows)."""
import pytest
import torch

import operators_ref as ref
from test_gpu_block_norm import BF16, Case, backward64, bl, check_backward, run_backward  # noqa: F401

pytestmark = pytest.mark.gpu

FUSED_MAX_K, SUMS = 8192, 4


def partials(bl, M, K):
    """Rows of partial sums in the workspace: [partials][4][K] floats, after two
    floats per row where the rows are not held in registers."""
    floats = bl.bitlinear_block_norm_backward_workspace_bytes(M, K) // 4
    if not 8 <= K <= FUSED_MAX_K:
        floats -= 2 * M
    assert floats % (SUMS * K) == 0
    return floats // (SUMS * K)


def check_rows_count(c, runs, want, tol):
    """The bound is narrow enough to see rows that are not added: the sums without
    all rows but the last of each run are beyond it almost everywhere."""
    x = c.stored.double()
    mean, r = ref.stats64(x, c.pre["kind"], c.pre["eps"])
    terms = c.Gn.double() * (x - mean) * r
    last = torch.arange(1, runs + 1) * c.M // runs - 1
    lost = want["grad_pre_weight"].detach() - terms[last].sum(0)
    seen = lost.abs() > 4 * tol["grad_pre_weight"] + 2 ** -20 * want["grad_pre_weight"].abs()
    assert seen.double().mean() > 0.5


def check(bl, c, gn, at_least):
    print(f"[case] block norm backward, rows: M={c.M} K={c.K}", flush=True)
    runs = partials(bl, c.M, c.K)
    assert c.M >= at_least * runs, "several rows in a run"
    r = run_backward(c, gn)
    check_backward(c, r)
    check_rows_count(c, runs, *backward64(c))


FORMS = [("layer", "token", True, BF16), ("layer", "channel", True, torch.float32),
         ("rms", "channel", False, torch.float32), ("rms", "token", False, BF16)]


@pytest.mark.parametrize("M,K", [(6000, 9), (5000, 264), (3000, 1001), (1100, 2048), (1100, 4096), (1100, 5001),
                                 (1100, 8185), (1100, 8192)])
@pytest.mark.parametrize("kind,gate,bias,gn", FORMS)
def test_runs_of_rows(bl, M, K, kind, gate, bias, gn):
    check(bl, Case(bl, M, K, "f32", "bf16", pre=kind, post=kind, gate=gate, bias=bias, scale=0.75, seed=M + K), gn, 2)


@pytest.mark.parametrize("M,K", [(600, 5), (1500, 1), (600, 8200), (600, 11008)])
@pytest.mark.parametrize("kind,gate,bias,gn", FORMS)
def test_chunks_of_rows(bl, M, K, kind, gate, bias, gn):
    c = Case(bl, M, K, "f32", "bf16", pre=kind, post=kind, gate=gate, bias=bias, scale=0.75, seed=M + K)
    if K == 1 and kind == "layer":  # a LayerNorm of one element is its bias: no gradient to see rows by
        check_backward(c, run_backward(c, gn))
        return
    check(bl, c, gn, 2)


@pytest.mark.parametrize("K", [5, 8])
def test_longest_runs(bl, K):
    """More rows than 2048 runs of 512: the runs stay at 512 rows and their number grows."""
    M = (1 << 20) + 300
    assert partials(bl, M, K) == (M + 511) // 512
    c = Case(bl, M, K, "f32", "bf16", pre="layer", post="rms", gate="channel", bias=True, seed=K)
    check_backward(c, run_backward(c))


def test_uneven_types_and_rows(bl):
    """bf16 stream and parameters over several rows a run, whole and ragged."""
    for M, K in ((1100, 4104), (2100, 1999)):
        check(bl, Case(bl, M, K, "bf16", "f32", "bf16", pre="rms", post="layer", gate="channel", bias=True, seed=K),
              torch.float32, 2)
