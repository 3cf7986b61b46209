"""Backward pass of the products' epilogue over many rows: widths that eight does
not divide, the last workgroup with fewer columns than one piece, fewer than
eight columns over several runs, and runs of up to 512 rows."""
import pytest
import torch

from parity_util import guarded
from test_gpu_epilogue import ACTS, TYPES, bl, check_backward  # noqa: F401

pytestmark = pytest.mark.gpu

# 257 and 1025: the last workgroup of 256 columns owns one; 263: seven; 1003, 5001: 235 and 137
SHAPES = [(513, 1003), (300, 257), (1030, 263), (2048, 5001), (130, 1025), (700, 5), (129, 1), (5000, 7)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_backward_many_rows(bl, M, N, act):
    print(f"[case] epilogue backward, rows: M={M} N={N} {act}", flush=True)
    parts = bl.bitlinear_epilogue_backward_workspace_bytes(M, N) // (4 * N)
    assert parts > 1, "several runs"
    check_backward(bl, M, N, act, "f32", "bf16", "bf16", M + N)


@pytest.mark.parametrize("gy,zt,gz", [(a, b, c) for a in TYPES for b in TYPES for c in TYPES])
@pytest.mark.parametrize("M,N", [(300, 257), (300, 5)])
def test_backward_many_rows_types(bl, gy, zt, gz, M, N):
    check_backward(bl, M, N, "gelu", gy, zt, gz, 7)


@pytest.mark.parametrize("N", [3, 9, 16])
def test_backward_longest_runs(bl, N):
    M = (1 << 20) + 300
    assert bl.bitlinear_epilogue_backward_workspace_bytes(M, N) // (4 * N) == (M + 511) // 512
    check_backward(bl, M, N, "silu", "f32", "f32", "bf16", N)


@pytest.mark.parametrize("M,N", SHAPES)
def test_backward_many_rows_writes_only_its_outputs(bl, M, N):
    g = torch.Generator(device="cuda").manual_seed(N)
    gy, z = torch.randn(M, N, generator=g, device="cuda"), torch.randn(M, N, generator=g, device="cuda")
    want = bl.bitlinear_epilogue_backward(gy, z, "gelu_tanh", 0.5, grad_residual=True)
    out = {k: guarded(v.shape, v.dtype) for k, v in want._asdict().items()}
    ws, wg = guarded((bl.bitlinear_epilogue_backward_workspace_bytes(M, N),), torch.uint8)
    got = bl.bitlinear_epilogue_backward(gy, z, "gelu_tanh", 0.5, workspace=ws, **{k: t for k, (t, _) in out.items()})
    wg.check("workspace", all_written=False)
    for k, (t, guard) in out.items():
        assert getattr(got, k) is t and torch.equal(t, getattr(want, k)), k
        guard.check(k)
