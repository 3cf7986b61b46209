"""Thin Python binding of ``libbitlinear.so`` (the C ABI in include/bitlinear.h).

Argument marshalling only: torch provides device memory and the current
stream; every step of the BitLinear pass runs in the library's HIP kernels.
There is no CPU or PyTorch fallback: if the library is missing, importing
this module raises.

Functions keep the C names (``bitlinear_pack_weights``,
``bitlinear_quant_acts``, ``bitlinear_forward``, ``bitlinear_linear``,
``bitlinear_backward_input``, ``bitlinear_backward_weight``) and take torch
tensors; ``linear`` chains activation quantisation and the forward product.

Around the product: ``bitlinear_forward_epilogue`` / ``bitlinear_linear_epilogue``
(``linear_epilogue`` picks one) add bias, activation and residual,
``bitlinear_block_norm`` takes the norms before and after a block with the gate
and the residual stream between them; each has its backward call.

A gated feed-forward block: ``bitlinear_forward_gated`` / ``bitlinear_linear_gated``
(``linear_gated`` picks one) run both up-projections, the activation and their
product, ``bitlinear_gated_backward`` goes back. A training step keeps 8-bit codes
between the two: ``bitlinear_checkpoint`` / ``bitlinear_checkpoint_restore`` (the
gated calls write and read them directly), ``bitlinear_backward_weight_codes`` takes
the weight gradient from the product's own codes, and
``bitlinear_backward_input_segmented`` the gradient of an input that a stack shares.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
from typing import NamedTuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbitlinear.so")

BL_OK, BL_ERR_INVALID_ARG, BL_ERR_UNSUPPORTED, BL_ERR_DEVICE = 0, 1, 2, 3
BL_F32, BL_BF16 = 0, 1
BL_PACK_2BIT, BL_PACK_BASE3, BL_PACK_1BIT = 0, 1, 2
BL_TERNARY, BL_BINARY = 0, 1

BL_ACT_NONE, BL_ACT_RELU, BL_ACT_RELU2, BL_ACT_SILU, BL_ACT_GELU, BL_ACT_GELU_TANH = range(6)
BL_NORM_NONE, BL_NORM_RMS, BL_NORM_LAYER = range(3)
BL_GATE_NONE, BL_GATE_CHANNEL, BL_GATE_TOKEN = range(3)

ACTS = {"none": BL_ACT_NONE, "relu": BL_ACT_RELU, "relu2": BL_ACT_RELU2, "silu": BL_ACT_SILU,
        "gelu": BL_ACT_GELU, "gelu_tanh": BL_ACT_GELU_TANH}
NORMS = {"none": BL_NORM_NONE, "rms": BL_NORM_RMS, "layer": BL_NORM_LAYER}
LAYOUTS = {"2bit": BL_PACK_2BIT, "base3": BL_PACK_BASE3, "1bit": BL_PACK_1BIT}
SCHEMES = {"ternary": BL_TERNARY, "binary": BL_BINARY}
_DTYPES = {torch.float32: BL_F32, torch.bfloat16: BL_BF16}

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m ternary_weight_linear_bitlinear_amd.build` "
        "(there is no fallback path)")

_lib = ctypes.CDLL(LIB_PATH)
_lib.bitlinear_source_hash.restype = ctypes.c_char_p
_lib.bitlinear_source_hash.argtypes = []


def _refuse_stale_library() -> None:
    """A library built from other sources than the ones beside it would be
    tested and timed in their place: refuse it."""
    from . import build as _build
    if not os.path.isdir(_build.CSRC):
        return  # an installed library without its sources: nothing to compare
    built = _lib.bitlinear_source_hash().decode()
    here = _build.source_hash()
    if built != here:
        raise ImportError(
            f"{LIB_PATH} was built from other sources (library {built}, sources {here}): rebuild "
            "it with `python -m ternary_weight_linear_bitlinear_amd.build`")


_refuse_stale_library()
_p, _i64, _int, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

_lib.bitlinear_packed_row_bytes.restype = _i64
_lib.bitlinear_packed_row_bytes.argtypes = [_i64, _int]
_lib.bitlinear_pack_workspace_bytes.restype = _sz
_lib.bitlinear_pack_workspace_bytes.argtypes = [_i64, _i64]
_lib.bitlinear_pack_weights.restype = _int
_lib.bitlinear_pack_weights.argtypes = [_p, _int, _i64, _i64, _int, _int, _f32, _p, _p, _p, _sz, _p]
_lib.bitlinear_pack_weights_noalloc.restype = _int
_lib.bitlinear_pack_weights_noalloc.argtypes = [_p, _int, _i64, _i64, _int, _int, _f32, _p, _p, _p]
_lib.bitlinear_pack_noalloc_max_scratch_bytes.restype = _sz
_lib.bitlinear_pack_noalloc_max_scratch_bytes.argtypes = []
_lib.bitlinear_quant_acts.restype = _int
_lib.bitlinear_quant_acts.argtypes = [_p, _int, _i64, _i64, _p, _p, _p]
_lib.bitlinear_forward.restype = _int
_lib.bitlinear_forward.argtypes = [_p, _p, _p, _int, _p, _i64, _i64, _i64, _p, _int, _p, _p]
_lib.bitlinear_linear.restype = _int
_lib.bitlinear_linear.argtypes = [_p, _int, _p, _int, _p, _i64, _i64, _i64, _p, _int, _p, _p]
_lib.bitlinear_forward_segmented.restype = _int
_lib.bitlinear_forward_segmented.argtypes = [_p, _p, _p, _int, _p, _p, _int, _i64, _i64, _p, _int,
                                             _p, _p]
_lib.bitlinear_linear_segmented.restype = _int
_lib.bitlinear_linear_segmented.argtypes = [_p, _int, _p, _int, _p, _p, _int, _i64, _i64, _p, _int,
                                            _p, _p]
_lib.bitlinear_forward_lut.restype = _int
_lib.bitlinear_forward_lut.argtypes = [_p, _p, _p, _int, _p, _i64, _i64, _i64, _p, _int, _p, _p]
_lib.bitlinear_backward_input.restype = _int
_lib.bitlinear_backward_input.argtypes = [_p, _int, _p, _int, _p, _i64, _i64, _i64, _p, _p]
_lib.bitlinear_backward_weight.restype = _int
_lib.bitlinear_backward_weight.argtypes = [_p, _p, _int, _i64, _i64, _i64, _p, _p]
_lib.bitlinear_forward_epilogue.restype = _int
_lib.bitlinear_forward_epilogue.argtypes = [_p, _p, _p, _int, _p, _p, _int, _i64, _i64, _p, _int,
                                            _int, _p, _f32, _p, _p, _int, _p]
_lib.bitlinear_linear_epilogue.restype = _int
_lib.bitlinear_linear_epilogue.argtypes = [_p, _int, _p, _int, _p, _p, _int, _i64, _i64, _p, _int,
                                           _int, _p, _f32, _p, _p, _int, _p]
_lib.bitlinear_epilogue_backward_workspace_bytes.restype = _sz
_lib.bitlinear_epilogue_backward_workspace_bytes.argtypes = [_i64, _i64]
_lib.bitlinear_epilogue_backward.restype = _int
_lib.bitlinear_epilogue_backward.argtypes = [_p, _int, _p, _int, _int, _f32, _i64, _i64, _p, _int,
                                             _p, _p, _p, _sz, _p]
_lib.bitlinear_block_norm.restype = _int
_lib.bitlinear_block_norm.argtypes = [_p, _int, _p, _int, _f32, _p, _int, _int, _p, _p, _f32,
                                      _int, _p, _p, _f32, _int, _i64, _i64, _p, _p, _p, _p, _p, _p]
_lib.bitlinear_block_norm_backward_workspace_bytes.restype = _sz
_lib.bitlinear_block_norm_backward_workspace_bytes.argtypes = [_i64, _i64]
_lib.bitlinear_block_norm_backward.restype = _int
_lib.bitlinear_block_norm_backward.argtypes = [_p, _p, _int, _p, _int, _p, _int, _p, _f32, _p, _int,
                                               _int, _p, _p, _int, _p, _int, _i64, _i64, _p, _p,
                                               _p, _p, _p, _p, _p, _p, _sz, _p]
_lib.bitlinear_forward_gated.restype = _int
_lib.bitlinear_forward_gated.argtypes = [_p, _p, _p, _int, _p, _i64, _i64, _i64, _p, _int, _int,
                                         _p, _p, _p, _p, _int, _p]
_lib.bitlinear_linear_gated.restype = _int
_lib.bitlinear_linear_gated.argtypes = [_p, _int, _p, _int, _p, _i64, _i64, _i64, _p, _int, _int,
                                        _p, _p, _int, _p]
_lib.bitlinear_gated_backward_workspace_bytes.restype = _sz
_lib.bitlinear_gated_backward_workspace_bytes.argtypes = [_i64, _i64]
_lib.bitlinear_gated_backward.restype = _int
_lib.bitlinear_gated_backward.argtypes = [_p, _int, _p, _int, _p, _p, _int, _i64, _i64, _p, _int,
                                          _p, _p, _sz, _p]
_lib.bitlinear_checkpoint_groups.restype = _i64
_lib.bitlinear_checkpoint_groups.argtypes = [_i64]
_lib.bitlinear_checkpoint.restype = _int
_lib.bitlinear_checkpoint.argtypes = [_p, _int, _i64, _i64, _p, _p, _p]
_lib.bitlinear_checkpoint_restore.restype = _int
_lib.bitlinear_checkpoint_restore.argtypes = [_p, _p, _i64, _i64, _p, _int, _p]
_lib.bitlinear_backward_weight_codes.restype = _int
_lib.bitlinear_backward_weight_codes.argtypes = [_p, _int, _p, _p, _i64, _i64, _i64, _p, _int, _p, _sz, _p]
_lib.bitlinear_backward_weight_codes_workspace_bytes.restype = _sz
_lib.bitlinear_backward_weight_codes_workspace_bytes.argtypes = [_i64, _i64, _i64, _int]
_lib.bitlinear_backward_input_segmented_workspace_bytes.restype = _sz
_lib.bitlinear_backward_input_segmented_workspace_bytes.argtypes = [_i64, _i64, _i64, _int]
_lib.bitlinear_backward_input_segmented.restype = _int
_lib.bitlinear_backward_input_segmented.argtypes = [_p, _int, _p, _int, _p, _p, _int, _i64, _i64,
                                                    _p, _int, _p, _sz, _p]
_lib.bitlinear_forward_plan.restype = _int
_lib.bitlinear_forward_plan.argtypes = [_i64, _i64, _i64, _int, _int, _int, ctypes.c_char_p, _sz]
_lib.bitlinear_status_string.restype = ctypes.c_char_p
_lib.bitlinear_status_string.argtypes = [_int]
_lib.bitlinear_version.restype = _int
_lib.bitlinear_version.argtypes = []

EXPORTED = ["bitlinear_packed_row_bytes", "bitlinear_pack_workspace_bytes",
            "bitlinear_pack_weights", "bitlinear_pack_weights_noalloc",
            "bitlinear_pack_noalloc_max_scratch_bytes", "bitlinear_quant_acts", "bitlinear_forward",
            "bitlinear_linear", "bitlinear_forward_segmented", "bitlinear_linear_segmented",
            "bitlinear_forward_lut", "bitlinear_backward_input", "bitlinear_backward_weight",
            "bitlinear_forward_epilogue", "bitlinear_linear_epilogue",
            "bitlinear_epilogue_backward_workspace_bytes", "bitlinear_epilogue_backward",
            "bitlinear_block_norm", "bitlinear_block_norm_backward_workspace_bytes",
            "bitlinear_block_norm_backward", "bitlinear_forward_gated", "bitlinear_linear_gated",
            "bitlinear_gated_backward_workspace_bytes", "bitlinear_gated_backward",
            "bitlinear_checkpoint_groups", "bitlinear_checkpoint", "bitlinear_checkpoint_restore",
            "bitlinear_backward_weight_codes_workspace_bytes", "bitlinear_backward_weight_codes",
            "bitlinear_backward_input_segmented_workspace_bytes", "bitlinear_backward_input_segmented",
            "bitlinear_forward_plan", "bitlinear_status_string",
            "bitlinear_version",
            "bitlinear_source_hash"]
FUSED_MAX_M = 4


class BitLinearError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {_lib.bitlinear_status_string(status).decode()} (status {status})")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != BL_OK:
        raise BitLinearError(status, where)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _layout(layout) -> int:
    return LAYOUTS[layout] if isinstance(layout, str) else int(layout)


def library() -> ctypes.CDLL:
    return _lib


# ----------------------------------------------------------------------------
def bitlinear_packed_row_bytes(K: int, layout="2bit") -> int:
    return int(_lib.bitlinear_packed_row_bytes(K, _layout(layout)))


def bitlinear_pack_workspace_bytes(N: int, K: int) -> int:
    return int(_lib.bitlinear_pack_workspace_bytes(N, K))


def bitlinear_version() -> int:
    return int(_lib.bitlinear_version())


def bitlinear_forward_plan(M: int, N: int, K: int, layout="2bit", out_dtype=torch.float32,
                           fused: bool = False) -> list[str]:
    """The kernel launches bitlinear_forward (or, with fused=True,
    bitlinear_linear on bf16 x) would make for an M x N x K product, one
    string per launch; nothing is launched."""
    buf = ctypes.create_string_buffer(8192)
    n = _lib.bitlinear_forward_plan(M, N, K, _layout(layout), _DTYPES[out_dtype], int(fused),
                                    buf, len(buf))
    if n < 0:
        raise BitLinearError(BL_ERR_INVALID_ARG, "bitlinear_forward_plan")
    lines = buf.value.decode().splitlines()
    assert len(lines) == n
    return lines


def bitlinear_status_string(status: int) -> str:
    return _lib.bitlinear_status_string(status).decode()


def bitlinear_pack_weights(W: torch.Tensor, layout="2bit", scheme="ternary", eps: float = 1e-5,
                           packed: torch.Tensor | None = None, gamma: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, stream=None):
    """Quantise and pack W [N, K] (fp32 or bf16, on the GPU).

    Returns (packed uint8 [N, row_bytes], gamma float32 [1]) on W's device."""
    assert W.dim() == 2 and W.is_contiguous() and W.dtype in _DTYPES
    N, K = W.shape
    lay = _layout(layout)
    rb = bitlinear_packed_row_bytes(K, lay)
    dev = W.device
    if packed is None:
        packed = torch.empty((N, rb), dtype=torch.uint8, device=dev)
    if gamma is None:
        gamma = torch.empty(4, dtype=torch.float32, device=dev)[:1]
    wsb = bitlinear_pack_workspace_bytes(N, K)
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
    _check(_lib.bitlinear_pack_weights(_ptr(W), _DTYPES[W.dtype], N, K,
                                       SCHEMES[scheme] if isinstance(scheme, str) else int(scheme),
                                       lay, float(eps), _ptr(packed), _ptr(gamma),
                                       _ptr(workspace), workspace.numel(), _stream(stream)),
           "bitlinear_pack_weights")
    return packed, gamma


def bitlinear_pack_weights_noalloc(W: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor,
                                   layout="2bit", scheme="ternary", eps: float = 1e-5,
                                   stream=None):
    """bitlinear_pack_weights into caller-provided packed / gamma, with the
    library's own scratch instead of a workspace (nothing is allocated)."""
    assert W.dim() == 2 and W.is_contiguous() and W.dtype in _DTYPES
    N, K = W.shape
    _check(_lib.bitlinear_pack_weights_noalloc(
        _ptr(W), _DTYPES[W.dtype], N, K, SCHEMES[scheme] if isinstance(scheme, str) else int(scheme),
        _layout(layout), float(eps), _ptr(packed), _ptr(gamma), _stream(stream)),
        "bitlinear_pack_weights_noalloc")
    return packed, gamma


def bitlinear_pack_noalloc_max_scratch_bytes() -> int:
    return int(_lib.bitlinear_pack_noalloc_max_scratch_bytes())


def bitlinear_quant_acts(x: torch.Tensor, xq: torch.Tensor | None = None,
                         scale: torch.Tensor | None = None, stream=None):
    """Per-token INT8 quantisation of x [M, K]; returns (xq int8 [M, K], scale f32 [M])."""
    assert x.dim() == 2 and x.is_contiguous() and x.dtype in _DTYPES
    M, K = x.shape
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty(max(M, 1), dtype=torch.float32, device=x.device)[:M]
    _check(_lib.bitlinear_quant_acts(_ptr(x), _DTYPES[x.dtype], M, K, _ptr(xq), _ptr(scale),
                                     _stream(stream)), "bitlinear_quant_acts")
    return xq, scale


def bitlinear_forward(xq: torch.Tensor, scale: torch.Tensor, packed: torch.Tensor,
                      gamma: torch.Tensor, N: int, K: int, layout="2bit",
                      out_dtype=torch.float32, y: torch.Tensor | None = None,
                      acc: torch.Tensor | bool | None = None, stream=None):
    """y = (xq c^T) * gamma * scale / 127; returns y, or (y, acc) when acc is requested."""
    M = xq.shape[0]
    assert xq.dim() == 2 and xq.shape[1] == K and xq.dtype == torch.int8
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    want_acc = acc is not None and acc is not False
    if acc is True:
        acc = torch.empty((M, N), dtype=torch.int32, device=xq.device)
    _check(_lib.bitlinear_forward(_ptr(xq), _ptr(scale), _ptr(packed), _layout(layout),
                                  _ptr(gamma), M, N, K, _ptr(y), _DTYPES[y.dtype],
                                  _ptr(acc) if want_acc else None, _stream(stream)),
           "bitlinear_forward")
    return (y, acc) if want_acc else y


def bitlinear_linear(x: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor, N: int,
                     layout="2bit", out_dtype=torch.float32, y: torch.Tensor | None = None,
                     acc: torch.Tensor | bool | None = None, stream=None):
    """Fused quantise + multiply for M <= 4 tokens; returns y, or (y, acc)."""
    assert x.dim() == 2 and x.is_contiguous() and x.dtype in _DTYPES
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    want_acc = acc is not None and acc is not False
    if acc is True:
        acc = torch.empty((M, N), dtype=torch.int32, device=x.device)
    _check(_lib.bitlinear_linear(_ptr(x), _DTYPES[x.dtype], _ptr(packed), _layout(layout),
                                 _ptr(gamma), M, N, K, _ptr(y), _DTYPES[y.dtype],
                                 _ptr(acc) if want_acc else None, _stream(stream)),
           "bitlinear_linear")
    return (y, acc) if want_acc else y


def bitlinear_forward_lut(xq: torch.Tensor, scale: torch.Tensor, packed: torch.Tensor,
                          gamma: torch.Tensor, N: int, K: int, out_dtype=torch.float32,
                          y: torch.Tensor | None = None, acc: torch.Tensor | bool | None = None,
                          stream=None):
    """One token against base-3 codes through activation-side lookup tables."""
    M = xq.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    want_acc = acc is not None and acc is not False
    if acc is True:
        acc = torch.empty((M, N), dtype=torch.int32, device=xq.device)
    _check(_lib.bitlinear_forward_lut(_ptr(xq), _ptr(scale), _ptr(packed), BL_PACK_BASE3,
                                      _ptr(gamma), M, N, K, _ptr(y), _DTYPES[y.dtype],
                                      _ptr(acc) if want_acc else None, _stream(stream)),
           "bitlinear_forward_lut")
    return (y, acc) if want_acc else y


def _seg_table(seg_rows):
    rows = [int(r) for r in seg_rows]
    return (ctypes.c_int64 * len(rows))(*rows), len(rows), sum(rows)


def bitlinear_forward_segmented(xq: torch.Tensor, scale: torch.Tensor, packed: torch.Tensor,
                                gammas: torch.Tensor, seg_rows, K: int, layout="2bit",
                                out_dtype=torch.float32, y: torch.Tensor | None = None,
                                acc: torch.Tensor | bool | None = None, stream=None):
    """bitlinear_forward over a stack of row segments, each with its own gamma
    (gammas[s]); y [M, sum(seg_rows)]."""
    M = xq.shape[0]
    table, nseg, N = _seg_table(seg_rows)
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    want_acc = acc is not None and acc is not False
    if acc is True:
        acc = torch.empty((M, N), dtype=torch.int32, device=xq.device)
    _check(_lib.bitlinear_forward_segmented(_ptr(xq), _ptr(scale), _ptr(packed), _layout(layout),
                                            _ptr(gammas), table, nseg, M, K, _ptr(y),
                                            _DTYPES[y.dtype], _ptr(acc) if want_acc else None,
                                            _stream(stream)), "bitlinear_forward_segmented")
    return (y, acc) if want_acc else y


def bitlinear_linear_segmented(x: torch.Tensor, packed: torch.Tensor, gammas: torch.Tensor,
                               seg_rows, layout="2bit", out_dtype=torch.float32,
                               y: torch.Tensor | None = None,
                               acc: torch.Tensor | bool | None = None, stream=None):
    """Fused quantise + multiply (M <= 4) over a stack of row segments."""
    assert x.dim() == 2 and x.is_contiguous() and x.dtype in _DTYPES
    M, K = x.shape
    table, nseg, N = _seg_table(seg_rows)
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    want_acc = acc is not None and acc is not False
    if acc is True:
        acc = torch.empty((M, N), dtype=torch.int32, device=x.device)
    _check(_lib.bitlinear_linear_segmented(_ptr(x), _DTYPES[x.dtype], _ptr(packed),
                                           _layout(layout), _ptr(gammas), table, nseg, M, K,
                                           _ptr(y), _DTYPES[y.dtype],
                                           _ptr(acc) if want_acc else None, _stream(stream)),
           "bitlinear_linear_segmented")
    return (y, acc) if want_acc else y


def bitlinear_backward_input(grad_y: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor,
                             K: int, layout="2bit", grad_x: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor:
    """grad_x [M, K] fp32 = gamma * grad_y [M, N] (bf16) x codes of packed [N, row_bytes]."""
    assert grad_y.dim() == 2 and grad_y.is_contiguous() and grad_y.dtype in _DTYPES
    M, N = grad_y.shape
    if grad_x is None:
        grad_x = torch.empty((M, K), dtype=torch.float32, device=grad_y.device)
    _check(_lib.bitlinear_backward_input(_ptr(grad_y), _DTYPES[grad_y.dtype], _ptr(packed),
                                         _layout(layout), _ptr(gamma), M, N, K, _ptr(grad_x),
                                         _stream(stream)), "bitlinear_backward_input")
    return grad_x


def bitlinear_backward_weight(grad_y: torch.Tensor, x: torch.Tensor,
                              grad_w: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """grad_w [N, K] fp32 = grad_y^T (bf16 [M, N]) x x (bf16 [M, K])."""
    assert grad_y.dim() == 2 and x.dim() == 2 and grad_y.shape[0] == x.shape[0]
    assert grad_y.is_contiguous() and x.is_contiguous() and grad_y.dtype == x.dtype
    M, N = grad_y.shape
    K = x.shape[1]
    if grad_w is None:
        grad_w = torch.empty((N, K), dtype=torch.float32, device=x.device)
    _check(_lib.bitlinear_backward_weight(_ptr(grad_y), _ptr(x), _DTYPES[x.dtype], M, N, K,
                                          _ptr(grad_w), _stream(stream)),
           "bitlinear_backward_weight")
    return grad_w


def linear(x: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor, N: int, layout="2bit",
           out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """BitLinear forward of x [M, K] against packed weights: one fused launch for
    M <= 4, otherwise quantise then multiply."""
    if x.shape[0] <= FUSED_MAX_M:
        return bitlinear_linear(x, packed, gamma, N, layout, out_dtype, stream=stream)
    xq, scale = bitlinear_quant_acts(x, stream=stream)
    return bitlinear_forward(xq, scale, packed, gamma, N, x.shape[1], layout, out_dtype,
                             stream=stream)


# ---- bias, activation and residual in the epilogue; norms around a block ----
# These calls check what the C ABI cannot see (shapes, types, devices, strides)
# and raise BitLinearError for it as for the library's own refusals. They run on
# the device of their first tensor and its current stream; `stream` makes another
# one current first, so that what a call allocates (outputs, workspace) belongs to
# the stream that its kernels run on. The decode products take a few microseconds,
# so the checks are kept to one pass over each tensor's attributes and what depends
# on sizes alone is cached.
_f32, _bf16 = torch.float32, torch.bfloat16
_FLT_MAX = 3.4028234663852886e38


def _refuse(where: str, why: str):
    e = BitLinearError(BL_ERR_INVALID_ARG, where)
    e.args = (f"{e.args[0]}: {why}",)
    raise e


def _addr(where: str, name: str, t: torch.Tensor, shape, dtype, dev: int) -> int:
    """Address of a contiguous tensor on GPU `dev` of this type and shape."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        _refuse(where, f"{name} is {t.dtype}, not {dtype}")
    if t.shape != shape:
        _refuse(where, f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.get_device() != dev:
        _refuse(where, f"{name} is on {t.device}, not on GPU {dev}")
    _refuse(where, f"{name} is not contiguous")


def _lead(where: str, name: str, t: torch.Tensor):
    """Shape, type, GPU and address of the tensor that the others have to match."""
    dtype, shape = t.dtype, t.shape
    if (dtype is not _f32 and dtype is not _bf16) or len(shape) != 2:
        _refuse(where, f"{name} is {dtype} of shape {tuple(shape)}")
    if not t.is_contiguous():
        _refuse(where, f"{name} is not contiguous")
    return shape, dtype, t.get_device(), t.data_ptr()


def _float(where: str, name: str, t: torch.Tensor):
    dtype = t.dtype
    if dtype is not _f32 and dtype is not _bf16:
        _refuse(where, f"{name} is {dtype}")
    return dtype


def _on(where: str, stream, t: torch.Tensor):
    """The context that makes `stream`, one of t's GPU, the current one."""
    if stream.device != t.device:
        _refuse(where, f"the stream is of {stream.device}, the tensors are on {t.device}")
    return torch.cuda.stream(stream)


def _run(where: str, dev: int, call, args) -> None:
    """One library call on GPU `dev` and its current stream."""
    if dev < 0:
        _refuse(where, "tensors are on the cpu")
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            status = call(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        status = call(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status != BL_OK:
        raise BitLinearError(status, where)


def _one_of(where: str, name: str, v, table) -> int:
    got = table.get(v)
    if got is None:
        if isinstance(v, str):
            _refuse(where, f"{name} is {v!r}, not one of {', '.join(table)}")
        got = int(v)
    return got


def _check_scale(where: str, v) -> None:
    if not -_FLT_MAX <= v <= _FLT_MAX:
        _refuse(where, f"residual_scale is {v}")


@functools.lru_cache(maxsize=1024)
def _segments(rows):
    """Row counts as the C table (never written), their number and their sum."""
    return _seg_table((rows,) if isinstance(rows, int) else rows)


def _rows_of(seg_rows):
    """seg_rows as a key of _segments: a tuple of counts, or one count, as plain
    numbers (a tensor would be a key by its identity, whatever it holds)."""
    if not isinstance(seg_rows, (list, tuple)):
        try:
            return operator.index(seg_rows)
        except TypeError:
            pass
    return tuple([int(r) for r in seg_rows])


_row_bytes = functools.lru_cache(maxsize=1024)(bitlinear_packed_row_bytes)


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(call: str, *sizes) -> int:
    """A size helper of the library for plain numbers (a tensor would be a key by its
    identity, whatever it holds): the public helpers make numbers of what they are given."""
    return int(getattr(_lib, call)(*sizes))


def _product_epilogue(where, call, lead, M, K, dev, packed, gammas, seg_rows, layout, bias, act, residual,
                      residual_scale, out_dtype, y, z):
    lay = _one_of(where, "layout", layout, LAYOUTS)
    table, nseg, N = _segments(seg_rows if type(seg_rows) is int else _rows_of(seg_rows))
    if out_dtype is None:
        out_dtype = y.dtype if y is not None else residual.dtype if residual is not None else _f32
    if out_dtype is not _f32 and out_dtype is not _bf16:
        _refuse(where, f"out_dtype is {out_dtype}")
    shape = (M, N)
    if y is None:
        y = torch.empty(M, N, dtype=out_dtype, device=packed.device)
    want_z = z is not None and z is not False
    if z is True:
        z = torch.empty(M, N, dtype=out_dtype, device=packed.device)
    if (gammas.dtype is not _f32 or gammas.numel() < nseg or gammas.get_device() != dev
            or not gammas.is_contiguous()):
        _refuse(where, f"gammas holds {gammas.numel()} of {gammas.dtype} on {gammas.device} for {nseg} segments, "
                       "or is not contiguous")
    _check_scale(where, residual_scale)
    args = (*lead, _addr(where, "packed", packed, (N, _row_bytes(K, lay)), torch.uint8, dev), lay,
            gammas.data_ptr(), table, nseg, M, K,
            None if bias is None else _addr(where, "bias", bias, (N,), _float(where, "bias", bias), dev),
            BL_F32 if bias is None else _DTYPES[bias.dtype], _one_of(where, "act", act, ACTS),
            None if residual is None else _addr(where, "residual", residual, shape, out_dtype, dev),
            residual_scale, _addr(where, "z", z, shape, out_dtype, dev) if want_z else None,
            _addr(where, "y", y, shape, out_dtype, dev), BL_F32 if out_dtype is _f32 else BL_BF16)
    _run(where, dev, call, args)
    return (y, z) if want_z else y


def bitlinear_forward_epilogue(xq: torch.Tensor, scale: torch.Tensor, packed: torch.Tensor,
                               gammas: torch.Tensor, seg_rows, K: int, layout="2bit", bias=None,
                               act="none", residual=None, residual_scale: float = 1.0,
                               out_dtype=None, y: torch.Tensor | None = None,
                               z: torch.Tensor | bool | None = None,
                               stream=None):
    """y = act(z) + residual_scale * residual with z = the product of
    bitlinear_forward (bitlinear_forward_segmented) + bias.

    seg_rows: N, or the row counts of stacked matrices (gammas[s] each).
    residual may be y itself; it is added as stored, so a bf16 residual is rounded
    before the sum. out_dtype defaults to y's, then residual's type,
    then fp32; y, z and residual share it. Returns y, or (y, z) when z is
    requested."""
    if stream is not None:
        with _on("bitlinear_forward_epilogue", stream, xq):
            return bitlinear_forward_epilogue(xq, scale, packed, gammas, seg_rows, K, layout, bias, act, residual,
                                              residual_scale, out_dtype, y, z)
    where = "bitlinear_forward_epilogue"
    if xq.dim() != 2:
        _refuse(where, f"xq has shape {tuple(xq.shape)}")
    M, dev = xq.shape[0], xq.get_device()
    lead = (_addr(where, "xq", xq, (M, K), torch.int8, dev), _addr(where, "scale", scale, (M,), _f32, dev))
    K = xq.shape[1]
    return _product_epilogue(where, _lib.bitlinear_forward_epilogue, lead, M, K, dev, packed, gammas, seg_rows,
                             layout, bias, act, residual, residual_scale, out_dtype, y, z)


def bitlinear_linear_epilogue(x: torch.Tensor, packed: torch.Tensor, gammas: torch.Tensor, seg_rows,
                              layout="2bit", bias=None, act="none", residual=None,
                              residual_scale: float = 1.0, out_dtype=None,
                              y: torch.Tensor | None = None, z: torch.Tensor | bool | None = None,
                              stream=None):
    """bitlinear_forward_epilogue fused with the quantisation of x, M <= 4 tokens."""
    if stream is not None:
        with _on("bitlinear_linear_epilogue", stream, x):
            return bitlinear_linear_epilogue(x, packed, gammas, seg_rows, layout, bias, act, residual,
                                             residual_scale, out_dtype, y, z)
    where = "bitlinear_linear_epilogue"
    (M, K), dtype, dev, x_at = _lead(where, "x", x)
    lead = (x_at, BL_F32 if dtype is _f32 else BL_BF16)
    return _product_epilogue(where, _lib.bitlinear_linear_epilogue, lead, M, K, dev, packed, gammas, seg_rows,
                             layout, bias, act, residual, residual_scale, out_dtype, y, z)


def linear_epilogue(x: torch.Tensor, packed: torch.Tensor, gammas: torch.Tensor, seg_rows,
                    layout="2bit", bias=None, act="none", residual=None,
                    residual_scale: float = 1.0, out_dtype=None, y: torch.Tensor | None = None,
                    z: torch.Tensor | bool | None = None,
                    stream=None):
    """``linear`` with bias, activation and residual: one fused launch for
    M <= 4, otherwise quantise then multiply."""
    if stream is not None:
        with _on("linear_epilogue", stream, x):
            return linear_epilogue(x, packed, gammas, seg_rows, layout, bias, act, residual, residual_scale,
                                   out_dtype, y, z)
    if x.dim() != 2 or x.shape[0] <= FUSED_MAX_M:
        return bitlinear_linear_epilogue(x, packed, gammas, seg_rows, layout, bias, act, residual, residual_scale,
                                         out_dtype, y, z)
    where = "linear_epilogue"
    (M, K), dtype, dev, x_at = _lead(where, "x", x)
    xq = torch.empty(M, K, dtype=torch.int8, device=x.device)
    scale = torch.empty(M, dtype=_f32, device=x.device)
    _run(where, dev, _lib.bitlinear_quant_acts,
         (x_at, BL_F32 if dtype is _f32 else BL_BF16, M, K, xq.data_ptr(), scale.data_ptr()))
    return bitlinear_forward_epilogue(xq, scale, packed, gammas, seg_rows, K, layout, bias, act, residual,
                                      residual_scale, out_dtype, y, z)


def _workspace(where: str, ws, need: int, t: torch.Tensor):
    """Address and bytes of the caller's workspace, or of a new one beside t (held by the returned tensor)."""
    if ws is None:
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=t.device)
    elif ws.get_device() != t.get_device() or not ws.is_contiguous():
        _refuse(where, "workspace is on another device or not contiguous")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


class EpilogueGrads(NamedTuple):
    grad_z: torch.Tensor | None
    grad_bias: torch.Tensor | None
    grad_residual: torch.Tensor | None


def bitlinear_epilogue_backward_workspace_bytes(M: int, N: int) -> int:
    return _workspace_bytes("bitlinear_epilogue_backward_workspace_bytes", operator.index(M), operator.index(N))


def bitlinear_epilogue_backward(grad_y: torch.Tensor, z: torch.Tensor | None, act="none",
                                residual_scale: float = 1.0, out_dtype=None,
                                grad_z: torch.Tensor | bool | None = True,
                                grad_bias: torch.Tensor | bool | None = True,
                                grad_residual: torch.Tensor | bool | None = None,
                                workspace: torch.Tensor | None = None,
                                stream=None) -> EpilogueGrads:
    """Gradients of y = act(z) + residual_scale * residual, z = product + bias:
    grad_z [M, N] (out_dtype, grad_y's type by default), grad_bias [N] fp32,
    grad_residual [M, N] of grad_y's type. Each is a buffer, True (allocate) or
    None (leave out); none may overlap grad_y or z. z may be None for act "none"."""
    if stream is not None:
        with _on("bitlinear_epilogue_backward", stream, grad_y):
            return bitlinear_epilogue_backward(grad_y, z, act, residual_scale, out_dtype, grad_z, grad_bias,
                                               grad_residual, workspace)
    where = "bitlinear_epilogue_backward"
    shape, dtype, dev, gy_at = _lead(where, "grad_y", grad_y)
    M, N = shape
    own = grad_z is not None and grad_z is not True and grad_z is not False
    if out_dtype is None:
        out_dtype = grad_z.dtype if own else dtype
    if out_dtype is not _f32 and out_dtype is not _bf16:
        _refuse(where, f"out_dtype is {out_dtype}")
    if not own:
        grad_z = torch.empty(M, N, dtype=out_dtype, device=grad_y.device) if grad_z else None
    if grad_bias is True:
        grad_bias = torch.empty(N, dtype=_f32, device=grad_y.device)
    elif grad_bias is False:
        grad_bias = None
    if grad_residual is True:
        grad_residual = torch.empty_like(grad_y)
    elif grad_residual is False:
        grad_residual = None
    _check_scale(where, residual_scale)
    need = bitlinear_epilogue_backward_workspace_bytes(M, N) if grad_bias is not None else 0
    hold, ws, ws_bytes = (None, None, 0) if need == 0 else _workspace(where, workspace, need, grad_y)
    args = (gy_at, BL_F32 if dtype is _f32 else BL_BF16,
            None if z is None else _addr(where, "z", z, shape, _float(where, "z", z), dev),
            BL_F32 if z is None else _DTYPES[z.dtype], _one_of(where, "act", act, ACTS), residual_scale, M, N,
            None if grad_z is None else _addr(where, "grad_z", grad_z, shape, out_dtype, dev), _DTYPES[out_dtype],
            None if grad_bias is None else _addr(where, "grad_bias", grad_bias, (N,), _f32, dev),
            None if grad_residual is None else _addr(where, "grad_residual", grad_residual, shape, dtype, dev),
            ws, ws_bytes)
    _run(where, dev, _lib.bitlinear_epilogue_backward, args)
    return EpilogueGrads(grad_z, grad_bias, grad_residual)


class Norm(NamedTuple):
    """A norm of bitlinear_block_norm: "rms" or "layer", its [K] weight and bias
    (None: 1 and 0) and eps."""
    kind: str | int = "rms"
    weight: torch.Tensor | None = None
    bias: torch.Tensor | None = None
    eps: float = 1e-5


class BlockNorm(NamedTuple):
    h_out: torch.Tensor | None
    n: torch.Tensor | None
    xq: torch.Tensor | None
    scale: torch.Tensor | None
    stats: torch.Tensor | None


class BlockNormGrads(NamedTuple):
    grad_h: torch.Tensor
    grad_block: torch.Tensor | None
    grad_gate: torch.Tensor | None
    grad_post_weight: torch.Tensor | None
    grad_post_bias: torch.Tensor | None
    grad_pre_weight: torch.Tensor | None
    grad_pre_bias: torch.Tensor | None


_NO_NORM = Norm(BL_NORM_NONE)


def _norm_args(where, shape, dev, x_dtype, pre, post, gate):
    """The parameters' arguments: (gate, gate kind, post kind, weight, bias, post
    eps), (pre kind, weight, bias, pre eps), p_dtype."""
    qk, qw, qb, qe = post or _NO_NORM
    pk, pw, pb, pe = pre or _NO_NORM
    row = shape[1:]
    gk = BL_GATE_NONE if gate is None else BL_GATE_TOKEN if gate.dim() == 2 else BL_GATE_CHANNEL
    first = qw if qw is not None else pw if pw is not None else qb if qb is not None else pb
    if first is None and gk == BL_GATE_CHANNEL:
        first = gate
    P = _f32 if first is None else _float(where, "a parameter", first)
    g = None
    if gk:
        g = _addr(where, "gate", gate, shape, x_dtype, dev) if gk == BL_GATE_TOKEN else \
            _addr(where, "gate", gate, row, P, dev)
    return ((g, gk, _one_of(where, "post.kind", qk, NORMS),
             None if qw is None else _addr(where, "post.weight", qw, row, P, dev),
             None if qb is None else _addr(where, "post.bias", qb, row, P, dev), qe),
            (_one_of(where, "pre.kind", pk, NORMS),
             None if pw is None else _addr(where, "pre.weight", pw, row, P, dev),
             None if pb is None else _addr(where, "pre.bias", pb, row, P, dev), pe),
            BL_F32 if P is _f32 else BL_BF16)


def bitlinear_block_norm(h: torch.Tensor, block: torch.Tensor | None = None,
                         pre: Norm | None = None, post: Norm | None = None,
                         gate: torch.Tensor | None = None, residual_scale: float = 1.0,
                         out_dtype=None, normed: bool = True, quant: bool = False,
                         h_out: torch.Tensor | None = None, n: torch.Tensor | None = None,
                         xq: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                         stats: torch.Tensor | bool | None = None,
                         stream=None) -> BlockNorm:
    """h_out = residual_scale * h + gate * post(block) and n = pre(h_out), in one
    pass over h [M, K] and block [M, K].

    block None: h_out is h (not written) and only pre runs. gate: [K], or [M, K]
    of block's type. n has block's type (out_dtype without a block, h's by
    default); normed=False leaves it out. quant: also the INT8 codes and scale of
    n, as bitlinear_quant_acts(n in fp32). stats (a buffer or True): what the
    backward call needs. h_out may be h."""
    if stream is not None:
        with _on("bitlinear_block_norm", stream, h):
            return bitlinear_block_norm(h, block, pre, post, gate, residual_scale, out_dtype, normed, quant, h_out,
                                        n, xq, scale, stats)
    where = "bitlinear_block_norm"
    shape, H, dev, h_at = _lead(where, "h", h)
    M, K = shape
    if block is not None:
        X = _float(where, "block", block)
    else:
        X = out_dtype or (n.dtype if n is not None else H)
    if (X is not _f32 and X is not _bf16) or (out_dtype is not None and out_dtype is not X):
        _refuse(where, f"block is {X}, out_dtype {out_dtype}")
    post_a, pre_a, P = _norm_args(where, shape, dev, X, pre, post, gate)
    if block is not None and h_out is None:
        h_out = torch.empty_like(h)
    if pre is None or not normed:
        if n is not None:
            _refuse(where, "n is given without a norm that writes it")
    elif n is None:
        n = torch.empty(M, K, dtype=X, device=h.device)
    if quant or xq is not None or scale is not None:
        if xq is None:
            xq = torch.empty(M, K, dtype=torch.int8, device=h.device)
        if scale is None:
            scale = torch.empty(M, dtype=_f32, device=h.device)
    if stats is True:
        stats = torch.empty(M, 4, dtype=_f32, device=h.device)
    elif stats is False:
        stats = None
    _check_scale(where, residual_scale)
    args = (h_at, BL_F32 if H is _f32 else BL_BF16,
            None if block is None else _addr(where, "block", block, shape, X, dev),
            BL_F32 if X is _f32 else BL_BF16, residual_scale, *post_a, *pre_a, P, M, K,
            None if h_out is None else _addr(where, "h_out", h_out, shape, H, dev),
            None if n is None else _addr(where, "n", n, shape, X, dev),
            None if xq is None else _addr(where, "xq", xq, shape, torch.int8, dev),
            None if scale is None else _addr(where, "scale", scale, (M,), _f32, dev),
            None if stats is None else _addr(where, "stats", stats, (M, 4), _f32, dev))
    _run(where, dev, _lib.bitlinear_block_norm, args)
    return BlockNorm(h if block is None else h_out, n, xq, scale, stats)


def _param_grad(where, name, t, p, row, dev):
    """A [K] parameter gradient and its address: the buffer t, a new one where there
    is a parameter p, or none."""
    if t is not None:
        return t, _addr(where, name, t, row, _f32, dev)
    if p is None:
        return None, None
    t = torch.empty(row[0], dtype=_f32, device=p.device)
    return t, t.data_ptr()


def bitlinear_block_norm_backward_workspace_bytes(M: int, K: int) -> int:
    return _workspace_bytes("bitlinear_block_norm_backward_workspace_bytes", operator.index(M), operator.index(K))


def bitlinear_block_norm_backward(grad_h_out: torch.Tensor | None, grad_n: torch.Tensor | None,
                                  h_out: torch.Tensor, block: torch.Tensor | None,
                                  stats: torch.Tensor, pre: Norm | None = None,
                                  post: Norm | None = None, gate: torch.Tensor | None = None,
                                  residual_scale: float = 1.0, params: bool = True,
                                  grad_h: torch.Tensor | None = None,
                                  grad_block: torch.Tensor | None = None,
                                  grad_gate: torch.Tensor | None = None,
                                  grad_post_weight: torch.Tensor | None = None,
                                  grad_post_bias: torch.Tensor | None = None,
                                  grad_pre_weight: torch.Tensor | None = None,
                                  grad_pre_bias: torch.Tensor | None = None,
                                  workspace: torch.Tensor | None = None,
                                  stream=None) -> BlockNormGrads:
    """Gradients of bitlinear_block_norm. h_out, stats: as that call returned
    them; grad_h_out: the gradient of h_out from its other uses (None: zero);
    grad_n: the gradient of n (None without pre), or of the quantised input
    (straight-through). Parameter gradients are fp32 [K] (a gate per token: [M, K]
    of block's type); params=False leaves out those that no buffer is given for. No
    output may overlap an input (grad_h is not grad_h_out)."""
    if stream is not None:
        with _on("bitlinear_block_norm_backward", stream, h_out):
            return bitlinear_block_norm_backward(grad_h_out, grad_n, h_out, block, stats, pre, post, gate,
                                                 residual_scale, params, grad_h, grad_block, grad_gate,
                                                 grad_post_weight, grad_post_bias, grad_pre_weight, grad_pre_bias,
                                                 workspace)
    where = "bitlinear_block_norm_backward"
    shape, H, dev, h_at = _lead(where, "h_out", h_out)
    M, K = shape
    row = shape[1:]
    X = H if block is None else _float(where, "block", block)
    post_a, pre_a, P = _norm_args(where, shape, dev, X, pre, post, gate)
    token = post_a[1] == BL_GATE_TOKEN
    if grad_h is None:
        grad_h = torch.empty_like(h_out)
    if grad_block is None and block is not None:
        grad_block = torch.empty_like(block)
    qw = qb = pw = pb = None
    if post is not None and params:
        _, qw, qb, _ = post
    if pre is not None and params:
        _, pw, pb, _ = pre
    grad_post_weight, qw = _param_grad(where, "grad_post_weight", grad_post_weight, qw, row, dev)
    grad_post_bias, qb = _param_grad(where, "grad_post_bias", grad_post_bias, qb, row, dev)
    grad_pre_weight, pw = _param_grad(where, "grad_pre_weight", grad_pre_weight, pw, row, dev)
    grad_pre_bias, pb = _param_grad(where, "grad_pre_bias", grad_pre_bias, pb, row, dev)
    if not token:
        grad_gate, gate_p = _param_grad(where, "grad_gate", grad_gate, gate if params else None, row, dev)
    elif grad_gate is not None:
        gate_p = _addr(where, "grad_gate", grad_gate, shape, X, dev)
    elif params:
        grad_gate = torch.empty_like(gate)
        gate_p = grad_gate.data_ptr()
    else:
        gate_p = None
    _check_scale(where, residual_scale)
    hold, ws, ws_bytes = _workspace(where, workspace, bitlinear_block_norm_backward_workspace_bytes(M, K), h_out)
    args = (None if grad_h_out is None else _addr(where, "grad_h_out", grad_h_out, shape, H, dev),
            None if grad_n is None else _addr(where, "grad_n", grad_n, shape, _float(where, "grad_n", grad_n), dev),
            BL_F32 if grad_n is None else _DTYPES[grad_n.dtype],
            h_at, BL_F32 if H is _f32 else BL_BF16,
            None if block is None else _addr(where, "block", block, shape, X, dev),
            BL_F32 if X is _f32 else BL_BF16, _addr(where, "stats", stats, (M, 4), _f32, dev), residual_scale,
            *post_a[:5], *pre_a[:2], P, M, K, _addr(where, "grad_h", grad_h, shape, H, dev),
            None if grad_block is None else _addr(where, "grad_block", grad_block, shape, X, dev),
            gate_p, qw, qb, pw, pb, ws, ws_bytes)
    _run(where, dev, _lib.bitlinear_block_norm_backward, args)
    return BlockNormGrads(grad_h, grad_block, grad_gate, grad_post_weight, grad_post_bias,
                          grad_pre_weight, grad_pre_bias)


# ---- gated feed-forward products and activations kept in 8 bits --------------
class Checkpoint(NamedTuple):
    """A tensor [M, K] in 8 bits: codes [M, K] int8 and a scale for each 64 columns of
    a row, [M, ceil(K / 64)] fp32. A value is code * (scale / 127)."""
    codes: torch.Tensor
    scale: torch.Tensor


class GatedProduct(NamedTuple):
    y: torch.Tensor
    z: torch.Tensor | None
    kept: Checkpoint | None


class GatedGrads(NamedTuple):
    grad_z: torch.Tensor | None
    grad_bias: torch.Tensor | None


def bitlinear_checkpoint_groups(K: int) -> int:
    """Scales of a kept row of K columns."""
    return -(-K // 64) if K > 0 else 0


def _kept(where, kept, M, K, dev, t):
    """A checkpoint of [M, K] and its addresses: the caller's (checked), or a new one
    beside t where `kept` is True."""
    shape = (M, bitlinear_checkpoint_groups(K))
    if kept is True:
        kept = Checkpoint(torch.empty(M, K, dtype=torch.int8, device=t.device),
                          torch.empty(shape, dtype=_f32, device=t.device))
        return kept, kept.codes.data_ptr(), kept.scale.data_ptr()
    if not isinstance(kept, tuple) or len(kept) != 2:
        _refuse(where, f"kept is {type(kept).__name__}, not a Checkpoint")
    codes, scale = kept
    return kept, _addr(where, "kept.codes", codes, (M, K), torch.int8, dev), \
        _addr(where, "kept.scale", scale, shape, _f32, dev)


def _code(dtype) -> int:
    return BL_F32 if dtype is _f32 else BL_BF16


def _out_dtype(where, out_dtype, given):
    """The type of an output: as asked for, or that of the caller's buffer, or fp32."""
    dtype = out_dtype or (given.dtype if given is not None else _f32)
    if dtype is not _f32 and dtype is not _bf16:
        _refuse(where, f"out_dtype is {dtype}")
    return dtype


def _gated(where, call, lead, M, K, dev, packed, gammas, F, layout, bias, act, out_dtype, y, z, kept, beside):
    lay = _one_of(where, "layout", layout, LAYOUTS)
    F = operator.index(F)
    out_dtype = _out_dtype(where, out_dtype, y)
    if y is None:
        y = torch.empty(M, F, dtype=out_dtype, device=packed.device)
    if z is True:
        z = torch.empty(M, 2 * F, dtype=out_dtype, device=packed.device)
    elif z is False:
        z = None
    if kept is False:
        kept = None
    keep = ()
    if beside:  # the call that can leave a checkpoint
        keep = (None, None)
        if kept is not None:
            kept, *keep = _kept(where, kept, 2 * M, F, dev, packed)
    elif kept is not None:
        _refuse(where, "the fused call leaves no checkpoint")
    if gammas.dtype is not _f32 or gammas.numel() < 2 or gammas.get_device() != dev or not gammas.is_contiguous():
        _refuse(where, f"gammas holds {gammas.numel()} of {gammas.dtype} on {gammas.device} for 2 matrices, "
                       "or is not contiguous")
    args = (*lead, _addr(where, "packed", packed, (2 * F, _row_bytes(K, lay)), torch.uint8, dev), lay,
            gammas.data_ptr(), F, M, K,
            None if bias is None else _addr(where, "bias", bias, (2 * F,), _float(where, "bias", bias), dev),
            BL_F32 if bias is None else _DTYPES[bias.dtype], _one_of(where, "act", act, ACTS),
            None if z is None else _addr(where, "z", z, (M, 2 * F), out_dtype, dev), *keep,
            _addr(where, "y", y, (M, F), out_dtype, dev), _code(out_dtype))
    _run(where, dev, call, args)
    return GatedProduct(y, z, kept)


def bitlinear_forward_gated(xq: torch.Tensor, scale: torch.Tensor, packed: torch.Tensor,
                            gammas: torch.Tensor, F: int, K: int, layout="2bit", bias=None, act="silu",
                            out_dtype=None, y: torch.Tensor | None = None,
                            z: torch.Tensor | bool | None = None,
                            kept: Checkpoint | bool | None = None, stream=None) -> GatedProduct:
    """y [M, F] = act(z[:, :F]) * z[:, F:] with z = the product of a stack of two
    matrices of F rows (gate, then the other; gammas[0], gammas[1]) + bias [2F].

    z (a buffer or True): also the pre-activations [M, 2F], of y's type. kept (a
    Checkpoint or True): them in 8 bits for bitlinear_gated_backward, as
    bitlinear_checkpoint gives for z in fp32 seen as [2M, F]. out_dtype defaults to
    y's type, then fp32. No output may overlap another argument."""
    if stream is not None:
        with _on("bitlinear_forward_gated", stream, xq):
            return bitlinear_forward_gated(xq, scale, packed, gammas, F, K, layout, bias, act, out_dtype, y, z, kept)
    where = "bitlinear_forward_gated"
    if xq.dim() != 2:
        _refuse(where, f"xq has shape {tuple(xq.shape)}")
    M, dev = xq.shape[0], xq.get_device()
    lead = (_addr(where, "xq", xq, (M, K), torch.int8, dev), _addr(where, "scale", scale, (M,), _f32, dev))
    return _gated(where, _lib.bitlinear_forward_gated, lead, M, xq.shape[1], dev, packed, gammas, F, layout, bias,
                  act, out_dtype, y, z, kept, True)


def bitlinear_linear_gated(x: torch.Tensor, packed: torch.Tensor, gammas: torch.Tensor, F: int,
                           layout="2bit", bias=None, act="silu", out_dtype=None,
                           y: torch.Tensor | None = None, z: torch.Tensor | bool | None = None,
                           stream=None) -> GatedProduct:
    """bitlinear_forward_gated fused with the quantisation of x, M <= 4 tokens, without
    a checkpoint."""
    if stream is not None:
        with _on("bitlinear_linear_gated", stream, x):
            return bitlinear_linear_gated(x, packed, gammas, F, layout, bias, act, out_dtype, y, z)
    where = "bitlinear_linear_gated"
    (M, K), dtype, dev, x_at = _lead(where, "x", x)
    return _gated(where, _lib.bitlinear_linear_gated, (x_at, _code(dtype)), M, K, dev, packed, gammas, F, layout,
                  bias, act, out_dtype, y, z, None, False)


def linear_gated(x: torch.Tensor, packed: torch.Tensor, gammas: torch.Tensor, F: int, layout="2bit",
                 bias=None, act="silu", out_dtype=None, y: torch.Tensor | None = None,
                 z: torch.Tensor | bool | None = None, kept: Checkpoint | bool | None = None,
                 stream=None) -> GatedProduct:
    """``linear`` for a gated pair of matrices: one fused launch for M <= 4 without a
    checkpoint, otherwise quantise then multiply."""
    if stream is not None:
        with _on("linear_gated", stream, x):
            return linear_gated(x, packed, gammas, F, layout, bias, act, out_dtype, y, z, kept)
    if x.dim() != 2 or (x.shape[0] <= FUSED_MAX_M and (kept is None or kept is False)):
        return bitlinear_linear_gated(x, packed, gammas, F, layout, bias, act, out_dtype, y, z)
    where = "linear_gated"
    (M, K), dtype, dev, x_at = _lead(where, "x", x)
    xq = torch.empty(M, K, dtype=torch.int8, device=x.device)
    scale = torch.empty(M, dtype=_f32, device=x.device)
    _run(where, dev, _lib.bitlinear_quant_acts, (x_at, _code(dtype), M, K, xq.data_ptr(), scale.data_ptr()))
    return bitlinear_forward_gated(xq, scale, packed, gammas, F, K, layout, bias, act, out_dtype, y, z, kept)


def bitlinear_gated_backward_workspace_bytes(M: int, F: int) -> int:
    return _workspace_bytes("bitlinear_gated_backward_workspace_bytes", operator.index(M), operator.index(F))


def bitlinear_gated_backward(grad_y: torch.Tensor, z: torch.Tensor | Checkpoint, act="silu",
                             out_dtype=None, grad_z: torch.Tensor | bool | None = True,
                             grad_bias: torch.Tensor | bool | None = True,
                             workspace: torch.Tensor | None = None, stream=None) -> GatedGrads:
    """Gradients of y = act(z[:, :F]) * z[:, F:] for grad_y [M, F]: grad_z [M, 2F]
    (out_dtype, grad_y's type by default) and its column sums grad_bias [2F] fp32.
    z: the pre-activations [M, 2F], or the Checkpoint that the forward call left. Each
    output is a buffer, True (allocate) or None (leave out); none may overlap an input."""
    if stream is not None:
        with _on("bitlinear_gated_backward", stream, grad_y):
            return bitlinear_gated_backward(grad_y, z, act, out_dtype, grad_z, grad_bias, workspace)
    where = "bitlinear_gated_backward"
    (M, F), dtype, dev, gy_at = _lead(where, "grad_y", grad_y)
    own = grad_z is not None and grad_z is not True and grad_z is not False
    if out_dtype is None:
        out_dtype = grad_z.dtype if own else dtype
    out_dtype = _out_dtype(where, out_dtype, None)
    if not own:
        grad_z = torch.empty(M, 2 * F, dtype=out_dtype, device=grad_y.device) if grad_z else None
    if grad_bias is True:
        grad_bias = torch.empty(2 * F, dtype=_f32, device=grad_y.device)
    elif grad_bias is False:
        grad_bias = None
    if isinstance(z, tuple):
        _, codes, code_scale = _kept(where, z, 2 * M, F, dev, grad_y)
        z_args = (None, BL_F32, codes, code_scale)
    else:
        z_args = (_addr(where, "z", z, (M, 2 * F), _float(where, "z", z), dev), _DTYPES[z.dtype], None, None)
    need = bitlinear_gated_backward_workspace_bytes(M, F) if grad_bias is not None else 0
    hold, ws, ws_bytes = (None, None, 0) if need == 0 else _workspace(where, workspace, need, grad_y)
    args = (gy_at, _code(dtype), *z_args, _one_of(where, "act", act, ACTS), M, F,
            None if grad_z is None else _addr(where, "grad_z", grad_z, (M, 2 * F), out_dtype, dev), _code(out_dtype),
            None if grad_bias is None else _addr(where, "grad_bias", grad_bias, (2 * F,), _f32, dev), ws, ws_bytes)
    _run(where, dev, _lib.bitlinear_gated_backward, args)
    return GatedGrads(grad_z, grad_bias)


def bitlinear_checkpoint(x: torch.Tensor, kept: Checkpoint | None = None, stream=None) -> Checkpoint:
    """x [M, K] in 8 bits, a scale for each 64 columns of a row."""
    if stream is not None:
        with _on("bitlinear_checkpoint", stream, x):
            return bitlinear_checkpoint(x, kept)
    where = "bitlinear_checkpoint"
    (M, K), dtype, dev, x_at = _lead(where, "x", x)
    kept, codes, scale = _kept(where, True if kept is None else kept, M, K, dev, x)
    _run(where, dev, _lib.bitlinear_checkpoint, (x_at, _code(dtype), M, K, codes, scale))
    return kept


def bitlinear_checkpoint_restore(kept: Checkpoint, out_dtype=None, y: torch.Tensor | None = None,
                                 stream=None) -> torch.Tensor:
    """The kept values as a tensor [M, K] (out_dtype: y's type by default, then fp32)."""
    where = "bitlinear_checkpoint_restore"
    if not isinstance(kept, tuple) or len(kept) != 2:
        _refuse(where, f"kept is {type(kept).__name__}, not a Checkpoint")
    codes = kept[0]
    if stream is not None:
        with _on(where, stream, codes):
            return bitlinear_checkpoint_restore(kept, out_dtype, y)
    if codes.dim() != 2:
        _refuse(where, f"kept.codes has shape {tuple(codes.shape)}")
    (M, K), dev = codes.shape, codes.get_device()
    _, codes_at, scale_at = _kept(where, kept, M, K, dev, codes)
    out_dtype = _out_dtype(where, out_dtype, y)
    if y is None:
        y = torch.empty(M, K, dtype=out_dtype, device=codes.device)
    _run(where, dev, _lib.bitlinear_checkpoint_restore,
         (codes_at, scale_at, M, K, _addr(where, "y", y, (M, K), out_dtype, dev), _code(out_dtype)))
    return y


def bitlinear_backward_weight_codes_workspace_bytes(M: int, N: int, K: int, out_dtype=torch.float32) -> int:
    where = "bitlinear_backward_weight_codes_workspace_bytes"
    return _workspace_bytes(where, operator.index(M), operator.index(N), operator.index(K),
                            _code(_out_dtype(where, out_dtype, None)))


def bitlinear_backward_input_segmented_workspace_bytes(M: int, N: int, K: int, grad_dtype=torch.float32) -> int:
    where = "bitlinear_backward_input_segmented_workspace_bytes"
    if grad_dtype not in _DTYPES:
        _refuse(where, f"grad_dtype is {grad_dtype}")
    return _workspace_bytes(where, operator.index(M), operator.index(N), operator.index(K), _code(grad_dtype))


def bitlinear_backward_weight_codes(grad_y: torch.Tensor, xq: torch.Tensor, scale: torch.Tensor,
                                    out_dtype=None, grad_w: torch.Tensor | None = None,
                                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """grad_w [N, K] = sum_m grad_y[m, n] * (scale[m] / 127) * xq[m, k], from the codes
    that the forward product had (out_dtype: grad_w's type by default, then fp32)."""
    if stream is not None:
        with _on("bitlinear_backward_weight_codes", stream, grad_y):
            return bitlinear_backward_weight_codes(grad_y, xq, scale, out_dtype, grad_w, workspace)
    where = "bitlinear_backward_weight_codes"
    (M, N), dtype, dev, gy_at = _lead(where, "grad_y", grad_y)
    if xq.dim() != 2:
        _refuse(where, f"xq has shape {tuple(xq.shape)}")
    K = xq.shape[1]
    out_dtype = _out_dtype(where, out_dtype, grad_w)
    if grad_w is None:
        grad_w = torch.empty(N, K, dtype=out_dtype, device=grad_y.device)
    need = bitlinear_backward_weight_codes_workspace_bytes(M, N, K, out_dtype)
    hold, ws, ws_bytes = (None, None, 0) if need == 0 else _workspace(where, workspace, need, grad_y)
    _run(where, dev, _lib.bitlinear_backward_weight_codes,
         (gy_at, _code(dtype), _addr(where, "xq", xq, (M, K), torch.int8, dev),
          _addr(where, "scale", scale, (M,), _f32, dev), M, N, K,
          _addr(where, "grad_w", grad_w, (N, K), out_dtype, dev), _code(out_dtype), ws, ws_bytes))
    return grad_w


def bitlinear_backward_input_segmented(grad_y: torch.Tensor, packed: torch.Tensor, gammas: torch.Tensor,
                                       seg_rows, K: int, layout="2bit", out_dtype=None,
                                       grad_x: torch.Tensor | None = None,
                                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """grad_x [M, K] of the input that a stack of matrices shares (seg_rows: N, or the
    row counts; gammas[s] each; out_dtype: grad_x's type by default, then fp32)."""
    if stream is not None:
        with _on("bitlinear_backward_input_segmented", stream, grad_y):
            return bitlinear_backward_input_segmented(grad_y, packed, gammas, seg_rows, K, layout, out_dtype, grad_x,
                                                      workspace)
    where = "bitlinear_backward_input_segmented"
    lay = _one_of(where, "layout", layout, LAYOUTS)
    table, nseg, N = _segments(_rows_of(seg_rows))
    (M, cols), dtype, dev, gy_at = _lead(where, "grad_y", grad_y)
    if cols != N:
        _refuse(where, f"grad_y has {cols} columns for {N} rows of weights")
    if gammas.dtype is not _f32 or gammas.numel() < nseg or gammas.get_device() != dev or not gammas.is_contiguous():
        _refuse(where, f"gammas holds {gammas.numel()} of {gammas.dtype} on {gammas.device} for {nseg} segments, "
                       "or is not contiguous")
    K = operator.index(K)
    out_dtype = _out_dtype(where, out_dtype, grad_x)
    if grad_x is None:
        grad_x = torch.empty(M, K, dtype=out_dtype, device=grad_y.device)
    need = bitlinear_backward_input_segmented_workspace_bytes(M, N, K, dtype)
    hold, ws, ws_bytes = (None, None, 0) if need == 0 else _workspace(where, workspace, need, grad_y)
    _run(where, dev, _lib.bitlinear_backward_input_segmented,
         (gy_at, _code(dtype), _addr(where, "packed", packed, (N, _row_bytes(K, lay)), torch.uint8, dev), lay,
          gammas.data_ptr(), table, nseg, M, K, _addr(where, "grad_x", grad_x, (M, K), out_dtype, dev),
          _code(out_dtype), ws, ws_bytes))
    return grad_x
