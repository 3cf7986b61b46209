"""What the device code promises the compiler, read from small compiles of the
kernels' headers (no GPU needed)."""
import os
import re
import subprocess

import pytest

from ternary_weight_linear_bitlinear_amd import build

DECODE = """
template __global__ void linear_decode_epilogue_kernel<kLayout2Bit, 8, 2, 4, true, 1, uint16_t, float>(
    const uint16_t *, const uint8_t *, const GammaMap, int, int64_t, int64_t, int64_t, float *, const Epilogue<float>);
template __global__ void skinny_epilogue_kernel<kLayout2Bit, 8, 2, 1, 16, true, float>(
    const int8_t *, const float *, const uint8_t *, const GammaMap, int, int64_t, int64_t, int64_t, float *,
    const Epilogue<float>);
template __global__ void linear_decode_kernel<kLayout2Bit, 8, 2, 4, true, 1, uint16_t, float>(
    const uint16_t *, const uint8_t *, const GammaMap, int, int64_t, int64_t, int64_t, float *, int32_t *);
template __global__ void skinny_kernel<kLayout2Bit, 8, 2, 1, 16, true, float>(
    const int8_t *, const float *, const uint8_t *, const GammaMap, int, int64_t, int64_t, int64_t, float *, int32_t *);
"""


def compile_snippet(tmp_path, header, body):
    """(return code, error text, unoptimised device code) of `body` in the library's namespace."""
    src, out = tmp_path / "snippet.hip", tmp_path / "snippet.ll"
    src.write_text(f'#include "{header}"\nnamespace bl {{ namespace {{\n{body}\n}} }}\n')
    r = subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "--cuda-device-only", "-S", "-emit-llvm", "-Xclang",
                        "-disable-llvm-passes", str(src), "-o", str(out)], capture_output=True, text=True, timeout=300)
    return r.returncode, r.stderr, out.read_text() if os.path.exists(out) else ""


def unaliased_outputs(code, name):
    """Of the functions of this name: how many pointers each declares unaliased."""
    found = re.findall(r"^define [^\n]*@(\S*?%s[^\s(]*)\(([^\n]*)\)" % name, code, re.M)
    assert found, name
    return [args.count(" noalias ") for _, args in found if "ENK" not in _]


def test_products_in_place_make_no_false_promise(tmp_path):
    """The residual of the extended epilogue may be y itself: its kernels declare
    only their inputs unaliased (and the sums, which they do not write). The plain
    kernels write nothing that they read, and declare every array."""
    rc, err, code = compile_snippet(tmp_path, "skinny_core.hpp", DECODE)
    assert rc == 0, err
    # x, packed (and the sums in the block); xq, scale, packed (and the sums)
    assert unaliased_outputs(code, "29linear_decode_epilogue_kernel") == [2]
    assert unaliased_outputs(code, "22skinny_epilogue_kernel") == [3]
    assert sorted(unaliased_outputs(code, "19linear_decode_block")) == [3, 4]
    assert sorted(unaliased_outputs(code, "12skinny_block")) == [4, 5]
    assert unaliased_outputs(code, "20linear_decode_kernel") == [4]
    assert unaliased_outputs(code, "13skinny_kernel") == [5]


@pytest.mark.parametrize("BN,fits", [(64, False), (128, True), (256, True)])
def test_staged_rows_hold_their_permutation(tmp_path, BN, fits):
    """A staged row of BN sums has BN / 4 chunks, and its permutation chunk ^ row takes
    rows up to 31: narrower rows than 128 would leave their memory, and do not compile."""
    slots = {(r * (BN // 4) + (c ^ r)) for r in range(32) for c in range(BN // 4)}
    assert (slots == set(range(32 * BN // 4))) is fits
    rc, err, _ = compile_snippet(tmp_path, "gemm_core.hpp", f"template __device__ int frag_slot<{BN}>(int, int);")
    assert (rc == 0) is fits, err


def test_fetched_pieces_keep_their_type(tmp_path):
    """What the decode epilogue fetches ahead is held in the type that it is loaded
    in and taken apart by value, not read back through pointers of other types."""
    body = """
        static_assert(std::is_same_v<decltype(EpilogueAhead<float>::res), uint4>);
        static_assert(std::is_same_v<decltype(EpilogueAhead<uint16_t>::res), uint2>);"""
    rc, err, _ = compile_snippet(tmp_path, "skinny_core.hpp", body)
    assert rc == 0, err
