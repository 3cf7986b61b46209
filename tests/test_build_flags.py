"""What the build's compiler flags refuse (no GPU needed)."""
import subprocess

import pytest

from ternary_weight_linear_bitlinear_amd import build

KERNEL = """#include <hip/hip_runtime.h>
__global__ void sum(const int *x, int *y, int n) {
    int s = 0;
%s
    for (int i = threadIdx.x; i < n; i += 64) {
        s += x[i];
        %s
    }
    y[threadIdx.x] = s;
}
"""


@pytest.mark.parametrize("pragma,body,builds", [
    ("#pragma unroll 2", "", True),
    ("", "s += __builtin_amdgcn_update_dpp(0, s, 0xB1, 0xf, 0xf, false);", True),
    # lanes that read one another keep a loop of unknown length as it is
    ("#pragma unroll 2", "s += __builtin_amdgcn_update_dpp(0, s, 0xB1, 0xf, 0xf, false);", False)])
def test_a_pragma_that_does_nothing_is_an_error(tmp_path, pragma, body, builds):
    src = tmp_path / "sum.hip"
    src.write_text(KERNEL % (pragma, body))
    r = subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "-c", str(src), "-o", str(tmp_path / "sum.o")],
                       capture_output=True, text=True, timeout=300)
    assert (r.returncode == 0) is builds, r.stderr
