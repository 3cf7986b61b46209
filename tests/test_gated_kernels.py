"""The gated products' kernels in the library are those that a call can reach (read from
the library's symbols), and the rule that picks among the decode batches' (no GPU needed)."""
import re
import subprocess

import pytest

from ternary_weight_linear_bitlinear_amd import build


def kernels(name):
    """Template arguments of every instantiation of a kernel, as the compiler mangles them."""
    out = subprocess.run(["nm", build.LIB_PATH], capture_output=True, text=True, check=True).stdout
    found = re.findall(r" [a-zA-Z] _ZN2bl12_GLOBAL__N_1%d%sI(\S+?)EEv" % (len(name), name), out)
    args = [tuple(a or b for a, b in re.findall(r"L[ib](\d+)E|([ft])", f)) for f in found]
    assert args, name
    return set(args)


def test_decode_of_few_tokens_streams_no_tiles():
    """More than 512 tiles of 16 rows are 8192 rows and more, which take two row groups a
    workgroup: one that streams tiles (the fifth argument) is never asked for."""
    found = kernels("linear_decode_gated_kernel")
    assert not [a for a in found if a[4] == "1"]
    # layouts x (M = 1: three shapes and two row groups; up to 4: one, two, two wide, four) x types
    assert len(found) == 3 * 8 * 4


def test_base3_rows_of_several_rounds_take_three_groups():
    """Four and six row groups (the fourth argument) hold base-3 rows (1) of one round only:
    those of several (the sixth) take three."""
    found = kernels("skinny_gated_kernel")
    assert not [a for a in found if a[0] == "1" and int(a[3]) > 3 and a[5] == "1"]
    assert {a[3] for a in found if a[0] == "1" and a[5] == "1"} == {"1", "2", "3"}


@pytest.mark.parametrize("layout,M,N,several_rounds,groups", [
    ("kLayoutBase3", 16, 16384, "true", 0), ("kLayoutBase3", 9, 13000, "true", 0),  # two, as a plain product
    ("kLayoutBase3", 16, 16400, "true", 3), ("kLayoutBase3", 16, 57344, "true", 3),
    ("kLayoutBase3", 16, 16384, "false", 4), ("kLayoutBase3", 16, 22016, "false", 6),
    ("kLayout2Bit", 16, 16384, "true", 4), ("kLayout1Bit", 40, 24576, "true", 6), ("kLayout2Bit", 9, 24592, "false", 4),
    ("kLayout2Bit", 8, 22016, "false", 0), ("kLayout2Bit", 16, 12288, "false", 0)])
def test_row_groups_of_a_decode_batch(tmp_path, layout, M, N, several_rounds, groups):
    """Base-3 rows of several rounds take three groups from the row count on where two make
    more rounds of workgroups than three do (up to there 16 to 22% slower in three)."""
    src = tmp_path / "groups.hip"
    src.write_text(f'''#include "skinny_core.hpp"
static_assert(bl::gated_row_groups(bl::{layout}, {M}, {N}, {several_rounds}) == {groups});
''')
    r = subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "--cuda-host-only", "-fsyntax-only", str(src)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
