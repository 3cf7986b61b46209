"""The gated products' kernels in the library are those that a call can reach (read from
the library's symbols; no GPU needed)."""
import re
import subprocess

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
