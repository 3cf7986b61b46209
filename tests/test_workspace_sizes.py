"""The workspaces' size helpers answer for the numbers that they are given (no GPU needed)."""
import pytest
import torch

from ternary_weight_linear_bitlinear_amd import bitlinear as bl

HELPERS = [(bl.bitlinear_epilogue_backward_workspace_bytes, (4096,)), (bl.bitlinear_block_norm_backward_workspace_bytes, (4096,)),
           (bl.bitlinear_gated_backward_workspace_bytes, (4096,)),
           (bl.bitlinear_backward_weight_codes_workspace_bytes, (256, 256)),
           (bl.bitlinear_backward_input_segmented_workspace_bytes, (8192, 4096))]


@pytest.mark.parametrize("helper,rest", HELPERS, ids=lambda v: getattr(v, "__name__", None))
def test_a_count_in_a_tensor(helper, rest):
    """The size is that of the count that the tensor holds now, not when it was last asked for."""
    M = torch.tensor(200)
    sizes = []
    for n in (200, 4000, 600, 200):
        M.fill_(n)
        sizes.append(helper(M, *rest))
        assert sizes[-1] == helper(n, *rest)
    assert len(set(sizes)) > 1


@pytest.mark.parametrize("helper,rest", HELPERS, ids=lambda v: getattr(v, "__name__", None))
def test_no_count(helper, rest):
    for bad in (2.0, "200", None, torch.tensor(200.0)):
        with pytest.raises(TypeError):
            helper(bad, *rest)


@pytest.mark.parametrize("helper", [bl.bitlinear_backward_weight_codes_workspace_bytes,
                                    bl.bitlinear_backward_input_segmented_workspace_bytes])
def test_a_type_that_the_call_refuses(helper):
    """No size for a type that the call itself would not take."""
    for bad in (torch.float16, torch.float64, torch.int8, "f32"):
        with pytest.raises(bl.BitLinearError):
            helper(300, 4096, 4096, bad)
    assert helper(300, 4096, 4096, torch.float32) == helper(300, 4096, 4096)
