"""Arguments of the delta rule's Python binding that the checks meet before the
library's own (CPU: tensors that nothing can be launched on)."""
import pytest
import torch

import selective_state_space_31_amd as pkg

Z = torch.zeros


def test_keys_without_columns():
    """headdim_k = 0 is refused as a size, before the default scale is formed."""
    for lead, f in (((2, 5), pkg.ssm_delta_rule_fwd), ((2,), lambda *a: pkg.ssm_delta_state_update(Z(2, 4, 0, 6), *a))):
        with pytest.raises(ValueError, match="headdim"):
            f(Z(*lead, 2, 0), Z(*lead, 2, 0), Z(*lead, 4, 6), Z(*lead, 4))
    with pytest.raises(ValueError, match="headdim"):
        pkg.ssm_delta_rule_bwd(Z(2, 5, 2, 0), Z(2, 5, 2, 0), Z(2, 5, 4, 6), Z(2, 5, 4), Z(2, 5, 4, 6))


@pytest.mark.parametrize("cu", [[0, 5], (0, 5), 5, "no"])
def test_offsets_that_are_no_tensor(cu):
    a = (Z(5, 2, 8), Z(5, 2, 8), Z(5, 4, 6), Z(5, 4))
    with pytest.raises(TypeError, match="cu_seqlens"):
        pkg.ssm_delta_rule_fwd_varlen(*a, cu)
    with pytest.raises(TypeError, match="cu_seqlens"):
        pkg.ssm_delta_rule_bwd_varlen(*a, cu, a[2])
