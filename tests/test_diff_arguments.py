"""Arguments that the differentiable calls refuse before any device call."""
import pytest
import torch

from block_sparse_video_rearrange_b200 import diff


@pytest.mark.parametrize("num_groups", [1, 4, 16])
def test_a_number_of_groups_that_x_does_not_have(num_groups):
    x, g = torch.zeros(1, 4, 2, 8), torch.ones(2, 8)
    with pytest.raises(ValueError, match="groups"):
        diff.group_norm(x, g, g, num_groups)
