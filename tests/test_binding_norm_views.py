"""The torch binding without a GPU: norm operands whose heads are not side by side are refused, not copied."""
import pytest
import torch

import selective_state_space_14_amd as ssd
from tests.test_binding_streams import OnGpu


@pytest.mark.parametrize("R,g,W,strides", [(4, 2, 3, (20, 3, 2)), (1, 2, 3, (20, 3, 2)), (5, 3, 7, (60, 7, 3))])
def test_columns_apart(R, g, W, strides):
    """Heads W elements apart whose columns are not next to each other: a result in a copy of y would be lost."""
    x = torch.zeros(R, g, W).as_subclass(OnGpu)
    odd = torch.zeros(400).as_strided((R, g, W), strides).as_subclass(OnGpu)
    for call in (lambda: ssd.ssd_norm_fwd(x, y=odd), lambda: ssd.ssd_norm_fwd(odd, y=x), lambda: ssd.ssd_norm_fwd(x, z=odd, y=x.clone()),
                 lambda: ssd._norm_groups(ssd._Call(x, "x"), x.shape, {"x": (x, None), "grad_y": (odd, None)})):
        with pytest.raises(ValueError, match="innermost dimension must be contiguous"):
            call()


def test_heads_of_one_column():
    """There the columns' own stride says nothing."""
    x = torch.zeros(400).as_strided((4, 3, 1), (20, 1, 5)).as_subclass(OnGpu)
    n, g, at = ssd._norm_groups(ssd._Call(x, "x"), x.shape, {"x": (x, None)})
    assert (n, g, at["x"]) == (4, 3, (x.data_ptr(), 20))
