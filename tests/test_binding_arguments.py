"""The allocating calls of the binding check their arguments before they use them: ValueError for what is no matrix."""
import pytest
import torch

fc = pytest.importorskip("long_fft_convolution_amd")


@pytest.mark.parametrize("x,W", [((3,), (4, 3)), ((2, 3), (4,)), ((2, 3, 1), (4, 3)), ((), (4, 3)), ((2, 3), ())])
def test_products_of_what_is_no_matrix(x, W):
    x, W = torch.zeros(x), torch.zeros(W)
    with pytest.raises(ValueError, match="2 dimensions"):
        fc.linear_act(x, W)
    with pytest.raises(ValueError, match="2 dimensions"):
        fc.linear_act_bwd(torch.zeros(2, 4), x, W)
