"""Arguments that the 8-bit layer classes refuse, before anything is launched."""
import pytest
import torch

import w4a4_rotated_quantized_gb300 as q


def _mlp(K):
    mlp = object.__new__(q.QuarotFp8GatedMLP)  # its weights are not looked at
    mlp.features, mlp.norm_weight, mlp.eps = K, None, 1e-6
    return mlp


@pytest.mark.parametrize("shape", [(3, 2, 256), (6, 256), (1, 3, 256), (2, 3, 128)])
def test_mlp_refuses_a_residual_of_another_shape(shape):
    """As many elements are not enough: the rows of [3, 2, K] are other tokens than those of [2, 3, K]."""
    x = torch.zeros((2, 3, 256), dtype=torch.float16)
    with pytest.raises(q.QuarotError, match="residual has shape"):
        _mlp(256)(x, torch.zeros(shape, dtype=torch.float16))
