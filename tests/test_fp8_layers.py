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


def _linear(N, K):
    lin = object.__new__(q.QuarotFp8Linear)
    lin.out_features, lin.in_features, lin.w_q, lin.w_scale = N, K, None, None
    return lin


H = torch.float16


@pytest.mark.parametrize("y", [torch.zeros((300, 18), dtype=H), torch.zeros(5400, dtype=H), torch.zeros((9, 600), dtype=H),
                               torch.zeros((), dtype=H), torch.zeros((300, 18), dtype=H).t(),
                               torch.zeros((18, 600), dtype=H)[:, ::2]])
def test_linear_refuses_an_output_of_other_columns(y):
    """[N, M] has as many elements as [M, N], and is not the output."""
    x = torch.zeros((2, 9, 256), dtype=H)
    with pytest.raises(q.QuarotError, match="y must be contiguous with 300 columns"):
        _linear(300, 256)(x, y=y)
