"""A_cat and B_cat are given together or not at all."""
import pytest
import torch

import sparse_rank_linear_b200 as salr


class Tensor:
    """What the checks look at, of a bf16 CUDA tensor."""
    dtype, is_cuda, device = torch.bfloat16, True, "cuda:0"

    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0


class Square:
    def _shape(self):
        return 128, 128

    def info(self):
        return {"N": 128, "K": 128}


@pytest.mark.parametrize("A,B", [(Tensor(128, 8), None), (None, Tensor(8, 128))])
def test_one_adapter_matrix_alone_is_refused(A, B):
    X = Tensor(4, 128)
    for call in (lambda: salr.linear(X, Square(), A, B), lambda: salr.linear_backward(X, X, Square(), A, B),
                 lambda: salr.linear_host(X, Square(), A, B, X)):
        with pytest.raises(ValueError, match="A_cat and B_cat"):
            call()
