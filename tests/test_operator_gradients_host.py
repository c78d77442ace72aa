"""What the differentiable operators do to an upstream gradient before the kernels see it (on the CPU)."""

import pytest
import torch

from lm_head_linear_gb300 import ops


def view(offset, shape, stride, dtype):
    t = torch.arange(offset + shape[0] * max(stride[0], 1) + shape[1] * stride[1] + 16).to(dtype)
    return torch.as_strided(t, shape, stride, offset)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,stride", [(0, (32, 1)), (8, (40, 1)),  # as they are
                                           (1, (32, 1)), (2, (40, 1)),  # contiguous rows off 16 bytes
                                           (0, (33, 1)), (0, (0, 1)), (0, (0, 0)), (0, (1, 5)), (4, (64, 2))])
def test_gradients_come_out_as_the_kernels_take_them(dtype, offset, stride):
    t = view(offset, (5, 32), stride, dtype)
    d = ops._dense_rows(t)
    assert torch.equal(d, t) and d.dtype == t.dtype
    assert d.stride(1) == 1 and d.stride(0) >= 32 and d.stride(0) * d.element_size() % 16 == 0
    assert d.data_ptr() % 16 == 0
    if (offset, stride) in ((0, (32, 1)), (8, (40, 1))):
        assert d.data_ptr() == t.data_ptr()
