"""The matrix scale of a matrix of nearly 2^31 rows (one column): the largest value stands in the last row,
which a row counter of 31 bits would step past."""
import numpy as np
import pytest
import torch

from mixed_precision_quantized_mx_b200 import binding as mx

pytestmark = pytest.mark.gpu


def test_gscale_of_the_most_rows():
    rows = 2 ** 31 - 128
    L = mx.mx_fp4_layout_init(rows, 1)
    x = torch.zeros(rows, 1, dtype=torch.float16, device="cuda")
    x[0], x[rows // 2], x[rows - 1] = 1.0, -2.0, 3.0
    assert float(mx.mx_fp4_gscale(L, x)) == np.float32(3) / np.float32(2688)
