"""The gradient norm's limit on the elements of all tensors together: within it a launch's
partial sums fit the workspace, whatever is given more than once (refused on the host)."""
import ctypes

import numpy as np
import pytest

from nvfp4_w4a4_moe_permute_gb300 import build as B
from nvfp4_w4a4_moe_permute_gb300 import minite as M
from test_step_ops_refusals import FAKE, GRAD_TENSOR

SHAPE = 2


@pytest.mark.parametrize("count,n", [(2, 1 << 41), (3, (1 << 41) - 1), (128, 1 << 36), (129, 1 << 35), (1000, (1 << 33) - 1),
                                     (1 << 12, 1 << 30), (5000, (1 << 42) - 1)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_elements_of_all_tensors(count, n, dtype):
    B.build()
    t = np.zeros(count, dtype=GRAD_TENSOR)
    t["grad"], t["out"], t["n"], t["grad_dtype"], t["out_dtype"] = 1 << 12, 1 << 13, n, dtype, dtype
    assert M.load().minite_grad_norm(t.ctypes.data, count, 0, 1.0, FAKE, FAKE, ctypes.c_void_p(1 << 14), 1 << 30, None) == SHAPE
    assert M.load().minite_clip_grads(t.ctypes.data, count, FAKE, None) == SHAPE
