"""Rows of the routing kernels that are wider than their column counters: refused before anything is launched."""
import ctypes

import pytest

from mixed_precision_quantized_mx_b200 import binding as mx

MOST = 2 ** 31 - 1024
UNSUPPORTED, INVALID = 2, 1


@pytest.mark.parametrize("H,status", [(MOST + 1, UNSUPPORTED), (2 ** 31 - 1, UNSUPPORTED), (0, INVALID), (-5, INVALID),
                                      (MOST, INVALID), (24, INVALID)])   # the plan is missing: a call past the check of H
def test_columns(H, status):
    P, lib = mx.mx_experts_layout_init(1, 1, 1), mx.lib()
    null = ctypes.c_void_p(None)
    calls = {
        "gather": lambda: lib.mx_experts_gather(P, null, null, 0, H, H, null, H, null),
        "gather_bwd": lambda: lib.mx_experts_gather_bwd(P, null, null, 0, H, H, null, H, null),
        "combine": lambda: lib.mx_experts_combine(P, null, null, 0, H, H, null, null, 0, H, null),
        "combine_bwd": lambda: lib.mx_experts_combine_bwd(P, null, null, null, 0, H, H, H, null, null, H, null, null),
    }
    for name, call in calls.items():
        assert call() == status, (name, mx.lib().mx_last_error())


def test_an_expert_layer_of_too_many_features():
    LW, P = mx.mx_fp4_layout_init(MOST + 1, 64), mx.mx_experts_layout_init(1, 1, 1)
    null = ctypes.c_void_p(None)
    st = mx.lib().mx_fp4_experts(LW, null, P, null, null, 0, 64, null, null, null, 0, MOST + 1, null, 0, None, null)
    assert st == UNSUPPORTED
