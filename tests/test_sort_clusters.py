"""The sort's cluster: 16 CTAs only where the device can place them, else 8, with the same plan."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_reference as ref
from mixed_precision_quantized_mx_b200 import binding as mx


def internal(name, argtypes):
    """a C++ function of the library that no header exports"""
    f = getattr(mx.lib(), name)
    f.restype, f.argtypes = ctypes.c_int, argtypes
    return f


def ctas(n, wide):
    return internal("_ZN2mx9sort_ctasEib", [ctypes.c_int, ctypes.c_bool])(n, wide)


def test_the_largest_cluster_goes_by_the_device():
    sizes = (0, 1, 1024, 1025, 2049, 4097, 16384, 16385, 70001, 1 << 24)
    assert [ctas(n, True) for n in sizes] == [1, 1, 1, 2, 4, 8, 8, 16, 16, 16]
    assert [ctas(n, False) for n in sizes] == [1, 1, 1, 2, 4, 8, 8, 8, 8, 8]


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E", [(16385, 1, 1024), (70001, 1, 33), (20000, 8, 256)])
@pytest.mark.parametrize("cluster", [1, 8])
def test_fewer_ctas_give_the_same_plan(T, k, E, cluster):
    ids = np.random.default_rng(T).integers(-1, E + 1, (T, k)).astype(np.int32)
    t = torch.tensor(ids, device="cuda")
    plan = mx.ExpertsPlan(mx.mx_experts_layout_init(T, k, E))
    mx.mx_experts_sort(plan, t)
    whole = plan.buffer.clone()
    plan.buffer.fill_(0x55)
    p = ctypes.c_void_p
    sort = internal("_ZN2mx22launch_experts_sort_onERK17mx_experts_layoutPKiPviP11CUstream_st",
                    [ctypes.POINTER(mx.ExpertsLayout), p, p, ctypes.c_int, p])
    assert sort(plan.P, t.data_ptr(), plan.ptr, cluster, torch.cuda.current_stream().cuda_stream) == 0
    got = (plan.order, plan.pos, plan.dest, plan.offsets, plan.tiles)
    for a, want in zip(got, ref.sort_slots(ids.ravel(), E)):
        assert np.array_equal(a.cpu().numpy(), want)
    other = mx.ExpertsPlan(plan.P, buffer=whole)
    for a, b in zip(got, (other.order, other.pos, other.dest, other.offsets, other.tiles)):
        assert torch.equal(a, b)
