"""Host side of the microscaled layers, on the CPU: the entry points are replaced by fakes."""
import struct

import pytest
import torch

from mixed_precision_quantized_mx_b200 import binding as mx
from mixed_precision_quantized_mx_b200 import layer as layers


def blob(rows, K, groups):
    L = mx.mx_fp4_layout_init(rows, K, mx.FP4_E4M3_16, groups)
    header = struct.pack("<6I", 0x34465845, 1, rows, K, mx.FP4_E4M3_16, groups)
    b = torch.zeros(L.total_bytes, dtype=torch.uint8)
    b[:len(header)] = torch.tensor(list(header), dtype=torch.uint8)
    return b


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("mx_fp4_linear", "mx_fp4_linear_sorted", "mx_fp4_experts"):
        monkeypatch.setattr(mx, name, lambda *a, _name=name, **k: seen.append((_name, a, k)))
    return seen


def test_what_a_layer_keeps_by_size_is_bounded(calls, monkeypatch):
    monkeypatch.setattr(layers, "KEPT_SIZES", 16)
    linear = layers.MicroscaledLinear.from_blob(blob(40, 100, 1))
    experts = layers.MicroscaledExperts.from_blob(blob(40, 100, 3))
    for T in list(range(1, 60)) + [5, 59, 1]:
        linear(torch.zeros(T, 100))
        experts(torch.zeros(T, 100), torch.zeros(T, 2, dtype=torch.int32), torch.zeros(T, 2))
        assert 1 <= len(linear._sizes) <= 16 and 1 <= len(experts._sizes) <= 16
    # the sizes that the calls got are those of their own tokens
    for name, a, _ in calls:
        if name == "mx_fp4_linear":
            need = mx.mx_fp4_linear_workspace_size(linear.layout, a[2].shape[0])
            assert (a[4].numel() if a[4] is not None else 0) == need
        else:
            P = a[2]
            assert P.T == a[4].shape[0] and a[7].numel() == mx.mx_fp4_experts_workspace_size(experts.layout, P)


def test_every_call_gets_the_layers_status_word(calls):
    linear = layers.MicroscaledLinear.from_blob(blob(40, 100, 1))
    experts = layers.MicroscaledExperts.from_blob(blob(40, 100, 3))
    linear(torch.zeros(7, 100))
    experts(torch.zeros(7, 100), torch.zeros(7, 2, dtype=torch.int32), torch.zeros(7, 2))
    P = mx.mx_experts_layout_init(7, 2, 3)
    plan = mx.ExpertsPlan(P, buffer=torch.zeros(P.total_bytes, dtype=torch.uint8))
    experts.project(torch.zeros(7, 100), plan)
    assert [c[0] for c in calls] == ["mx_fp4_linear", "mx_fp4_experts", "mx_fp4_linear_sorted"]
    for (_, _, k), layer in zip(calls, (linear, experts, experts)):
        assert k["status"] is layer._status
    layer = experts
    layer.check_status()
    layer._status.fill_(5)
    with pytest.raises(mx.MXError) as e:
        layer.check_status()
    assert e.value.status == 5 and int(layer._status) == 0
