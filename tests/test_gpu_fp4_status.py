"""A wait that runs out inside a kernel, as a user of the layers sees it: the call returns, check_status raises
once, and the layer works on.  The waits run out because no copies are issued (test_stall), after 20 ms."""
import functools

import pytest
import torch

from mixed_precision_quantized_mx_b200 import MXError
from mixed_precision_quantized_mx_b200 import binding as mx
from mixed_precision_quantized_mx_b200.layer import MicroscaledExperts, MicroscaledLinear

pytestmark = pytest.mark.gpu
TIMEOUT = 5                                      # MX_ERR_TIMEOUT


def stalled(monkeypatch, name):
    """the layer's own call of the entry point, without copies in its kernels"""
    monkeypatch.setattr(mx, name, functools.partial(getattr(mx, name), wait_timeout_us=20000, test_stall=1))


def check(layer, call, monkeypatch, entry):
    want = call()
    layer.check_status()
    with monkeypatch.context() as m:
        stalled(m, entry)
        call()
    with pytest.raises(MXError) as e:
        layer.check_status()
    assert e.value.status == TIMEOUT
    layer.check_status()                         # said once
    assert torch.equal(call(), want)
    layer.check_status()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,path", [(2, 0), (40, 0), (300, 2)])
def test_linear(fmt, M, path, monkeypatch):
    layer = MicroscaledLinear(torch.randn(300, 2048, device="cuda"), fmt)
    x = torch.randn(M, 2048, device="cuda")
    check(layer, lambda: layer(x, path=path), monkeypatch, "mx_fp4_linear")


@pytest.mark.parametrize("T", [2, 100])
def test_experts(T, monkeypatch):
    layer = MicroscaledExperts(torch.randn(4, 300, 1024, device="cuda"))
    x, w = torch.randn(T, 1024, device="cuda"), torch.rand(T, 2, device="cuda")
    ids = torch.randint(0, 4, (T, 2), dtype=torch.int32, device="cuda")
    check(layer, lambda: layer(x, ids, w), monkeypatch, "mx_fp4_experts")
    plan = layer.sort(ids)
    check(layer, lambda: layer.project(x, plan), monkeypatch, "mx_fp4_linear_sorted")


def test_a_captured_call_reports_to_its_layer(monkeypatch):
    layer = MicroscaledLinear(torch.randn(300, 1024, device="cuda"))
    other = MicroscaledLinear.from_blob(layer.blob)
    x = torch.randn(8, 1024, device="cuda")
    layer(x)
    g = torch.cuda.CUDAGraph()
    with monkeypatch.context() as m:
        stalled(m, "mx_fp4_linear")
        with torch.cuda.graph(g):
            layer(x)
    layer.check_status()                         # captured, not run
    g.replay()
    other.check_status()                         # each layer has a word of its own
    with pytest.raises(MXError):
        layer.check_status()
