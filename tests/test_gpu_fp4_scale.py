"""The 16-column format's matrix scale as the layers take it by default, and layers of random sizes against
the definition in 64 bits: scale bits, stored blob and outputs.

The last bit of the scale matters: with bf16 weights a / (6 g) is a ratio of two 8-bit numbers times 448, so
many blocks lie on a tie of E4M3 or next to one.  Products are off by at most (K / 64 + 64) 2^-23 S for sums of
size S = sum |a w| (a step of the tensor core adds 64 products and the accumulator), plus half a step of the
output's type.
"""
import numpy as np
import pytest
import torch

import fp4_reference as ref
from mixed_precision_quantized_mx_b200 import binding as mx
from mixed_precision_quantized_mx_b200.layer import MicroscaledExperts, MicroscaledLinear

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# bf16 maxima (significand of 128 .. 255) whose quotient by 2688 and product with fl(1 / 2688) differ
SIGNIFICANDS = (132, 140, 228, 244, 254)


def quotient(m):
    return np.float32(m) / np.float32(2688)


def product(m):
    return np.float32(m) * (np.float32(1) / np.float32(2688))


def weights(seed, N, K, significand):
    """normal bf16 weights whose largest is significand * 2^-10"""
    w = np.clip(np.random.default_rng(seed).standard_normal((N, K)) * 0.02, -0.1, 0.1)
    w[N // 2, K // 3] = -significand * 2.0 ** -10
    t = torch.tensor(w, dtype=torch.bfloat16, device="cuda")
    return t, t.double().cpu().numpy()


def check_blob(L, blob, ws, scales):
    codes, sb, g, _ = ref.unpack(L, blob.cpu().numpy())
    assert np.array_equal(g, np.asarray(scales, np.float32))
    for i, w in enumerate(ws):
        want, s = ref.quantise(w, L.format, scales[i])
        nb = s.shape[1]
        assert np.array_equal(codes[i, :, :L.K], want), i
        assert np.array_equal(ref.scale_values(sb[i, :, :nb], L.format), s), i


def check_output(Y, x, w, K, weight=1.0):
    want, S = weight * (x @ w.T), weight * (np.abs(x) @ np.abs(w).T)
    fi = torch.finfo(Y.dtype)
    tol = (K / 64 + 64) * 2.0 ** -23 * S
    tol = tol + fi.eps / 2 * (np.abs(want) + tol) + fi.smallest_normal * fi.eps
    err = np.abs(Y.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("significand", SIGNIFICANDS)
def test_a_linear_layer_takes_the_quotient(significand):
    N, K = 260, 2048
    t, w = weights(significand, N, K, significand)
    g = quotient(np.abs(w).max())
    assert g != product(np.abs(w).max())
    layer = MicroscaledLinear(t, act_scale=torch.tensor([0.004], device="cuda"))
    check_blob(layer.layout, layer.blob, [w], [g])
    for M in (1, 9):
        x = torch.tensor(np.random.default_rng(M).standard_normal((M, K)), dtype=torch.float32, device="cuda")
        xv = ref.values(x.double().cpu().numpy(), 0, np.float32(0.004))
        check_output(layer(x), xv, ref.values(w, 0, g), K)


def test_a_layer_of_experts_takes_each_quotient():
    N, K = 140, 1024
    both = [weights(s + 1000, N, K, s) for s in SIGNIFICANDS]
    ws = [w for _, w in both]
    g = [quotient(np.abs(w).max()) for w in ws]
    # whether the last bit shows in block scales goes by the maximum: for some of these it does
    assert any((ref.quantise(w, 0, a)[1] != ref.quantise(w, 0, product(np.abs(w).max()))[1]).any() for w, a in zip(ws, g))
    layer = MicroscaledExperts(torch.stack([t for t, _ in both]), act_scale=torch.tensor([0.004], device="cuda"))
    check_blob(layer.layout, layer.blob, ws, g)
    E = len(ws)
    x = torch.tensor(np.random.default_rng(3).standard_normal((E, K)), dtype=torch.float32, device="cuda")
    ids = torch.arange(E, dtype=torch.int32, device="cuda")[:, None]
    xv = ref.values(x.double().cpu().numpy(), 0, np.float32(0.004))
    Y = layer(x, ids, torch.full((E, 1), 0.5, device="cuda"))      # half of a sum is exact
    for e in range(E):
        check_output(Y[e:e + 1], xv[e:e + 1], ref.values(ws[e], 0, g[e]), K, 0.5)


@pytest.mark.parametrize("seed", range(16))
def test_layers_of_random_sizes(seed):
    """codes, scales and outputs against the definition, none of them taken from the library's own quantiser"""
    rng = np.random.default_rng(seed)
    fmt, dt = seed % 2, list(TYPES)[seed % 3]
    M, N, K = (int(np.exp(rng.uniform(np.log(a), np.log(b)))) for a, b in ((1, 300), (1, 600), (1, 3000)))
    t = torch.tensor(rng.standard_normal((N, K)) * 0.02, dtype=TYPES[dt], device="cuda")
    x = torch.tensor(rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.01, 20, 1), dtype=TYPES[dt], device="cuda")
    w, xn = t.double().cpu().numpy(), x.double().cpu().numpy()
    ga, gw = (np.float32(np.abs(xn).max() / 2688), quotient(np.abs(w).max())) if fmt == 0 else (np.float32(1), np.float32(1))
    layer = MicroscaledLinear(t, fmt, act_scale=torch.tensor([ga], device="cuda") if fmt == 0 else None)
    check_blob(layer.layout, layer.blob, [w], [gw])
    LA = mx.mx_fp4_layout_init(M, K, fmt)
    blob = torch.empty(LA.total_bytes, dtype=torch.uint8, device="cuda")
    mx.mx_fp4_quant(LA, x, blob, gscale=layer.act_scale)
    check_blob(LA, blob, [xn], [ga])
    check_output(layer(x, out_dtype=torch.float32), ref.values(xn, fmt, ga), ref.values(w, fmt, gw), K)
