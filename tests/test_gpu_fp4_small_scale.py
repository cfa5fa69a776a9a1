"""The quantiser at both ends of the matrix scale's range (2^-100 to 2^117), and around the limit below which
it scales a matrix up: values next to every boundary of the codes and of the block scales, against the
definition in 64 bits.  Codes and scales have to be equal."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
from mixed_precision_quantized_mx_b200 import binding as mx
from mixed_precision_quantized_mx_b200.layer import MicroscaledLinear

pytestmark = pytest.mark.gpu
E2M1 = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
E4M3 = [(2 * i + 1) * 2.0 ** -10 for i in range(8)] + [1 + (2 * i + 1) / 16 for i in range(8)] + [432.0]
EXPONENTS = (-100, -99, -97, -94, -92, -91, -90, -89, -60, 0, 100, 115, 116)


def near(v, offsets):
    """fp32 numbers next to v"""
    return (np.float32(v).view(np.int32) + np.asarray(offsets, np.int32)).view(np.float32)


def block_rows(g):
    """rows of 64 columns for one matrix scale"""
    rows, g = [], np.float32(g)
    with np.errstate(over="ignore"):
        for s in (2.0 ** -9, 3 * 2.0 ** -9, 1.125 * 2.0 ** -6, 1.0, 1.75, 256.0):
            d = np.float32(np.float32(s) * g)
            if not np.isfinite(np.float32(6) * d):
                continue
            row = np.zeros(64, np.float32)
            for i, t in enumerate(E2M1):
                row[16 * (i // 2) + 1 + 7 * (i % 2):][:7] = near(np.float32(t) * d, range(-3, 4))
            row[::16] = np.float32(6) * d                    # the block's largest: its scale is s
            rows += [row, -row]
        for t in E4M3:
            a = near(np.float32(t) * np.float32(np.float32(6) * g), (-2, -1, 0, 1))
            if np.isfinite(a).all():
                row = np.zeros(64, np.float32)
                row[::16] = a
                rows.append(row)
    return rows


@pytest.mark.parametrize("exponent", EXPONENTS)
def test_codes_and_scales(exponent):
    rng = np.random.default_rng(exponent + 200)
    m = np.concatenate([[0, 1, 2 ** 23 - 1, 2 ** 23 - 2], rng.integers(0, 2 ** 23, 60)])
    gs = ((1 + m * 2.0 ** -23) * 2.0 ** exponent).astype(np.float32)
    x = [block_rows(g) for g in gs]
    n = min(map(len, x))
    x = np.array([r[:n] for r in x])
    L = mx.mx_fp4_layout_init(n, 64, 0, len(gs))
    blob = torch.zeros(L.total_bytes, dtype=torch.uint8, device="cuda")
    mx.mx_fp4_quant(L, torch.tensor(x, device="cuda"), blob, gscale=torch.tensor(gs, device="cuda"))
    codes, sb, got, _ = ref.unpack(L, blob.cpu().numpy())
    assert np.array_equal(got, gs)                           # the stored scale is the one that was given
    for i, g in enumerate(gs):
        want, s = ref.quantise(x[i].astype(np.float64), 0, g)
        assert np.array_equal(ref.scale_values(sb[i, :, :4], 0), s), g
        assert np.array_equal(codes[i, :, :64], want), g


def test_saturated_blocks_of_a_small_scale():
    """values far beyond 448 * 6 g, up to the largest number: codes of size 6, the largest scale"""
    x = np.float32([[1e-20, -3e38, 1.0, 2.0 ** -85, -2.0 ** -88] + [0.0] * 11, [2.0 ** -87] * 8 + [-2.0 ** -89] * 8])
    for g in (2.0 ** -100, 1.5 * 2.0 ** -95):
        L = mx.mx_fp4_layout_init(2, 16, 0)
        blob = torch.zeros(L.total_bytes, dtype=torch.uint8, device="cuda")
        mx.mx_fp4_quant(L, torch.tensor(x, device="cuda"), blob, gscale=torch.tensor([g], device="cuda"))
        codes, sb, _, _ = ref.unpack(L, blob.cpu().numpy())
        want, s = ref.quantise(x.astype(np.float64), 0, g)
        assert np.array_equal(codes[0, :, :16], want) and np.array_equal(ref.scale_values(sb[0, :, :1], 0), s)


@pytest.mark.parametrize("exponent", [-100, -91])
def test_the_product_that_quantises_takes_the_same_codes(exponent):
    """up to 4 tokens the product's kernel quantises: the same outputs, bit for bit"""
    g = torch.tensor([1.9 * 2.0 ** exponent], device="cuda")
    rows = np.array(block_rows(float(g)))
    x = torch.tensor(np.tile(rows[:4], (1, 5)), device="cuda")
    layer = MicroscaledLinear(torch.randn(130, 320, device="cuda"), act_scale=g)
    LA = mx.mx_fp4_layout_init(4, 320, 0)
    blob = torch.empty(LA.total_bytes, dtype=torch.uint8, device="cuda")
    mx.mx_fp4_quant(LA, x, blob, gscale=g)
    Y = torch.empty(4, 130, device="cuda")
    mx.mx_fp4_gemm(layer.layout, layer.blob, LA, blob, Y)
    assert bool(Y.any()) and torch.equal(layer(x), Y)
