"""Operands at the ends of their types' range whose products are ordinary numbers: tiny activations (subnormal in bf16,
scale bytes down to 0 in MXFP4) times a large weight, and large ones times a tiny weight, in every path."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_layer import Layer, bf16, dev

pytestmark = pytest.mark.gpu


def ranged(n, base, up):
    """A layer whose X and dY are about 2^-up and whose weight is about 2^up."""
    g = np.random.default_rng(n + abs(up))
    rows, cols = 96, 288 if base == "mx" else 320
    layer = Layer(n, rows, cols, 0, base, seed=n)
    layer.X, layer.G = (bf16(np.ldexp(g.standard_normal(s), -up)) for s in ((n, cols), (n, rows)))
    layer.Xd, layer.Gd = dev(layer.X, torch.bfloat16), dev(layer.G, torch.bfloat16)
    W = np.ldexp(g.standard_normal((rows, cols)), up).astype(np.float32)
    if base == "mx":
        codes, byte = oracle.mx_quantize(W)
        packed, scales = oracle.mx_pack(codes, byte)
        layer.W = bf16(oracle.mx_values(codes, byte, cols))
        layer.kw = dict(packed=dev(packed, torch.uint8), scales=dev(scales, torch.uint8))
    else:
        codes, absmax = oracle.quantize_residual(W.ravel())
        layer.W = bf16(oracle.dequantize(codes, absmax, 64).reshape(rows, cols))
        layer.kw = dict(packed=dev(oracle.pack_nibbles(codes), torch.uint8), absmax=dev(absmax))
    return layer


@pytest.mark.parametrize("up", [100, 120, 125, -100, -120, -125])
@pytest.mark.parametrize("n", [3, 70])
@pytest.mark.parametrize("base", ["nf", "mx"])
def test_products_of_tiny_and_large(lib, base, n, up):
    layer = ranged(n, base, up)
    assert np.isfinite(layer.W).all() and layer.X.any() and layer.W.any()
    layer.check_forward(layer.forward(lib))
    layer.check_backward(layer.backward(lib, dx_dtype=torch.float32))
