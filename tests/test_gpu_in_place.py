"""Calls whose output may be their input give, in place, what they give beside it."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 5, 8, 4096, (1 << 24) + 13])   # the last: several rounds of the grid
def test_dropout_in_place(lib, n, dtype):
    X = torch.randn(n, device="cuda").to(dtype)
    want = lib.loftq_dropout(X, 0.4, 9, 1)
    assert lib.loftq_dropout(X, 0.4, 9, 1, out=X) is X and torch.equal(X, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 256), (7, 1003), (1000, 4100)])
def test_residual_in_place(lib, rows, cols, dtype):
    W = torch.randn(rows, cols, device="cuda").to(dtype)
    packed, scales = lib.loftq_mxfp4_quantize(W)
    want = lib.loftq_mxfp4_dequantize(packed, scales, (rows, cols), W=W, out_dtype=dtype)
    got = lib.loftq_mxfp4_dequantize(packed, scales, (rows, cols), W=W, out=W)
    assert got is W and torch.equal(W, want)
