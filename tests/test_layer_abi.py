"""Refusals of the training and serving calls: every one is made before anything is
enqueued (no GPU needed), through the C ABI and through the binding's own checks."""
import ctypes

import pytest
import torch

FAKE = 0x10000   # aligned, never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BIG = 1 << 40


@pytest.fixture(scope="module")
def b():
    from loftq_qlora_initialization_amd import binding
    return binding


def drop(b, p=0.1, step=None):
    return ctypes.byref(b.LoftqDropout(p, 1, 2, step))


def test_dropout_refusals(b):
    f = b._c_dropout
    assert f(FAKE, 2, 8, drop(b), FAKE, None) == INVALID            # dtype
    assert f(FAKE, 0, -1, drop(b), FAKE, None) == INVALID           # n
    assert f(FAKE, 0, 8, None, FAKE, None) == INVALID               # no dropout given
    assert f(None, 0, 8, drop(b), FAKE, None) == INVALID
    assert f(FAKE + 4, 0, 8, drop(b), FAKE, None) == INVALID        # misaligned
    assert f(FAKE, 0, 8, drop(b, step=FAKE + 4), FAKE, None) == INVALID
    for p in (-0.1, 1.5, float("nan"), float("inf")):
        assert f(FAKE, 0, 8, drop(b, p), FAKE, None) == INVALID
    assert f(None, 0, 0, drop(b), None, None) == OK                 # nothing to do


def fwd(b, mx, n=16, rows=64, cols=128, packed=FAKE, scale=FAKE, qa=None, qs=None, bits=4, B=FAKE, A=FAKE, r=8, alpha=1.0,
        drop=None, X=FAKE, Y=FAKE, ydt=0, ws=FAKE, ws_bytes=BIG):
    base = (packed, scale) if mx else (packed, scale, qa, qs, bits)
    f = b._c_mx_fwd if mx else b._c_fwd_drop
    return f(X, n, rows, cols, *base, B, A, r, alpha, drop, Y, ydt, ws, ws_bytes, None)


def bwd(b, mx, n=16, rows=64, cols=128, packed=FAKE, scale=FAKE, qa=None, qs=None, bits=4, B=FAKE, A=FAKE, r=8, alpha=1.0,
        drop=None, dY=FAKE, X=FAKE, dX=FAKE, xdt=1, dB=FAKE, dA=FAKE, ws=FAKE, ws_bytes=BIG):
    base = (packed, scale) if mx else (packed, scale, qa, qs, bits)
    f = b._c_mx_bwd if mx else b._c_bwd
    return f(dY, X, n, rows, cols, *base, B, A, r, alpha, drop, dX, xdt, dB, dA, ws, ws_bytes, None)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("call", [fwd, bwd])
def test_layer_refusals(b, call, mx):
    def bad(**kw):
        return call(b, mx, **kw)
    for kw in (dict(n=-1), dict(n=1 << 31), dict(rows=-1), dict(rows=1 << 31), dict(packed=None), dict(packed=FAKE + 8),
               dict(scale=None), dict(scale=FAKE + 8), dict(B=None), dict(A=None), dict(B=FAKE + 4), dict(r=0),
               dict(alpha=float("nan")), dict(alpha=float("inf")), dict(X=None), dict(X=FAKE + 2), dict(ws=None),
               dict(ws=FAKE + 8), dict(alpha=3e38, drop=drop(b, 0.9)), dict(drop=drop(b, 2.0)), dict(drop=drop(b, step=FAKE + 4))):
        assert bad(**kw) == INVALID, kw
    for kw in (dict(r=65), dict(cols=0), dict(cols=100), dict(cols=16), dict(n=(1 << 31) - 1, rows=1 << 20),
               dict(cols=1 << 22)):
        assert bad(**kw) == UNSUPPORTED, kw
    assert bad(ws_bytes=255) == WORKSPACE
    if not mx:
        assert bad(bits=5) == UNSUPPORTED and bad(cols=96) == UNSUPPORTED
        assert bad(qa=FAKE) == INVALID and bad(qs=FAKE) == INVALID
        assert bad(qa=FAKE + 8, qs=FAKE) == INVALID


@pytest.mark.parametrize("mx", [False, True])
def test_forward_and_backward_outputs(b, mx):
    assert fwd(b, mx, Y=None) == INVALID and fwd(b, mx, Y=FAKE + 4) == INVALID and fwd(b, mx, ydt=2) == INVALID
    assert fwd(b, mx, n=0) == OK and fwd(b, mx, rows=0) == OK       # nothing to write
    assert bwd(b, mx, dY=None) == INVALID and bwd(b, mx, dY=FAKE + 2) == INVALID
    assert bwd(b, mx, dB=None) == INVALID and bwd(b, mx, dA=None) == INVALID and bwd(b, mx, dA=FAKE + 4) == INVALID
    assert bwd(b, mx, dX=FAKE + 4) == INVALID and bwd(b, mx, xdt=3) == INVALID
    assert bwd(b, mx, dX=None, dB=None, dA=None) == INVALID         # nothing asked for
    assert bwd(b, mx, B=None, A=None) == INVALID                    # gradients of no adapter
    assert bwd(b, mx, rows=0) == UNSUPPORTED and bwd(b, mx, rows=1 << 22) == UNSUPPORTED
    assert bwd(b, mx, n=0, dB=None, dA=None) == OK


@pytest.mark.parametrize("mx", [False, True])
def test_workspace_queries(b, mx):
    f = b.mxfp4_forward_workspace_bytes if mx else b.qlora_forward_dropout_workspace_bytes
    g = b.mxfp4_backward_workspace_bytes if mx else b.qlora_backward_workspace_bytes
    for q in (f, g):
        assert q(-1, 64, 64, 8) == 0 and q(16, -1, 64, 8) == 0 and q(16, 64, 64, 65) == 0 and q(1 << 31, 64, 64, 8) == 0
        need = q(100, 320, 192, 16)
        assert need > 0 and need <= q(101, 320, 192, 16) and need < q(100, 640, 192, 16)
    call = fwd
    need = f(16, 64, 128, 8)
    assert call(b, mx, ws_bytes=need - 1) == WORKSPACE
    assert bwd(b, mx, ws_bytes=g(16, 64, 128, 8) - 1) == WORKSPACE


def test_mxfp4_refusals(b):
    q, d = b._c_mx_quant, b._c_mx_deq
    assert q(FAKE, 2, 4, 4, None, None, 0, FAKE, FAKE, None) == INVALID
    assert q(FAKE, 0, -4, 4, None, None, 0, FAKE, FAKE, None) == INVALID
    assert q(None, 0, 4, 4, None, None, 0, FAKE, FAKE, None) == INVALID
    assert q(FAKE, 0, 4, 4, None, None, 0, FAKE + 8, FAKE, None) == INVALID
    assert q(FAKE, 0, 4, 4, FAKE, None, 4, FAKE, FAKE, None) == INVALID
    assert q(FAKE, 0, 4, 4, FAKE, FAKE, 0, FAKE, FAKE, None) == INVALID
    assert q(FAKE, 0, (1 << 31) - 1, 1 << 20, None, None, 0, FAKE, FAKE, None) == UNSUPPORTED
    assert q(None, 0, 0, 4, None, None, 0, None, None, None) == OK
    assert d(FAKE, FAKE, 4, 4, None, 0, FAKE, 2, None) == INVALID
    assert d(FAKE, FAKE, 4, 4, FAKE, 5, FAKE, 0, None) == INVALID
    assert d(FAKE, None, 4, 4, None, 0, FAKE, 0, None) == INVALID
    assert d(FAKE, FAKE, 4, 4, None, 0, FAKE + 4, 0, None) == INVALID
    assert d(FAKE, FAKE, (1 << 31) - 1, 1 << 20, None, 0, FAKE, 0, None) == UNSUPPORTED
    assert d(None, None, 4, 0, None, 0, None, 0, None) == OK
    assert b._c_mx_packed(3, 257) == 3 * 256 and b._c_mx_scales(3, 257) == 3 * 16
    assert b._c_mx_packed(-1, 4) == 0 and b._c_mx_scales(1, -4) == 0


def test_binding_refuses_host_tensors(b):
    X = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        b.loftq_dropout(X, 0.1, 1)
    with pytest.raises(ValueError):
        b.loftq_mxfp4_quantize(X)
    with pytest.raises(ValueError):
        b.loftq_qlora_forward_dropout(X, X, (64, 64), absmax=X)
    with pytest.raises(ValueError):
        b.loftq_mxfp4_backward(X, X, X, X, (64, 64))
