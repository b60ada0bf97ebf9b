"""Where an infinity or a NaN of X or dY goes: into every output whose formula it enters, and into no other.  keep()
puts a zero in the place of what it drops; the formulas' other factors meet that zero as any other."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_layer import Layer, host

pytestmark = pytest.mark.gpu
N, ROWS, COLS, R = 40, 64, 128, 8
RNG = dict(p=0.5, seed=1, offset=2)
BAD = [float("nan"), float("inf"), float("-inf")]


@pytest.fixture(params=["nf", "mx"])
def layer(lib, request):
    return Layer(N, ROWS, COLS, R, request.param, seed=7)


def replaced(t, at, value):
    t = t.clone()
    t[at] = value
    return t


@pytest.mark.parametrize("bad", BAD)
def test_in_dy(lib, layer, bad):
    keep = oracle.keep_mask((N, COLS), **RNG)
    clean = layer.backward(lib, dx_dtype=torch.float32, **RNG)
    layer.Gd, layer.G = replaced(layer.Gd, (3, 5), bad), layer.G.copy()
    layer.G[3, 5] = bad
    dX, dB, dA = layer.backward(lib, dx_dtype=torch.float32, **RNG)
    tokens, features = torch.arange(N, device="cuda") != 3, torch.arange(ROWS, device="cuda") != 5
    assert not torch.isfinite(dX[3]).any() and torch.equal(dX[tokens], clean[0][tokens])
    assert not torch.isfinite(dB[5]).any() and torch.equal(dB[features], clean[1][features])
    # every rank of the row of dY B is infinite or NaN: so is all of dA, and NaN where X is dropped
    kept = torch.from_numpy(keep[3]).cuda()
    assert not torch.isfinite(dA).any() and torch.isnan(dA[:, ~kept]).all()
    with np.errstate(invalid="ignore"):
        want = oracle.layer_backward(layer.G, layer.X, layer.W, layer.A, layer.B, 1.5 * oracle.drop_scale(0.5), keep)
    for got, ref in zip((dX, dB, dA), want):
        assert np.array_equal(np.isfinite(host(got)), np.isfinite(ref))


@pytest.mark.parametrize("bad", BAD)
def test_in_x(lib, layer, bad):
    keep = oracle.keep_mask((N, COLS), **RNG)
    c = int(np.flatnonzero(keep[11])[0])
    Y0, clean = layer.forward(lib, **RNG), layer.backward(lib, **RNG)
    layer.Xd = replaced(layer.Xd, (11, c), bad)
    Y, (dX, dB, dA) = layer.forward(lib, **RNG), layer.backward(lib, **RNG)
    tokens, columns = torch.arange(N, device="cuda") != 11, torch.arange(COLS, device="cuda") != c
    assert not torch.isfinite(Y[11]).any() and torch.equal(Y[tokens], Y0[tokens])
    assert torch.equal(dX, clean[0])                                            # X is no factor of dX
    assert not torch.isfinite(dB).any()                                         # its token's row of X A^T is in all of dB
    assert not torch.isfinite(dA[:, c]).any() and torch.equal(dA[:, columns], clean[2][:, columns])


@pytest.mark.parametrize("bad", BAD)
def test_in_x_where_it_is_dropped(lib, layer, bad):
    keep = oracle.keep_mask((N, COLS), **RNG)
    c = int(np.flatnonzero(~keep[11])[0])
    Y0, clean = layer.forward(lib, **RNG), layer.backward(lib, **RNG)
    layer.Xd = replaced(layer.Xd, (11, c), bad)
    Y, grads = layer.forward(lib, **RNG), layer.backward(lib, **RNG)
    assert all(torch.equal(a, b) for a, b in zip(grads, clean))
    tokens = torch.arange(N, device="cuda") != 11   # the base reads X undropped
    assert not torch.isfinite(Y[11]).any() and torch.equal(Y[tokens], Y0[tokens])
