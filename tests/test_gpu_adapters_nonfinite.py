"""Where an infinity or a NaN of a token goes in a pool whose slots have ranks of their own: into every output whose
formula it enters, and into no other.  What lies past a slot's own rank enters no formula, so the gradients there
stay zeros, and a slot of rank 0 adds nothing, whatever its tokens hold."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_adapters import Batch, dev, host

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), float("-inf")]


def pool(n, rank, seed):
    """Slots of rank 0, 1, 5 and all of them, with tokens in each."""
    b = Batch(n, 72, 136, 4, rank, ids="0", seed=seed)
    b.ids = np.arange(n) % 4
    b.idd = dev(b.ids, torch.int32)
    b.ranks = np.array([0, 1, 5, rank])
    b.rd = dev(b.ranks, torch.int32)
    return b


def past(b, slot):
    return int(b.ranks[slot])


# one tile for each slot, whose partial sums are added where they are read, or once before; several chunks of a slot
@pytest.mark.parametrize("n", [12, 290, 3000])
@pytest.mark.parametrize("rank", [16, 24])
@pytest.mark.parametrize("slot", [0, 1, 2, 3])
@pytest.mark.parametrize("bad", BAD)
def test_in_x(lib, n, rank, slot, bad):
    b = pool(n, rank, seed=21)
    plan = b.plan(lib)
    Y, (dX, dB, dA) = b.forward(lib, plan), b.backward(lib, plan)
    token, r = 4 + slot, past(b, slot)
    b.X[token, 9] = bad
    b.Xd[token, 9] = bad
    Y1, (dX1, dB1, dA1) = b.forward(lib, plan), b.backward(lib, plan)
    others = torch.arange(n, device="cuda") != token
    assert torch.equal(Y1[others], Y[others]) and torch.equal(dX1, dX)
    if r == 0:
        assert torch.equal(Y1, Y)
    rest = [s for s in range(4) if s != slot]
    assert torch.equal(dB1[rest], dB[rest]) and torch.equal(dA1[rest], dA[rest])
    assert not dB1[slot, :, r:].any() and not dA1[slot, r:].any()
    columns = torch.arange(136, device="cuda") != 9
    assert torch.equal(dA1[slot][:, columns], dA[slot][:, columns])
    with np.errstate(invalid="ignore"):
        ref_y = oracle.adapters_forward(b.X, b.B, b.A, b.ids, b.gains * 1.5, b.ranks, None, b.Y0)
        _, ref_b, ref_a = oracle.adapters_backward(b.G, b.X, b.B, b.A, b.ids, b.gains * 1.5, b.ranks, None, b.dX0)
    for got, ref in ((Y1, ref_y), (dB1, ref_b), (dA1, ref_a)):
        assert np.array_equal(np.isfinite(host(got)), np.isfinite(ref))


@pytest.mark.parametrize("n", [12, 290, 3000])
@pytest.mark.parametrize("rank", [16, 24])
@pytest.mark.parametrize("slot", [0, 1, 2, 3])
@pytest.mark.parametrize("bad", BAD)
def test_in_dy(lib, n, rank, slot, bad):
    b = pool(n, rank, seed=22)
    plan = b.plan(lib)
    dX, dB, dA = b.backward(lib, plan)
    token, r = 4 + slot, past(b, slot)
    b.G[token, 9] = bad
    b.Gd[token, 9] = bad
    dX1, dB1, dA1 = b.backward(lib, plan)
    others = torch.arange(n, device="cuda") != token
    assert torch.equal(dX1[others], dX[others])
    if r == 0:
        assert torch.equal(dX1, dX)
    rest = [s for s in range(4) if s != slot]
    assert torch.equal(dB1[rest], dB[rest]) and torch.equal(dA1[rest], dA[rest])
    assert not dB1[slot, :, r:].any() and not dA1[slot, r:].any()
    with np.errstate(invalid="ignore"):
        ref = oracle.adapters_backward(b.G, b.X, b.B, b.A, b.ids, b.gains * 1.5, b.ranks, None, b.dX0)
    for got, want in zip((dX1, dB1, dA1), ref):
        assert np.array_equal(np.isfinite(host(got)), np.isfinite(want))
