"""Pins of the oracle's dropout, MXFP4 and adapted-layer gradient."""
import numpy as np
import pytest

import oracle

M64 = (1 << 64) - 1


def _mix(z):
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & M64
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & M64
    return z ^ (z >> 31)


@pytest.mark.parametrize("seed,offset,p", [(0, 0, 0.5), (42, 7, 0.1), (2 ** 64 - 1, 2 ** 40, 0.9)])
def test_keep_mask_worked_with_python_integers(seed, offset, p):
    gamma = 0x9E3779B97F4A7C15
    key = _mix((seed + (offset + 1) * gamma) & M64)
    thr = oracle.drop_threshold(p)
    want = []
    for i in range(37):
        word = _mix((key + (i // 4 + 1) * gamma) & M64)
        want.append((word >> (16 * (i % 4))) % 65536 >= thr)
    assert oracle.keep_mask((37,), p, seed, offset).tolist() == want
    assert oracle.keep_mask((5,), p, seed, offset, first=11).tolist() == want[11:16]


def test_dropout_share_and_ends():
    n = 1 << 16
    for p in (0.05, 0.5):
        kept = oracle.keep_mask((n,), p, 3, 4).mean()
        # binomial: five standard deviations
        assert abs(kept - (1 - oracle.drop_threshold(p) / 65536)) < 5 * np.sqrt(p * (1 - p) / n)
    assert oracle.keep_mask((64,), 0.0, 1, 2).all() and oracle.drop_scale(0.0) == 1.0
    assert not oracle.keep_mask((64,), 1.0, 1, 2).any() and oracle.drop_scale(1.0) == 0.0
    assert oracle.drop_threshold(0.5) == 32768 and oracle.drop_scale(0.5) == 2.0
    assert (oracle.keep_mask((256,), 0.5, 1, 2) != oracle.keep_mask((256,), 0.5, 1, 3)).any()


def test_mx_rounding_at_every_midpoint():
    # the block's first element fixes the scale at 1 (largest magnitude 4)
    mids = [(0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0)]
    ulp = 2.0 ** -20
    x = [4.0]
    want = [4.0]
    for m, tie in mids[:-1]:
        below = max(v for v in oracle.E2M1 if v < m)
        above = min(v for v in oracle.E2M1 if v > m)
        x += [m, m - ulp, m + ulp, -m]
        want += [tie, below, above, -tie]
    R = np.zeros((1, 32), dtype=np.float32)
    R[0, :len(x)] = x
    codes, byte = oracle.mx_quantize(R)
    assert byte[0, 0] == 127
    assert oracle.mx_values(codes, byte, 32)[0, :len(x)].tolist() == want
    # 5 is a tie of 4 and 6 (even code: 4), 7.9 saturates at 6
    codes, byte = oracle.mx_quantize(np.array([[5.0, 5.0 + ulp, 7.9, -7.9]], dtype=np.float32))
    assert oracle.mx_values(codes, byte, 4)[0].tolist() == [4.0, 6.0, 6.0, -6.0]


@pytest.mark.parametrize("amax,byte", [(0.0, 0), (1.0, 125), (3.99, 126), (4.0, 127), (2.0 ** -126, 0), (2.0 ** -124, 1),
                                       (2.0 ** 127, 252), (3.4e38, 252), (1e-44, 0), (np.inf, 255), (np.nan, 255)])
def test_mx_scale_bytes(amax, byte):
    R = np.zeros((2, 33), dtype=np.float32)
    R[1, 32] = -amax
    got = oracle.mx_scale_bytes(R)
    assert got.shape == (2, 8) and got[1, 1] == byte and got[0].max() == 0 and got[1, 0] == 0


def test_mx_round_trip_and_storage():
    g = np.random.default_rng(5)
    codes = g.integers(0, 16, (3, 512)).astype(np.uint8)
    codes[:, ::32] = codes[:, ::32] & 8 | 6   # magnitude 4 in each block: the scale comes back
    byte = g.integers(1, 250, (3, 16)).astype(np.uint8)
    v = oracle.mx_values(codes, byte, 512).astype(np.float32)
    c2, b2 = oracle.mx_quantize(v)
    assert np.array_equal(b2, byte) and np.array_equal(oracle.mx_values(c2, b2, 512), v)
    packed, scales = oracle.mx_pack(codes, byte)
    assert packed[0, 0] == codes[0, 0] << 4 | codes[0, 1] and scales.shape == (2, 3, 8) and scales[1, 2, 3] == byte[2, 11]
    c3, b3 = oracle.mx_unpack(packed, scales)
    assert np.array_equal(c3, codes) and np.array_equal(b3, byte)


@pytest.mark.parametrize("masked", [False, True])
def test_layer_backward_against_differences(masked):
    g = np.random.default_rng(6)
    n, rows, cols, r, gain = 5, 7, 9, 3, 1.7
    X, W, A, B, G = (g.standard_normal(s) for s in ((n, cols), (rows, cols), (r, cols), (rows, r), (n, rows)))
    keep = oracle.keep_mask((n, cols), 0.5, 1, 2) if masked else None
    loss = lambda X, A, B: float((G * oracle.layer_forward(X, W, A, B, gain, keep)).sum())   # noqa: E731
    dX, dB, dA = oracle.layer_backward(G, X, W, A, B, gain, keep)
    # the forward is linear in each argument: a step of 1 gives the derivative itself
    for arg, grad in ((0, dX), (1, dA), (2, dB)):
        for i in range(grad.shape[0]):
            for j in range(grad.shape[1]):
                args = [X, A, B]
                args[arg] = args[arg].copy()
                args[arg][i, j] += 1.0
                assert abs(loss(*args) - loss(X, A, B) - grad[i, j]) < 1e-10
