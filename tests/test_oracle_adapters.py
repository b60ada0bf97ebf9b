"""Pins of the oracle for many adapters beside one weight and for the AdamW step."""
import numpy as np
import pytest
import torch

import oracle


def case(seed, n=23, rows=17, cols=24, slots=3, rank=5):
    g = np.random.default_rng(seed)
    return dict(X=g.standard_normal((n, cols)), G=g.standard_normal((n, rows)), B=g.standard_normal((slots, rows, rank)),
                A=g.standard_normal((slots, rank, cols)), slot_of=g.integers(-1, slots + 1, n), gains=g.standard_normal(slots),
                keep=g.random((n, cols)) < 0.7)


def test_plan_by_hand():
    starts, order = oracle.adapters_plan(np.array([2, -1, 0, 2, 7, 0, 2]), 3)
    assert starts.tolist() == [0, 2, 2, 5, 7] and order.tolist() == [2, 5, 0, 3, 6, 1, 4]


def test_one_slot_is_the_layer_without_its_base():
    c = case(1, slots=1)
    c["slot_of"][:] = 0
    W = np.zeros((17, 24))
    Y = oracle.layer_forward(c["X"], W, c["A"][0], c["B"][0], c["gains"][0], c["keep"])
    assert np.allclose(oracle.adapters_forward(c["X"], c["B"], c["A"], c["slot_of"], c["gains"], keep=c["keep"]), Y)
    want = oracle.layer_backward(c["G"], c["X"], W, c["A"][0], c["B"][0], c["gains"][0], c["keep"])
    got = oracle.adapters_backward(c["G"], c["X"], c["B"], c["A"], c["slot_of"], c["gains"], keep=c["keep"])
    assert np.allclose(got[0], want[0]) and np.allclose(got[1][0], want[1]) and np.allclose(got[2][0], want[2])


def test_gradient_against_differences():
    c = case(2)
    ranks = np.array([5, 2, 0])

    def loss(**moved):
        args = {**{k: c[k] for k in ("X", "B", "A", "slot_of", "gains", "keep")}, **moved}
        return (c["G"] * oracle.adapters_forward(ranks=ranks, **args)).sum()

    dX, dB, dA = oracle.adapters_backward(c["G"], c["X"], c["B"], c["A"], c["slot_of"], c["gains"], ranks, c["keep"])
    g, h = np.random.default_rng(3), 1e-6
    for name, grad in (("X", dX), ("B", dB), ("A", dA)):
        d = g.standard_normal(grad.shape)
        change = (loss(**{name: c[name] + h * d}) - loss(**{name: c[name] - h * d})) / (2 * h)
        assert abs(change - (grad * d).sum()) <= 1e-6 * np.abs(grad * d).sum() + 1e-6


@pytest.mark.parametrize("decay,norm", [(0.0, None), (0.1, 0.5)])
def test_adamw_is_torchs(decay, norm):
    g = torch.Generator().manual_seed(4)
    ps = [torch.randn(n, generator=g, dtype=torch.float64) for n in (7, 300)]
    ours = [[p.numpy().copy(), np.zeros(p.numel()), np.zeros(p.numel())] for p in ps]
    opt = torch.optim.AdamW(ps, lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=decay, foreach=False)
    for t in range(1, 4):
        grads = [torch.randn(p.shape, generator=g, dtype=torch.float64) for p in ps]
        clip = 1.0
        if norm is not None:
            _, clip = oracle.adamw_clip([x.numpy() for x in grads], norm)
        for p, x in zip(ps, grads):
            p.grad = x.clone()
        if norm is not None:
            torch.nn.utils.clip_grad_norm_(ps, norm)
        opt.step()
        ours = [list(oracle.adamw_step(p, x.numpy(), m, v, 0.01, 0.8, 0.95, 1e-6, t, decay, clip))
                for (p, m, v), x in zip(ours, grads)]
        for p, o in zip(ps, ours):
            assert np.allclose(p.detach().numpy(), o[0], rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("kind,dtype", [("m", torch.float8_e4m3fn), ("v", torch.float8_e5m2)])
def test_state_formats_are_torchs(kind, dtype):
    g = np.random.default_rng(5)
    x = (g.standard_normal(1000) * 2.0 ** g.integers(-25, 3, 1000)).astype(np.float32)
    if kind == "v":
        x = np.abs(x)
    x[300:600] = 0
    x[600:700] *= np.float32(2.0 ** -120)
    codes, scale = oracle.state_codes(x, kind)
    assert scale.shape == (4,)
    inverse = np.where(scale > 0, np.float32(1) / np.where(scale > 0, scale, 1), 0).astype(np.float32)
    y = torch.from_numpy(x * np.repeat(inverse, 256)[:1000])
    want = y.to(dtype).view(torch.uint8).numpy()
    if kind == "v":
        live = (x > 0) & (np.repeat(scale, 256)[:1000] > 0)
        assert ((want == 0) & live).any() and (codes[(want == 0) & live] == 1).all()
        want = np.where((want == 0) & live, 1, want)
    assert np.array_equal(codes, want)
    value = torch.from_numpy(codes.copy()).view(dtype).float().numpy() * np.repeat(scale, 256)[:1000]
    assert np.array_equal(oracle.state_values(codes, scale, kind), value.astype(np.float64))
