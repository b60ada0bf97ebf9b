"""The operators for many adapters as they are used, one after another: two adapters trained together over one
frozen base with dropout, clipped AdamW steps and bf16 copies of the pool, then served in one mixed batch; every
stage against the oracle on the state that the stage before left."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_adapters import Batch, U, bf16, check, dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_train_and_serve(lib, bits):
    n, rows, cols, slots, rank, lr = 150, 128, 256, 3, 16, 1e-3
    W = 0.05 * torch.randn(rows, cols, generator=torch.Generator().manual_seed(1)).cuda()
    cfg = lib.default_config(rank=rank, iterative_steps=1, oversample=8)
    start = lib.loftq_init(W, cfg)
    nf = dict(packed=start["packed"], qabsmax=start["qabsmax"], dq_scale=start["dq_scale"], shape=(rows, cols))
    Wq = bf16(host(lib.loftq_nf4_dequantize(start["packed"], (rows, cols), qabsmax=start["qabsmax"], dq_scale=start["dq_scale"])))
    b = Batch(n, rows, cols, slots, rank, "runs", seed=2)
    b.Bd, b.Ad = start["B"].expand(slots, -1, -1).contiguous(), start["A"].expand(slots, -1, -1).contiguous()
    dB, dA = torch.empty_like(b.Bd), torch.empty_like(b.Ad)
    copies = [b.Bd.bfloat16(), b.Ad.bfloat16()]
    tensors = lib.AdamWTensors([b.Bd, b.Ad], [dB, dA], bits=bits, copies=copies, weight_decay=0.01, lr_scale=[4.0, 1.0])
    plan = b.plan(lib)
    for t in range(1, 4):
        rng = dict(p=0.1, seed=7, offset=t)
        b.B, b.A = bf16(host(b.Bd)), bf16(host(b.Ad))
        base = lib.loftq_qlora_forward_dropout(b.Xd, **nf)
        check(base, b.X @ Wq.T, (2 * cols + 16) * U * (np.abs(b.X) @ np.abs(Wq).T))
        b.Y0 = host(base)
        Y = b.forward(lib, plan, base=base, **rng)
        b.check_forward(Y, **rng)
        b.Gd = (Y * 1e-2).bfloat16()           # the gradient of a half square
        b.G = host(b.Gd)
        below = lib.loftq_qlora_backward(b.Gd, None, dx_dtype=torch.float32, **nf)[0]
        b.dX0 = host(below)
        grads = b.backward(lib, plan, base=below, out=(below, dB, dA), **rng)
        b.check_backward(grads, **rng)
        was = [host(x).ravel() for x in (b.Bd, b.Ad)]
        if bits == 8:
            states = [[oracle.state_values(x.view(torch.uint8).cpu().numpy().ravel(), s.cpu().numpy(), k)
                       for x, s in zip(xs, ss)] for xs, ss, k in ((tensors.m, tensors.m_scale, "m"), (tensors.v, tensors.v_scale, "v"))]
        else:
            states = [[host(x).ravel() for x in xs] for xs in (tensors.m, tensors.v)]
        gs = [host(x).ravel() for x in (dB, dA)]
        norm, clip = oracle.adamw_clip(gs, 0.3)
        got = lib.loftq_adamw(tensors, lr=lr, t=t, max_norm=0.3)
        assert abs(float(got) - norm) <= 2.0 ** -22 * norm
        for i, (x, rate) in enumerate(((b.Bd, 4 * lr), (b.Ad, lr))):
            want = oracle.adamw_step(was[i], gs[i], states[0][i], states[1][i], rate, 0.9, 0.999, 1e-8, t,
                                     float(np.float32(0.01)), clip)[0]
            # a step is at most rate (1 - b1^t) / (1 - b1) sqrt((1 - b2^t) / (1 - b2)) and a few more, of fp32 numbers
            assert np.all(abs(host(x).ravel() - want) <= 2.0 ** -20 * (abs(was[i]) + 20 * rate))
        assert all(torch.equal(c, x.bfloat16()) for c, x in zip(copies, (b.Bd, b.Ad)))
    # served from the bf16 copies, tokens of every adapter and of none in one batch; one token by itself
    for ids in (np.array([2, 0, -1, 1, 0, 2, 2, -1, 1, 0]), np.array([1])):
        s = Batch(len(ids), rows, cols, slots, rank, seed=3)
        s.ids, s.idd = ids, dev(ids, torch.int32)
        s.Bd, s.Ad, s.B, s.A = *copies, host(copies[0]), host(copies[1])
        Y = lib.loftq_qlora_forward(s.Xd, **nf)
        s.Y0 = host(Y)
        s.check_forward(s.forward(lib, base=Y, out=Y))
