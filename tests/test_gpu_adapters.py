"""Many adapters beside one shared weight, on the GPU against the oracle's formulas in fp64.

Bars.  Factors enter as bf16 values, so products of two operands are exact in fp32 and what differs is
rounding of sums: a sum of N terms added in fp32 in any order is off by at most (N - 1) u sum |terms|, with
u = 2^-23 per addition (nearest rounding has 2^-24; the matrix cores may truncate), and a second product over
the sums adds its own count.  With S the same formula on magnitudes, Y0 or dX0 included:
    Y: (cols + 3 rank + 16) u S     dX: (rows + 3 rank + 16) u S
    dB: (n + cols + 16) u S         dA: (n + rows + 16) u S
where 3 rank are the three pieces of the inner sums, and the 16 covers the joins of partial sums, the pieces'
rounding (2^-24 of each), the gain's product of three numbers and the last multiplication and addition.  An
output in bf16 adds half a step, 2^-8 |y|."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


def bf16(a):
    return oracle.bf16_round(np.asarray(a, dtype=np.float32)).astype(np.float64)


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def check(got, ref, tol):
    y = host(got)
    assert y.shape == ref.shape
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(y - ref)
    if err.size == 0:
        return
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert np.all(err <= tol), (worst, y[worst], ref[worst], tol[worst])


class Batch:
    """Random tokens, slots and a pool on the host (fp64 values) and the device.  `ids`: the tokens' slots."""

    def __init__(self, n, rows, cols, slots, rank, ids="mixed", ranks=False, factors=torch.float32, seed=0):
        g = np.random.default_rng(seed)
        self.n, self.rows, self.cols, self.slots, self.rank = n, rows, cols, slots, rank
        self.X, self.G = bf16(g.standard_normal((n, cols))), bf16(g.standard_normal((n, rows)))
        self.Xd, self.Gd = dev(self.X, torch.bfloat16), dev(self.G, torch.bfloat16)
        B, A = (0.1 * g.standard_normal(s).astype(np.float32) for s in ((slots, rows, rank), (slots, rank, cols)))
        self.B, self.A, self.Bd, self.Ad = bf16(B), bf16(A), dev(B, factors), dev(A, factors)
        self.gains = (0.5 + g.random(slots)).astype(np.float32)
        self.gd = dev(self.gains)
        if ids == "mixed":     # any order, some without an adapter, numbers that are no slot among them
            self.ids = g.integers(-1, slots + 1, n)
        elif ids == "runs":    # sequences of one slot each
            self.ids = np.repeat(g.integers(0, slots, -(-n // 37)), 37)[:n]
        elif ids == "none":
            self.ids = np.full(n, -1)
        else:                  # all tokens of one slot
            self.ids = np.full(n, int(ids))
        self.idd = dev(self.ids, torch.int32)
        self.ranks = self.rd = None
        if ranks:              # all of 0 .. rank, and numbers past either end
            self.ranks = (g.permutation(max(slots, rank + 3))[:slots] % (rank + 3)) - 1
            self.rd = dev(self.ranks, torch.int32)
        self.Y0, self.dX0 = (bf16(g.standard_normal(s)) for s in ((n, rows), (n, cols)))

    def plan(self, lib):
        return lib.loftq_adapters_plan(self.idd, self.slots)

    def base(self, which, dtype):
        return dev(which, dtype)

    def forward(self, lib, plan=None, alpha=1.5, dtype=torch.float32, **more):
        if "base" not in more:
            more["base"] = self.base(self.Y0, dtype)
        return lib.loftq_adapters_forward(self.Xd, self.Bd, self.Ad, plan or self.plan(lib), ranks=self.rd, gains=self.gd,
                                          alpha=alpha, **more)

    def backward(self, lib, plan=None, alpha=1.5, dtype=torch.bfloat16, **more):
        if "base" not in more:
            more["base"] = self.base(self.dX0, dtype)
        return lib.loftq_adapters_backward(self.Gd, self.Xd, self.Bd, self.Ad, plan or self.plan(lib), ranks=self.rd,
                                           gains=self.gd, alpha=alpha, **more)

    def _args(self, alpha, p, seed, offset):
        keep = oracle.keep_mask(self.X.shape, p, seed, offset) if p else None
        return self.gains.astype(np.float64) * alpha * oracle.drop_scale(p), keep

    def check_forward(self, Y, alpha=1.5, p=0.0, seed=0, offset=0, base=True):
        gains, keep = self._args(alpha, p, seed, offset)
        Y0 = self.Y0 if base else None
        ref = oracle.adapters_forward(self.X, self.B, self.A, self.ids, gains, self.ranks, keep, Y0)
        S = oracle.adapters_forward(abs(self.X), abs(self.B), abs(self.A), self.ids, abs(gains), self.ranks, keep,
                                    None if Y0 is None else abs(Y0))
        check(Y, ref, (self.cols + 3 * self.rank + 16) * U * S)

    def check_backward(self, grads, alpha=1.5, p=0.0, seed=0, offset=0, base=True):
        gains, keep = self._args(alpha, p, seed, offset)
        dX0 = self.dX0 if base else None
        ref = oracle.adapters_backward(self.G, self.X, self.B, self.A, self.ids, gains, self.ranks, keep, dX0)
        S = oracle.adapters_backward(abs(self.G), abs(self.X), abs(self.B), abs(self.A), self.ids, abs(gains), self.ranks,
                                     keep, None if dX0 is None else abs(dX0))
        for got, want, s, k in zip(grads, ref, S, (self.rows + 3 * self.rank, self.n + self.cols, self.n + self.rows)):
            if got is not None:
                check(got, want, (k + 16) * U * s)


# ---- the plan ----

@pytest.mark.parametrize("n,slots", [(0, 3), (1, 1), (2, 5), (63, 1), (64, 2), (65, 3), (300, 7), (4096, 1024), (4097, 5),
                                     (5000, 64), (20000, 1000), (70001, 33)])
@pytest.mark.parametrize("how", ["mixed", "one", "none", "runs"])
def test_plan(lib, n, slots, how):
    g = np.random.default_rng(n + slots)
    ids = {"mixed": g.integers(-2, slots + 2, n), "one": np.full(n, slots - 1), "none": np.full(n, -2 ** 31),
           "runs": np.repeat(g.integers(0, slots, n // 50 + 1), 50)[:n]}[how]
    plan = lib.loftq_adapters_plan(dev(ids, torch.int32), slots)
    starts, order = oracle.adapters_plan(ids, slots)
    assert np.array_equal(plan.starts.cpu().numpy(), starts)
    assert np.array_equal(plan.order.cpu().numpy(), order)


def test_plan_again_over_another(lib):
    g = np.random.default_rng(1)
    plan = None
    for how in range(3):
        ids = g.integers(0, 1 + 5 * how, 700) - 1
        plan = lib.loftq_adapters_plan(dev(ids, torch.int32), 9, plan=plan)
        starts, order = oracle.adapters_plan(ids, 9)
        assert np.array_equal(plan.starts.cpu().numpy(), starts) and np.array_equal(plan.order.cpu().numpy(), order)


# ---- forward and gradient ----

SHAPES = [  # n, rows, cols, slots, rank, ids, ranks
    (1, 1, 8, 1, 1, "0", False), (1, 40, 64, 4, 8, "2", False), (2, 16, 8, 2, 16, "mixed", False),
    (3, 129, 320, 5, 17, "mixed", True), (33, 100, 72, 3, 4, "0", False), (64, 257, 640, 64, 64, "mixed", True),
    (65, 256, 256, 1, 16, "0", False), (130, 384, 1032, 9, 33, "mixed", True), (257, 260, 128, 4, 48, "runs", False),
    (300, 77, 200, 300, 24, "mixed", True), (200, 1000, 264, 3, 64, "runs", True), (129, 64, 64, 2, 8, "none", False),
    (700, 72, 136, 2, 12, "1", False), (1300, 264, 96, 5, 40, "runs", True),
]


@pytest.mark.parametrize("factors", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_forward(lib, case, factors):
    b = Batch(*case, factors=factors, seed=sum(case[:5]))
    for p in (0.0, 0.1):
        rng = dict(p=p, seed=77, offset=5)
        for dtype in (torch.float32, torch.bfloat16):
            b.check_forward(b.forward(lib, dtype=dtype, **rng), **rng)
            b.check_forward(b.forward(lib, base=None, out_dtype=dtype, **rng), base=False, **rng)


@pytest.mark.parametrize("factors", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_backward(lib, case, factors):
    b = Batch(*case, factors=factors, seed=sum(case[:5]) + 1)
    for p in (0.0, 0.1):
        rng = dict(p=p, seed=78, offset=6)
        for dtype in (torch.float32, torch.bfloat16):
            b.check_backward(b.backward(lib, dtype=dtype, **rng), **rng)
            b.check_backward(b.backward(lib, base=None, dx_dtype=dtype, **rng), base=False, **rng)


@pytest.mark.parametrize("n,rows,cols,slots,rank", [(2100, 520, 1024, 3, 16), (4500, 264, 512, 2, 64), (600, 2056, 512, 40, 32)])
def test_longer(lib, n, rows, cols, slots, rank):
    b = Batch(n, rows, cols, slots, rank, "runs", seed=9)
    rng = dict(p=0.25, seed=3, offset=1)
    b.check_forward(b.forward(lib, **rng), **rng)
    b.check_backward(b.backward(lib, dtype=torch.float32, **rng), **rng)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,rows,cols,slots,rank", [(2048, 11008, 64, 8, 64), (2050, 64, 11008, 3, 16), (1030, 11004, 4104, 2, 24),
                                                    (2048, 11008, 128, 4, 32)])
def test_many_features(lib, n, rows, cols, slots, rank, dtype):
    """A wave takes several blocks of features, and several steps of the first product, in a loop."""
    b = Batch(n, rows, cols, slots, rank, ids="runs", ranks=rank == 64, seed=n + rows)
    plan, rng = b.plan(lib), dict(p=0.1, seed=5, offset=6)
    Y, grads = b.forward(lib, plan, dtype=dtype, **rng), b.backward(lib, plan, dtype=dtype, **rng)
    b.check_forward(Y, **rng)
    b.check_backward(grads, **rng)
    for _ in range(3):
        again = (b.forward(lib, plan, dtype=dtype, **rng), *b.backward(lib, plan, dtype=dtype, **rng))
        assert all(torch.equal(x, y) for x, y in zip(again, (Y, *grads)))


def test_everything_dropped(lib):
    b = Batch(70, 64, 128, 3, 8, seed=2)
    rng = dict(p=1.0, seed=3, offset=1)
    assert torch.equal(b.forward(lib, **rng), dev(b.Y0))
    dX, dB, dA = b.backward(lib, **rng)
    assert torch.equal(dX, dev(b.dX0, torch.bfloat16)) and not dB.any() and not dA.any()


def test_gradient_against_differences(lib):
    """Y is linear in B (and in A) for the other at rest, and bf16 steps pass the factors' rounding: between B = 0 and
    B = step, <G, Y> changes by <dB, step>, up to the rounding of the sums."""
    b = Batch(150, 96, 128, 3, 16, "runs", seed=4)
    rng = dict(p=0.2, seed=1, offset=2)
    plan = b.plan(lib)
    _, dB, dA = b.backward(lib, plan, **rng)
    for name, grad in (("Bd", dB), ("Ad", dA)):
        old = getattr(b, name)
        step = torch.randn_like(old).bfloat16().float()
        setattr(b, name, step)
        moved = host(b.forward(lib, plan, base=None, **rng))
        setattr(b, name, old)
        change = (b.G * moved).sum()
        size = (np.abs(b.G) * np.abs(moved)).sum() + (np.abs(host(grad)) * np.abs(host(step))).sum()
        assert abs(change - (host(grad) * host(step)).sum()) <= 4 * (150 + 96 + 128) * U * size


def test_one_slot_equals_the_layers_calls(lib):
    """Beside a base product without an adapter, a pool of one slot gives what the layer's own calls give with it."""
    b = Batch(90, 128, 256, 1, 16, "0", seed=6)
    W = 0.05 * torch.randn(128, 256, device="cuda")
    packed, absmax = lib.loftq_nf4_quantize(W)
    nf, rng = dict(packed=packed, absmax=absmax, shape=(128, 256)), dict(p=0.3, seed=2, offset=9)
    alpha = 1.5 * float(b.gains[0])
    layer = lib.loftq_qlora_forward_dropout(b.Xd, B=b.Bd[0], A=b.Ad[0], alpha=alpha, **nf, **rng)
    beside = b.forward(lib, base=lib.loftq_qlora_forward_dropout(b.Xd, **nf), **rng)
    assert torch.linalg.norm(layer - beside) <= 1e-6 * torch.linalg.norm(layer)
    dX, dB, dA = lib.loftq_qlora_backward(b.Gd, b.Xd, B=b.Bd[0], A=b.Ad[0], alpha=alpha, dx_dtype=torch.float32, **nf, **rng)
    base = lib.loftq_qlora_backward(b.Gd, None, dx_dtype=torch.float32, **nf)[0]
    for got, want in zip(b.backward(lib, base=base, **rng), (dX, dB[None], dA[None])):
        assert torch.linalg.norm(got - want) <= 1e-6 * torch.linalg.norm(want)


def test_in_place(lib):
    b = Batch(100, 72, 64, 3, 8, seed=7)
    plan = b.plan(lib)
    for dtype in (torch.float32, torch.bfloat16):
        want = b.forward(lib, plan, dtype=dtype)
        Y = b.base(b.Y0, dtype)
        assert b.forward(lib, plan, base=Y, out=Y) is Y and torch.equal(Y, want)
        want = b.backward(lib, plan, dtype=dtype)
        dX = b.base(b.dX0, dtype)
        got = b.backward(lib, plan, base=dX, out=(dX, torch.empty_like(want[1]), torch.empty_like(want[2])))
        assert got[0] is dX and all(torch.equal(x, y) for x, y in zip(got, want))


def test_parts_of_the_gradient(lib):
    b = Batch(140, 70, 128, 4, 8, seed=5)
    plan, rng = b.plan(lib), dict(p=0.1, seed=1, offset=2)
    dX, dB, dA = b.backward(lib, plan, **rng)
    only = b.backward(lib, plan, need_dx=False, **rng)
    assert only[0] is None and torch.equal(only[1], dB) and torch.equal(only[2], dA)
    x, b.Xd = b.Xd, None   # the input is not needed for dX
    got = b.backward(lib, plan, out=(torch.full_like(dX, 7.0), None, None), **rng)
    assert torch.equal(got[0], dX)
    b.Xd = x


def test_no_tokens(lib):
    b = Batch(0, 64, 128, 3, 8, seed=5)
    assert b.forward(lib).shape == (0, 64)
    dX, dB, dA = b.backward(lib, out=(dev(b.dX0, torch.bfloat16), torch.ones_like(b.Bd), torch.ones_like(b.Ad)))
    assert dX.shape == (0, 128) and not dB.any() and not dA.any()
    none = Batch(5, 0, 128, 3, 8, seed=5)
    assert none.forward(lib).shape == (5, 0)


def test_what_the_pool_holds_past_a_rank_is_not_used(lib):
    b = Batch(150, 90, 136, 6, 24, ranks=True, seed=8)
    plan, rng = b.plan(lib), dict(p=0.1, seed=1, offset=2)
    want = (b.forward(lib, plan, **rng), *b.backward(lib, plan, **rng))
    for s in range(6):
        r = int(np.clip(b.ranks[s], 0, 24))
        b.Bd[s, :, r:] = float("nan")
        b.Ad[s, r:] = float("inf")
    got = (b.forward(lib, plan, **rng), *b.backward(lib, plan, **rng))
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("factors", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,rows,rank", [(40, 129, 17), (300, 33, 1), (40, 7, 9), (300, 130, 25), (40, 64, 12)])
def test_slots_that_begin_at_any_element(lib, n, rows, rank, factors):
    """With odd rows and ranks a slot's factors, and their rows, begin anywhere in a vector; each slot's tokens and
    gradients are those of a pool of that slot alone, which begins at the start of one."""
    slots, cols = 5, 72
    b = Batch(n, rows, cols, slots, rank, seed=rank, factors=factors)
    Y, (dX, dB, dA) = b.forward(lib), b.backward(lib)
    b.check_forward(Y)
    b.check_backward((dX, dB, dA))
    for s in range(slots):
        one = Batch(n, rows, cols, 1, rank, seed=rank, factors=factors)
        one.Xd, one.Gd, one.Y0, one.dX0, one.gd = b.Xd, b.Gd, b.Y0, b.dX0, b.gd[s:s + 1].clone()
        one.Bd, one.Ad = b.Bd[s:s + 1].clone(), b.Ad[s:s + 1].clone()
        one.idd = torch.where(b.idd == s, 0, -1).int()
        mine = b.idd == s
        Y1, (dX1, dB1, dA1) = one.forward(lib), one.backward(lib)
        for got, want in ((Y[mine], Y1[mine]), (dX[mine], dX1[mine]), (dB[s], dB1[0]), (dA[s], dA1[0])):
            # sums over the columns may be divided otherwise among fewer tiles, which in bf16 can turn a rounding: 2^-8 each
            assert torch.linalg.norm(got.float() - want.float()) <= 2.0 ** -7 * torch.linalg.norm(want.float())


def test_slots_do_not_touch_each_other(lib):
    """NaN in one slot's factors, or in one token, reaches that slot's tokens, or that token, alone."""
    b = Batch(200, 64, 128, 4, 16, seed=10)
    plan = b.plan(lib)
    Y, (dX, dB, dA) = b.forward(lib, plan), b.backward(lib, plan)
    old = b.Ad.clone()
    b.Ad[1] = float("nan")
    Y1, (dX1, dB1, dA1) = b.forward(lib, plan), b.backward(lib, plan)
    b.Ad = old
    mine = torch.from_numpy(b.ids == 1).cuda()
    assert torch.isnan(Y1[mine]).all() and torch.equal(Y1[~mine], Y[~mine])
    assert torch.isnan(dX1[mine]).all() and torch.equal(dX1[~mine], dX[~mine])
    rest = [0, 2, 3]
    assert torch.equal(dB1[rest], dB[rest]) and torch.equal(dA1, dA)   # dA does not read A
    token = int(np.flatnonzero(b.ids == 2)[-1])   # the last of its slot, which its tile repeats
    for bad in (float("nan"), float("inf")):
        X = b.Xd.clone()
        b.Xd = X.clone()
        b.Xd[token, 5] = bad
        Y2, (dX2, dB2, dA2) = b.forward(lib, plan), b.backward(lib, plan)
        b.Xd = X
        others = torch.arange(200, device="cuda") != token
        assert not torch.isfinite(Y2[token]).any() and torch.equal(Y2[others], Y[others])
        assert torch.equal(dX2, dX) and torch.equal(dB2[[0, 1, 3]], dB[[0, 1, 3]])
        col = torch.arange(128, device="cuda") != 5
        assert not torch.isfinite(dA2[2, :, 5]).any() and torch.equal(dA2[2][:, col], dA[2][:, col])


def test_dropped_values_may_be_anything(lib):
    b = Batch(100, 64, 128, 3, 8, seed=11)
    plan, rng = b.plan(lib), dict(p=0.5, seed=1, offset=2)
    want = (b.forward(lib, plan, **rng), *b.backward(lib, plan, **rng))
    keep = torch.from_numpy(oracle.keep_mask((100, 128), 0.5, 1, 2)).cuda()
    b.Xd = torch.where(keep, b.Xd, torch.full_like(b.Xd, float("nan")))
    got = (b.forward(lib, plan, **rng), *b.backward(lib, plan, **rng))
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def fenced(t):
    raw = t.contiguous().view(torch.uint8).reshape(-1)
    big = torch.full((raw.numel() + (1 << 16),), 255, dtype=torch.uint8, device="cuda")
    big[: raw.numel()] = raw
    return big[: raw.numel()].view(t.dtype).view(t.shape)


@pytest.mark.parametrize("n,rows,cols,slots,rank", [(45, 100, 192, 3, 20), (70, 131, 328, 2, 8), (200, 128, 72, 5, 64)])
def test_nothing_behind_the_inputs_is_used(lib, n, rows, cols, slots, rank):
    """Inputs that end where NaN begins (every byte 255 behind each) give what they give by themselves."""
    b = Batch(n, rows, cols, slots, rank, seed=19)
    rng = dict(p=0.3, seed=9, offset=1)
    for factors in (torch.float32, torch.bfloat16):
        b.Bd, b.Ad = b.Bd.to(factors), b.Ad.to(factors)
        want = (b.forward(lib, **rng), *b.backward(lib, **rng))
        kept = {k: getattr(b, k) for k in ("Xd", "Gd", "Bd", "Ad", "gd", "idd")}
        for k, v in kept.items():
            setattr(b, k, fenced(v))
        got = (b.forward(lib, **rng), *b.backward(lib, **rng))
        for k, v in kept.items():
            setattr(b, k, v)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_outputs_are_overwritten_and_nothing_else(lib):
    """Stale contents of the workspaces and of the plan's memory do not matter, and what lies behind outputs and
    workspaces stays."""
    n, rows, cols, slots, rank = 150, 99, 192, 5, 8
    b = Batch(n, rows, cols, slots, rank, seed=6)
    rng = dict(p=0.1, seed=1, offset=2)
    want = [b.forward(lib, **rng), *b.backward(lib, **rng)]
    sizes = (lib.adapters_forward_workspace_bytes, lib.adapters_backward_workspace_bytes)
    for fill in (0, 255):   # 255: NaN in every type
        plan = lib.AdaptersPlan(n, slots)
        plan.buffer.view(torch.uint8).fill_(fill)
        lib.loftq_adapters_plan(b.idd, slots, plan=plan)
        need = [f(n, rows, cols, slots, rank) for f in sizes]
        ws = [torch.full((k + 256,), fill, dtype=torch.uint8, device="cuda") for k in need]
        bufs = [torch.full((t.numel() + 64,), float("nan"), dtype=t.dtype, device="cuda") for t in want]
        out = [x[: t.numel()].view(t.shape) for x, t in zip(bufs, want)]
        b.forward(lib, plan, out=out[0], ws=ws[0][:need[0]], **rng)
        b.backward(lib, plan, out=out[1:], ws=ws[1][:need[1]], **rng)
        for o, x, t in zip(out, bufs, want):
            assert torch.equal(o, t) and torch.isnan(x[t.numel():]).all()
        assert all((w[k:] == fill).all() for w, k in zip(ws, need))


def test_smaller_calls_in_a_large_workspace(lib):
    b = Batch(3000, 72, 1024, 7, 16, "runs", seed=12)
    ws = torch.empty(lib.adapters_forward_workspace_bytes(3000, 72, 1024, 7, 16), dtype=torch.uint8, device="cuda")
    wb = torch.empty(lib.adapters_backward_workspace_bytes(3000, 72, 1024, 7, 16), dtype=torch.uint8, device="cuda")
    for n in (1, 5, 64, 100, 500, 1000, 2999):
        s = Batch(n, 72, 1024, 7, 16, seed=n)
        s.check_forward(s.forward(lib, ws=ws))
        s.check_backward(s.backward(lib, ws=wb))


# tokens of each slot: as many slots of several chunks as their tokens allow, each with one token in its last; one slot of
# all but a few; no more than one chunk each; two of several among many of one, the first and the last slot of the pool
COUNTS = [[193] * 3, [257] * 4, [65] * 3 + [0, 1], [2000] + [1] * 40, [128] * 20, [700] + [3] * 98 + [900], [8193, 64 * 128, 8200]]


@pytest.mark.parametrize("rank", [8, 40])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}-{sum(c)}")
def test_partial_sums_of_slots_of_every_length(lib, counts, rank):
    """Within a workspace of the size that is asked for, with what lies behind it untouched."""
    n, rows, cols, slots = sum(counts), 75, 64, len(counts)
    b = Batch(n, rows, cols, slots, rank, seed=n)
    b.ids = np.random.default_rng(n).permutation(np.repeat(np.arange(slots), counts))
    b.idd = dev(b.ids, torch.int32)
    need = lib.adapters_backward_workspace_bytes(n, rows, cols, slots, rank)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    rng = dict(p=0.1, seed=1, offset=2)
    b.check_backward(b.backward(lib, ws=ws[:need], **rng), **rng)
    assert (ws[need:] == 255).all()


def test_same_results_again_and_on_streams(lib):
    """Calls with workspaces of their own may overlap on two streams over one plan."""
    b = Batch(300, 320, 512, 5, 16, seed=8)
    rng = dict(p=0.1, seed=1, offset=2)
    plan = b.plan(lib)
    want = (b.forward(lib, plan, **rng), *b.backward(lib, plan, **rng))
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                got.append((b.forward(lib, plan, **rng), *b.backward(lib, plan, **rng)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for once in got for x, y in zip(once, want))


def test_results_on_another_stream_with_the_current_one_busy(lib):
    """The memory of a call with stream= comes without a wait for the current stream, which writes all the while."""
    b = Batch(300, 512, 1024, 4, 16, seed=13)
    rng = dict(p=0.1, seed=1, offset=2)
    want = (b.forward(lib, **rng), *b.backward(lib, **rng))
    starts = b.plan(lib).starts.cpu()
    torch.cuda.synchronize()
    base = dict(forward=dev(b.Y0), backward=dev(b.dX0, torch.bfloat16))
    torch.cuda.synchronize()
    side, junk = torch.cuda.Stream(), []
    for _ in range(4):
        junk.append(torch.full((1 << 22,), 7, dtype=torch.uint8, device="cuda"))
        plan = lib.loftq_adapters_plan(b.idd, b.slots, stream=side)
        got = (b.forward(lib, plan, base=base["forward"], stream=side, **rng),
               *b.backward(lib, plan, base=base["backward"], stream=side, **rng))
        for nbytes in (1 << 12, 1 << 16, 1 << 20, 1 << 22, 1 << 24):
            junk.append(torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda"))
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(plan.starts.cpu(), starts) and all(torch.equal(x, y) for x, y in zip(got, want))
        del junk[:], got


def test_captured_serving(lib):
    """A decoding step in a graph: the base's product, the plan and the adapters, replayed on new tokens and new slots."""
    b = Batch(40, 192, 288, 6, 16, seed=18)
    packed, scales = lib.loftq_mxfp4_quantize(0.05 * torch.randn(192, 288, device="cuda"))
    mx = dict(packed=packed, scales=scales, shape=(192, 288))
    wm = torch.empty(lib.mxfp4_forward_workspace_bytes(40, 192, 288, 0), dtype=torch.uint8, device="cuda")
    wa = torch.empty(lib.adapters_forward_workspace_bytes(40, 192, 288, 6, 16), dtype=torch.uint8, device="cuda")
    X, ids, Y = b.Xd.clone(), b.idd.clone(), torch.empty(40, 192, device="cuda")
    plan = lib.AdaptersPlan(40, 6)

    def serve():
        lib.loftq_mxfp4_forward(X, out=Y, ws=wm, **mx)
        lib.loftq_adapters_plan(ids, 6, plan=plan)
        lib.loftq_adapters_forward(X, b.Bd, b.Ad, plan, gains=b.gd, base=Y, out=Y, ws=wa)

    serve()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        serve()
    for k in range(4):
        X.copy_(torch.randn(40, 288, device="cuda"))
        ids.copy_(torch.randint(-1, 6, (40,), device="cuda"))
        graph.replay()
        got = Y.clone()
        serve()
        torch.cuda.synchronize()
        assert torch.equal(got, Y)
        b.X, b.ids = X.double().cpu().numpy(), ids.cpu().numpy()
        b.Y0 = host(lib.loftq_mxfp4_forward(X, **mx))
        b.check_forward(Y, alpha=1.0)


def test_captured_training_step(lib):
    """Forward and gradient in one graph that counts its own step: each replay draws that step's mask."""
    b = Batch(200, 192, 256, 3, 16, "runs", seed=10)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    plan, Y0, dX0 = b.plan(lib), dev(b.Y0), dev(b.dX0, torch.bfloat16)
    wf = torch.empty(lib.adapters_forward_workspace_bytes(200, 192, 256, 3, 16), dtype=torch.uint8, device="cuda")
    wb = torch.empty(lib.adapters_backward_workspace_bytes(200, 192, 256, 3, 16), dtype=torch.uint8, device="cuda")
    Y, out = torch.empty_like(Y0), (torch.empty_like(dX0), torch.empty_like(b.Bd), torch.empty_like(b.Ad))

    def train():
        b.forward(lib, plan, base=Y0, p=0.3, seed=4, offset=0, step=step, out=Y, ws=wf)
        b.backward(lib, plan, base=dX0, p=0.3, seed=4, offset=0, step=step, out=out, ws=wb)
        step.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train()
    step.fill_(5)
    for k in range(5, 9):
        graph.replay()
        got = [t.clone() for t in (Y, *out)]
        want = [b.forward(lib, plan, base=Y0, p=0.3, seed=4, offset=k),
                *b.backward(lib, plan, base=dX0, p=0.3, seed=4, offset=k)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), k


def test_offsets_past_32_bits(lib):
    """X, Y, dY and dX of more than 2^31 elements: the last tokens' results against the oracle, the base before them."""
    n, rows, cols, rank = 140000, 16448, 16384, 4
    b = Batch(8, rows, cols, 2, rank, "runs", seed=11)
    tail, G8 = b.Xd, b.Gd
    ids = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    ids[-8:] = b.idd
    ids[5] = 0
    plan = lib.loftq_adapters_plan(ids, 2)
    b.Xd = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
    b.Xd[-8:] = tail
    Y = b.forward(lib, plan, base=None, out_dtype=torch.bfloat16)
    b.check_forward(Y[-8:], base=False)
    assert not Y[:-8].any()
    del Y
    b.Gd = torch.zeros(n, rows, dtype=torch.bfloat16, device="cuda")
    b.Gd[-8:] = G8
    dX, dB, dA = b.backward(lib, plan, base=None)
    b.check_backward((dX[-8:], dB, dA), base=False)
    assert not dX[:-8].any()


@pytest.mark.parametrize("rank", [4, 40])
def test_masks_past_32_bits(lib, rank):
    """The same sizes under a mask, whose words are numbered by the element of the whole call, in every product that reads
    or writes so much; of one rank tile and of three."""
    n, rows, cols, tail = 140000, 16448, 16384, 8
    b = Batch(tail, rows, cols, 2, rank, "runs", seed=12)
    p, rng = 0.25, dict(p=0.25, seed=9, offset=4)
    keep = oracle.keep_mask((tail, cols), p, 9, 4, first=(n - tail) * cols)
    gains = b.gains.astype(np.float64) * 1.5 * oracle.drop_scale(p)
    ids = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    ids[-tail:] = b.idd
    plan = lib.loftq_adapters_plan(ids, 2)
    X8, G8, dX0 = b.Xd, b.Gd, b.dX0
    b.Xd = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
    b.Xd[-tail:] = X8
    for dtype in (torch.bfloat16, torch.float32):
        Y = b.forward(lib, plan, base=None, out_dtype=dtype, **rng)
        size = (b.cols + 3 * rank + 16) * U * oracle.adapters_forward(abs(b.X), abs(b.B), abs(b.A), b.ids, gains, None, keep)
        check(Y[-tail:], oracle.adapters_forward(b.X, b.B, b.A, b.ids, gains, None, keep), size)
        assert not Y[:-tail].any()
        del Y
    b.Gd = torch.zeros(n, rows, dtype=torch.bfloat16, device="cuda")
    b.Gd[-tail:] = G8
    ref = oracle.adapters_backward(b.G, b.X, b.B, b.A, b.ids, gains, None, keep, dX0)
    S = oracle.adapters_backward(abs(b.G), abs(b.X), abs(b.B), abs(b.A), b.ids, gains, None, keep, abs(dX0))
    for dtype in (torch.bfloat16, torch.float32):
        base = torch.zeros(n, cols, dtype=dtype, device="cuda")
        base[-tail:] = dev(dX0, dtype)
        dX, dB, dA = b.backward(lib, plan, base=base, out=(base, torch.empty_like(b.Bd), torch.empty_like(b.Ad)), **rng)
        for got, want, s, k in zip((dX[-tail:], dB, dA), ref, S, (rows + 3 * rank, tail + cols, tail + rows)):
            check(got, want, (k + 16) * U * s)
        assert not dX[:-tail].any()
        del base, dX


@pytest.mark.parametrize("n", [5, 300])
def test_without_gains(lib, n):
    """No gains are gains of one."""
    b = Batch(n, 72, 136, 4, 24, ranks=True, seed=31)
    b.gains = np.ones(4, np.float32)
    rng, ones = dict(p=0.1, seed=1, offset=2), dev(b.gains)
    b.gd = None
    got = (b.forward(lib, **rng), *b.backward(lib, dtype=torch.float32, **rng))
    b.check_forward(got[0], **rng)
    b.check_backward(got[1:], **rng)
    b.gd = ones
    assert all(torch.equal(x, y) for x, y in zip(got, (b.forward(lib, **rng), *b.backward(lib, dtype=torch.float32, **rng))))
    empty = Batch(0, 72, 136, 4, 24, seed=31)
    empty.gd = None
    _, dB, dA = empty.backward(lib, out=(dev(empty.dX0, torch.bfloat16), torch.ones_like(empty.Bd), torch.ones_like(empty.Ad)))
    assert not dB.any() and not dA.any()


def test_binding_checks_on_device(lib):
    b = Batch(8, 64, 128, 3, 8, seed=14)
    plan = b.plan(lib)
    with pytest.raises(ValueError):
        b.forward(lib, plan, out=torch.empty(8, 65, device="cuda"))
    with pytest.raises(ValueError):
        b.forward(lib, lib.loftq_adapters_plan(b.idd[:7].contiguous(), 3))
    with pytest.raises(ValueError):
        b.forward(lib, lib.loftq_adapters_plan(b.idd, 4))
    with pytest.raises(ValueError):
        lib.loftq_adapters_plan(b.idd, 3, plan=lib.AdaptersPlan(9, 3))
    with pytest.raises(TypeError):
        lib.loftq_adapters_plan(b.idd.long(), 3)
    with pytest.raises(TypeError):
        b.forward(lib, plan, base=None, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        b.forward(lib, plan, base=dev(b.Y0), out=torch.empty(8, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(lib.LoftqError):
        b.forward(lib, plan, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        b.backward(lib, plan, out=(None, torch.empty(3, 64, 8, device="cuda"), torch.empty(3, 8, 127, device="cuda")))
    with pytest.raises(lib.LoftqError) as e:
        lib.AdaptersPlan(8, 1025)
    assert e.value.status == 2
    b.Ad = b.Ad.bfloat16()
    with pytest.raises(TypeError):
        b.forward(lib, plan)
    b.Xd = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")[:, ::2]
    with pytest.raises(ValueError):
        b.forward(lib, plan)
