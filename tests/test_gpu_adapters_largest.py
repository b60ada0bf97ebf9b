"""The calls for many adapters at the largest sizes that they take: whole numbers whose sums fp32 holds, so that every
result is exact, whatever the order of its terms."""
import pytest
import torch

pytestmark = pytest.mark.gpu
WIDEST, MOST = 1 << 22, 1 << 25


def signs(*shape, seed=0):
    """-1, 0 and 1"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8)


def test_refused_past_them(lib):
    """The sizes of the tests below are the last ones."""
    for n, rows, cols in ((MOST, 16, 8), (3, WIDEST, 8), (3, 8, WIDEST)):
        assert lib.adapters_forward_workspace_bytes(n, rows, cols, 1, 4) == 0
        assert lib.adapters_backward_workspace_bytes(n, rows, cols, 1, 4) == 0


def check(X, G, B, A, tokens, bare, slots, Y, grads):
    """tokens(s): slot s's; bare: those without an adapter."""
    dX, dB, dA = grads
    assert not Y[bare].any() and not dX[bare].any()
    for s in range(slots):
        at = tokens(s)
        x, g, b, a = X[at].double(), G[at].double(), B[s].double(), A[s].double()
        H, P = x @ a.T, g @ b
        for got, want in ((Y[at], H @ b.T), (dX[at], P @ a), (dB[s], g.T @ H), (dA[s], P.T @ x)):
            assert want.abs().max() < 2 ** 24 and torch.equal(got.double(), want)


@pytest.mark.parametrize("rows,cols", [(WIDEST - 1, 8), (8, WIDEST - 8), (WIDEST - 8, 16), (5, WIDEST - 16)])
@pytest.mark.parametrize("n", [3, 70])
def test_widest(lib, n, rows, cols):
    rank = 4
    X, G, B, A = (signs(*s, seed=i) for i, s in enumerate(((n, cols), (n, rows), (2, rows, rank), (2, rank, cols))))
    ids = torch.arange(n, device="cuda", dtype=torch.int32) % 3 - 1
    plan = lib.loftq_adapters_plan(ids, 2)
    Xd, Gd, Bd, Ad = X.bfloat16(), G.bfloat16(), B.float(), A.float()
    check(X, G, B, A, lambda s: (ids == s).nonzero()[:, 0], (ids < 0).nonzero()[:, 0], 2,
          lib.loftq_adapters_forward(Xd, Bd, Ad, plan),
          lib.loftq_adapters_backward(Gd, Xd, Bd, Ad, plan, dx_dtype=torch.float32))


@pytest.mark.parametrize("slots", [1, 1024])
def test_most_tokens(lib, slots):
    n, rows, cols, rank = MOST - 1, 16, 8, 4
    X, G, B, A = (signs(*s, seed=i + 9) for i, s in enumerate(((n, cols), (n, rows), (slots, rows, rank), (slots, rank, cols))))
    ids = torch.randint(-1, slots, (n,), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda", dtype=torch.int32)
    plan = lib.loftq_adapters_plan(ids, slots)
    group = torch.where(ids < 0, slots, ids)
    order = torch.argsort(group, stable=True)
    starts = torch.searchsorted(group[order], torch.arange(slots + 2, device="cuda", dtype=torch.int32)).tolist()
    assert torch.equal(plan.order.long(), order) and plan.starts.tolist() == starts
    Xd, Gd, Bd, Ad = X.bfloat16(), G.bfloat16(), B.float(), A.float()
    check(X, G, B, A, lambda s: order[starts[s]:starts[s + 1]], order[starts[slots]:], slots,
          lib.loftq_adapters_forward(Xd, Bd, Ad, plan),
          lib.loftq_adapters_backward(Gd, Xd, Bd, Ad, plan, dx_dtype=torch.float32))
