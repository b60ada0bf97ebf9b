"""Refusals and workspace queries of the calls for many adapters and of the optimizer's step: every one is made
before anything is enqueued (no GPU needed), through the C ABI and through the binding's own checks."""
import ctypes

import pytest
import torch

FAKE = 0x10000   # aligned, never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def b():
    from loftq_qlora_initialization_amd import binding
    return binding


def drop(b, p=0.1, step=None):
    return ctypes.byref(b.LoftqDropout(p, 1, 2, step))


def pool(b, B=FAKE, A=FAKE, dt=0, slots=4, rank=8, ranks=None, gains=None, alpha=1.0):
    return ctypes.byref(b.LoftqAdapters(B, A, dt, slots, rank, ranks, gains, alpha))


def test_plan_refusals(b):
    f = b._c_ad_plan
    assert f(FAKE, -1, 4, FAKE, BIG, None) == INVALID
    assert f(FAKE, 1 << 31, 4, FAKE, BIG, None) == INVALID
    assert f(FAKE, 8, 0, FAKE, BIG, None) == INVALID
    assert f(None, 8, 4, FAKE, BIG, None) == INVALID
    assert f(FAKE + 2, 8, 4, FAKE, BIG, None) == INVALID            # numbers of 4 bytes
    assert f(FAKE, 8, 4, None, BIG, None) == INVALID
    assert f(FAKE, 8, 4, FAKE + 8, BIG, None) == INVALID
    assert f(FAKE, 8, 1025, FAKE, BIG, None) == UNSUPPORTED
    assert f(FAKE, 1 << 25, 4, FAKE, BIG, None) == UNSUPPORTED
    assert f(FAKE, 8, 4, FAKE, b.adapters_plan_bytes(8, 4) - 1, None) == WORKSPACE
    assert b.adapters_plan_bytes(-1, 4) == 0 and b.adapters_plan_bytes(8, 0) == 0 and b.adapters_plan_bytes(8, 1025) == 0
    assert b.adapters_plan_bytes(0, 1) > 0


def fwd(b, n=16, rows=64, cols=128, ad=None, plan=FAKE, plan_bytes=BIG, drop=None, X=FAKE, Y0=FAKE, Y=FAKE, ydt=0, ws=FAKE,
        ws_bytes=BIG):
    return b._c_ad_fwd(X, n, rows, cols, ad or pool(b), plan, plan_bytes, drop, Y0, Y, ydt, ws, ws_bytes, None)


def bwd(b, n=16, rows=64, cols=128, ad=None, plan=FAKE, plan_bytes=BIG, drop=None, X=FAKE, dY=FAKE, dX0=FAKE, dX=FAKE, xdt=1,
        dB=FAKE, dA=FAKE, ws=FAKE, ws_bytes=BIG):
    return b._c_ad_bwd(dY, X, n, rows, cols, ad or pool(b), plan, plan_bytes, drop, dX0, dX, xdt, dB, dA, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_call_refusals(b, call):
    for kw in (dict(n=-1), dict(n=1 << 31), dict(rows=-1), dict(rows=1 << 31), dict(cols=-8), dict(X=None), dict(X=FAKE + 2),
               dict(ws=None), dict(ws=FAKE + 8), dict(plan=None), dict(plan=FAKE + 4), dict(drop=drop(b, 2.0)),
               dict(drop=drop(b, NAN)), dict(drop=drop(b, step=FAKE + 4))):
        assert call(b, **kw) == INVALID, kw
    for kw in (dict(B=None), dict(A=None), dict(B=FAKE + 4), dict(A=FAKE + 8), dict(dt=2), dict(slots=0), dict(rank=0),
               dict(ranks=FAKE + 2), dict(gains=FAKE + 1), dict(alpha=NAN), dict(alpha=INF)):
        assert call(b, ad=pool(b, **kw)) == INVALID, kw
    assert call(b, ad=pool(b, alpha=3e38), drop=drop(b, 0.9)) == INVALID
    for kw in (dict(cols=0), dict(cols=12), dict(cols=1 << 22), dict(rows=1 << 22), dict(n=1 << 25)):
        assert call(b, **kw) == UNSUPPORTED, kw
    for kw in (dict(rank=65), dict(slots=1025)):
        assert call(b, ad=pool(b, **kw)) == UNSUPPORTED, kw
    assert call(b, plan_bytes=b.adapters_plan_bytes(16, 4) - 1) == WORKSPACE
    size = b.adapters_forward_workspace_bytes if call is fwd else b.adapters_backward_workspace_bytes
    assert call(b, ws_bytes=size(16, 64, 128, 4, 8) - 1) == WORKSPACE


def test_no_pool(b):
    assert b._c_ad_fwd(FAKE, 16, 64, 128, None, FAKE, BIG, None, FAKE, FAKE, 0, FAKE, BIG, None) == INVALID
    assert b._c_ad_bwd(FAKE, FAKE, 16, 64, 128, None, FAKE, BIG, None, FAKE, FAKE, 1, FAKE, FAKE, FAKE, BIG, None) == INVALID


def test_outputs(b):
    assert fwd(b, Y=None) == INVALID and fwd(b, Y=FAKE + 4) == INVALID and fwd(b, Y0=FAKE + 4) == INVALID and fwd(b, ydt=2) == INVALID
    assert fwd(b, n=0) == OK and fwd(b, rows=0) == OK               # nothing to write
    assert fwd(b, n=(1 << 25) - 1, rows=(1 << 22) - 1) == UNSUPPORTED   # more than a launch takes
    assert bwd(b, dY=None) == INVALID and bwd(b, dY=FAKE + 2) == INVALID and bwd(b, dX0=FAKE + 2) == INVALID
    assert bwd(b, dB=None) == INVALID and bwd(b, dA=None) == INVALID and bwd(b, dA=FAKE + 4) == INVALID
    assert bwd(b, dX=FAKE + 4) == INVALID and bwd(b, xdt=3) == INVALID
    assert bwd(b, dX=None, dB=None, dA=None) == INVALID             # nothing asked for
    assert bwd(b, rows=0) == UNSUPPORTED
    assert bwd(b, n=0, dB=None, dA=None) == OK and bwd(b, n=0, dX=None, dB=None, dA=None) == OK


def test_pools_of_more_factors_than_a_launch_takes(b):
    wide = dict(rows=(1 << 22) - 8, cols=(1 << 22) - 8)
    assert fwd(b, **wide, ad=pool(b, slots=1024, rank=1)) == UNSUPPORTED
    assert bwd(b, **wide, ad=pool(b, slots=1024, rank=1)) == UNSUPPORTED
    assert b.adapters_forward_workspace_bytes(16, wide["rows"], 64, 1024, 1) == 0
    assert b.adapters_backward_workspace_bytes(16, 64, wide["cols"], 1024, 1) == 0
    assert b.adapters_forward_workspace_bytes(16, wide["rows"], 64, 128, 1) > 0


QUERIES = ["adapters_forward_workspace_bytes", "adapters_backward_workspace_bytes"]


@pytest.mark.parametrize("query", QUERIES)
@pytest.mark.parametrize("rows,cols", [(4096, 4096), (11008, 4096), (130, 64), (64, 16384), (5, 8)])
@pytest.mark.parametrize("slots", [1, 7, 64, 1024])
def test_query_grows_with_the_tokens_and_the_rank(b, query, rows, cols, slots):
    """So that the workspace of the longest batch serves every shorter one."""
    q = getattr(b, query)
    counts = list(range(0, 2100)) + [int(1.3 ** k) for k in range(30, 50)]
    before = None
    for r in (1, 16, 17, 64):
        need = [q(n, rows, cols, slots, r) for n in counts]
        assert need == sorted(need)
        assert before is None or all(x <= y for x, y in zip(before, need))
        before = need
    assert q(-1, rows, cols, slots, 8) == 0 and q(16, rows, cols, 0, 8) == 0 and q(16, rows, cols, slots, 65) == 0
    assert q(16, rows, 12, slots, 8) == 0 and q(1 << 25, rows, cols, slots, 8) == 0


def tensor(b, param=FAKE, grad=FAKE, m=FAKE, v=FAKE, m_scale=None, v_scale=None, copy=None, n=100, lr_scale=1.0, decay=0.0):
    return b.LoftqAdamwTensor(param, grad, m, v, m_scale, v_scale, copy, n, lr_scale, decay)


def plan(b, *tensors, count=None, pdt=0, gdt=0, bits=32, table=FAKE, table_bytes=BIG, out=True):
    p = b.LoftqAdamwPlan()
    array = (b.LoftqAdamwTensor * max(1, len(tensors)))(*tensors)
    return b._c_adamw_plan(array, len(tensors) if count is None else count, pdt, gdt, bits, table, table_bytes,
                           ctypes.byref(p) if out else None, None)


def test_adamw_plan_refusals(b):
    good = tensor(b)
    for kw in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(param=FAKE + 4), dict(grad=FAKE + 4),
               dict(m=FAKE + 4), dict(v=FAKE + 8), dict(copy=FAKE + 8), dict(n=-1), dict(lr_scale=NAN), dict(decay=INF)):
        assert plan(b, good, tensor(b, **kw)) == INVALID, kw
    assert plan(b, good, bits=8) == INVALID                         # no scales
    assert plan(b, tensor(b, m_scale=FAKE, v_scale=FAKE + 2), bits=8) == INVALID
    assert plan(b, good, pdt=2) == INVALID and plan(b, good, gdt=-1) == INVALID and plan(b, good, out=False) == INVALID
    assert plan(b, good, table=None) == INVALID and plan(b, good, table=FAKE + 8) == INVALID and plan(b, count=-1) == INVALID
    assert plan(b, good, bits=16) == UNSUPPORTED and plan(b, good, count=65537) == UNSUPPORTED
    assert plan(b, tensor(b, n=1 << 36)) == UNSUPPORTED and plan(b, *[tensor(b, n=1 << 35)] * 2) == UNSUPPORTED
    need = b._c_adamw_bytes((b.LoftqAdamwTensor * 1)(good), 1)
    assert need > 0 and plan(b, good, table_bytes=need - 1) == WORKSPACE
    assert b._c_adamw_bytes(None, 1) == 0 and b._c_adamw_bytes(None, -1) == 0 and b._c_adamw_bytes(None, 0) > 0


def test_adamw_refusals(b):
    p = b.LoftqAdamwPlan(FAKE, 1, 1, 32, 0, 0)

    def step(lr=0.1, beta1=0.9, beta2=0.999, eps=1e-8, max_norm=0.0, t=1, step=None, lr_factor=None, norm=None, plan=p):
        how = b.LoftqAdamw(lr, beta1, beta2, eps, max_norm, t, step, lr_factor)
        return b._c_adamw(None if plan is None else ctypes.byref(plan), ctypes.byref(how), norm, None)

    for kw in (dict(lr=-0.1), dict(lr=NAN), dict(lr=INF), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=NAN),
               dict(eps=0.0), dict(eps=-1e-8), dict(eps=1e-60), dict(eps=INF), dict(max_norm=-1.0), dict(max_norm=NAN),
               dict(max_norm=INF), dict(t=0), dict(t=-3), dict(step=FAKE + 4), dict(lr_factor=FAKE + 2), dict(norm=FAKE),
               dict(norm=FAKE + 2, max_norm=1.0), dict(plan=None), dict(plan=b.LoftqAdamwPlan(None, 1, 1, 32, 0, 0)),
               dict(plan=b.LoftqAdamwPlan(FAKE, -1, 1, 32, 0, 0))):
        assert step(**kw) == INVALID, kw
    assert b._c_adamw(ctypes.byref(p), None, None, None) == INVALID
    assert step(plan=b.LoftqAdamwPlan(FAKE, 0, 0, 32, 0, 0)) == OK   # nothing to do


def test_binding_refuses_host_tensors(b):
    X, ids = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    B, A = torch.zeros(2, 64, 8), torch.zeros(2, 8, 64)
    with pytest.raises(ValueError):
        b.loftq_adapters_plan(ids, 2)
    with pytest.raises(ValueError):
        b.loftq_adapters_forward(X, B, A, None)
    with pytest.raises(ValueError):
        b.loftq_adapters_backward(X, X, B, A, None)
    with pytest.raises(ValueError):
        b.AdamWTensors([B], [B])


@pytest.mark.parametrize("n,slots,most", [(128, 128, 0.4e9), (8192, 1024, 2.7e9), (8192, 64, 0.3e9), (65536, 512, 1.7e9)])
def test_gradient_workspace_has_no_room_for_sums_that_no_slot_writes(b, n, slots, most):
    """Partial sums are those of slots with more tokens than one workgroup adds: a few, whatever the pool's slots.  What
    grows with the slots is their factors' bf16 forms, (rows + 2 cols) rank 2 bytes each."""
    rows, cols, rank = 11008, 4096, 64
    forms = min(n, slots) * (rows + 2 * cols) * rank * 2
    assert forms < b.adapters_backward_workspace_bytes(n, rows, cols, slots, rank) < most


def test_states_without_their_other_half_are_refused(b):
    """They would be continued as zeros: codes without scales, one moment without the other."""
    p, g = [torch.zeros(300)], [torch.zeros(300)]
    m, v = [torch.zeros(300, dtype=torch.float8_e4m3fn)], [torch.zeros(300, dtype=torch.float8_e5m2)]
    s = [torch.zeros(2)]
    for states in (dict(m=m, v=v), dict(m=m, v=v, m_scale=s), dict(m=m, v=v, v_scale=s)):
        with pytest.raises(ValueError, match="m_scale and v_scale are given with"):
            b.AdamWTensors(p, g, **states)
    for states in (dict(m=m, m_scale=s), dict(v=v, v_scale=s, bits=8), dict(m=p), dict(v=p)):
        with pytest.raises(ValueError, match="m and v are given together"):
            b.AdamWTensors(p, g, **states)
    for states in (dict(m=p, v=p, m_scale=s, v_scale=s), dict(m_scale=s, v_scale=s, bits=8), dict(v_scale=s), dict(m=p, v=p, m_scale=s)):
        with pytest.raises(ValueError, match="m_scale and v_scale belong to"):
            b.AdamWTensors(p, g, **states)


def apart(b, at, n=1000, bits=32, copy=True):
    """A tensor whose pieces lie one behind another from address `at` on, 8192 bytes each."""
    places = [at + 8192 * i for i in range(7)]
    scales = places[4:6] if bits == 8 else (None, None)
    return tensor(b, *places[:4], *scales, places[6] if copy else None, n=n)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt", [(0, 0), (1, 1), (0, 1)])
def test_adamw_refuses_overlapping_tensors(b, bits, pdt, gdt):
    """Two workgroups of a step would read and write the same numbers: a parameter given twice, above all."""
    table, size = 1 << 30, (4, 2)
    one, other = apart(b, 1 << 20, bits=bits), apart(b, 1 << 21, bits=bits)

    def status(*tensors, table=table):
        return plan(b, *tensors, bits=bits, pdt=pdt, gdt=gdt, table=table, table_bytes=1 << 20)

    fields = ["param", "m", "v", "copy"] + (["m_scale", "v_scale"] if bits == 8 else [])
    ends = dict(param=1000 * size[pdt], m=1000 * bits // 8, v=1000 * bits // 8, copy=2000, m_scale=16, v_scale=16)
    assert status(one, other, one) == INVALID
    for name in fields:
        twin = apart(b, 1 << 21, bits=bits)
        setattr(twin, name, getattr(one, name))
        assert status(one, twin) == INVALID, name                     # the same memory
        setattr(twin, name, getattr(one, name) + (ends[name] - 1) // 16 * 16)
        assert status(one, twin) == INVALID, name                     # its last bytes
        assert status(one, other, table=getattr(one, name)) == INVALID
    within = apart(b, 1 << 20, bits=bits)
    within.grad = within.param                                        # read where another workgroup writes
    assert status(within) == INVALID
    across = apart(b, 1 << 21, bits=bits)
    across.grad = one.m
    assert status(one, across) == INVALID and status(across, one) == INVALID


def test_adamw_takes_neighbouring_tensors_and_shared_gradients(b):
    """No overlap: tensors end to end, gradients in common, tensors without elements anywhere.  Without a GPU the launch
    behind the checks fails, on its own account."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    one = tensor(b, *(1 << 20 | 4096 * i for i in range(4)), n=1024)
    next_to = tensor(b, *(1 << 21 | 4096 * i for i in range(4)), n=1024)
    next_to.grad = one.grad
    empty = tensor(b, *(1 << 20 for _ in range(4)), n=0)
    assert plan(b, one, next_to, empty, table=1 << 30) not in (OK, INVALID, UNSUPPORTED, WORKSPACE)
