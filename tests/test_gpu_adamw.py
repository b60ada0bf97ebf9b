"""The AdamW step over many tensors on the GPU against the oracle in fp64.

Bars, with u = 2^-24 (a rounding to nearest in fp32).  m: two products and a sum, the decay's and the clip's
rounding: 6 u (|b1 m| + |(1 - b1) g|).  v: the same with one product more, all terms positive: 8 u v.  p: the
old value's product and the difference, 3 u (|p| + |d|) for a step d, and d itself, whose factors (m, the root
of v, the bias corrections) are off by 6 u of the magnitudes of m, 4 u, and 8 u for its own operations and the 2
ulp of its quotient: 24 u of the step with magnitudes for m.  Parameters in bf16 add half a step, 2^-8 |p|.
8-bit states, as values: half a step of the format (2^-4 of the value for m, 2^-3 for v, or half of the smallest
code's value; all of it for v, which does not round to zero), and the scale's and the quotient's rounding."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HOW = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8)
FLOAT8 = (torch.float8_e4m3fn, torch.float8_e5m2)


def host(t):
    torch.cuda.synchronize()
    return (t.float() if t.dtype in FLOAT8 else t).double().cpu().numpy()


class Model:
    """Tensors of the given lengths, with states after some steps."""

    def __init__(self, lib, sizes, bits=32, param=torch.float32, grad=torch.float32, copies=False, seed=0, decay=0.1,
                 lr_scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(n, std):   # magnitudes over some binades
            return torch.randn(n, generator=g, device="cuda") * std * torch.exp(torch.randn(n, generator=g, device="cuda"))

        self.params = [normal(n, 0.1).to(param) for n in sizes]
        self.grads = [normal(n, 0.01).to(grad) for n in sizes]
        self.decay = [decay] * len(sizes) if not isinstance(decay, list) else decay
        self.lr_scale = [lr_scale] * len(sizes) if not isinstance(lr_scale, list) else lr_scale
        self.copies = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in sizes] if copies else None
        states = dict(m=[normal(n, 0.01) for n in sizes], v=[normal(n, 0.01) ** 2 for n in sizes])
        if bits == 8:
            coded = {k: [oracle.state_codes(x.cpu().numpy(), k) for x in v] for k, v in states.items()}
            for k, dtype in zip("mv", FLOAT8):
                states[k] = [torch.from_numpy(c).cuda().view(dtype) for c, _ in coded[k]]
                states[k + "_scale"] = [torch.from_numpy(s).cuda() for _, s in coded[k]]
        self.bits = bits
        self.tensors = lib.AdamWTensors(self.params, self.grads, copies=self.copies, weight_decay=decay,
                                        lr_scale=lr_scale, **states)

    def values(self):
        t = self.tensors
        out = []
        for i, p in enumerate(self.params):
            m, v = host(t.m[i]), host(t.v[i])
            if self.bits == 8:
                m, v = (oracle.state_values(x.view(torch.uint8).cpu().numpy(), s.cpu().numpy(), k)
                        for x, s, k in ((t.m[i], t.m_scale[i], "m"), (t.v[i], t.v_scale[i], "v")))
            out.append((host(p), host(self.grads[i]), m, v))
        return out

    def check(self, before, t, clip=1.0, **how):
        how = dict(HOW, **how)
        b1, b2 = how["beta1"], how["beta2"]
        for i, ((p, g, m, v), (p1, _, m1, v1)) in enumerate(zip(before, self.values())):
            if p.size == 0:
                continue
            lr = how["lr"] * float(np.float32(self.lr_scale[i]))
            decay = float(np.float32(self.decay[i]))
            want = oracle.adamw_step(p, g, m, v, lr, b1, b2, how["eps"], t, decay, clip)
            size_m = abs(b1 * m) + abs((1 - b1) * clip * g)
            root = np.sqrt(want[2] / (1 - b2 ** t)) + how["eps"]
            d = lr / (1 - b1 ** t) * size_m / root
            tol = 3 * U * (abs(p) + d) + 24 * U * d
            if self.params[i].dtype == torch.bfloat16:
                tol = tol + 2.0 ** -8 * (abs(want[0]) + tol)
            assert np.all(abs(p1 - want[0]) <= tol), np.max(abs(p1 - want[0]) - tol)
            if self.copies is not None:
                assert torch.equal(self.copies[i], self.params[i].bfloat16())
            if self.bits == 32:
                assert np.all(abs(m1 - want[1]) <= 6 * U * size_m)
                assert np.all(abs(v1 - want[2]) <= 8 * U * want[2])
                continue
            for got, ref, size, kind, scale, half in ((m1, want[1], size_m, "m", self.tensors.m_scale[i], 2.0 ** -4),
                                                      (v1, want[2], want[2], "v", self.tensors.v_scale[i], 2.0 ** -3)):
                codes, scales = oracle.state_codes(ref.astype(np.float32), kind)
                s = host(scale)
                assert np.all(abs(s - scales) <= 16 * U * np.abs(scales))
                e, f, bias, _ = oracle.STATE_FORMATS[kind]
                small = 2.0 ** (1 - bias - f) * np.repeat(s, 256)[:ref.size] * (1.0 if kind == "v" else 0.5)
                assert np.all(abs(got - ref) <= np.maximum(half * abs(ref), small) + 16 * U * size)
                # the same code, but where rounding in fp32 reaches a border: 16 u of the value against steps of
                # 2^-3 of it or more, so one in 2^16 of them at most, and a few in such a sample
                same = got == oracle.state_values(codes, s.astype(np.float32), kind)
                assert (~same).sum() <= 2 + same.size // 1000


SIZES = [[1], [3], [4], [255, 256, 257], [4096], [4095, 1, 0, 8193], [64 * 33, 70 * 64, 5]]


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("param", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_step(lib, sizes, bits, param, grad):
    m = Model(lib, sizes, bits, param, grad, seed=len(sizes) + bits)
    for t in (1, 2, 1000):
        before = m.values()
        assert lib.loftq_adamw(m.tensors, t=t, **HOW) is None
        m.check(before, t)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [1e-3, 1e6])
def test_clipping_and_copies(lib, bits, max_norm):
    m = Model(lib, [300, 5000, 64, 100000], bits, copies=True, seed=2)
    before = m.values()
    norm = lib.loftq_adamw(m.tensors, t=3, max_norm=max_norm, **HOW)
    want, clip = oracle.adamw_clip([b[1] for b in before], max_norm)
    assert abs(float(norm) - want) <= 2 * U * want
    m.check(before, 3, clip=clip)


def test_many_tensors(lib):
    """More than one table's worth, of many lengths; each with its own decay and rate."""
    sizes = [(37 * i) % 5000 + 1 for i in range(150)]
    m = Model(lib, sizes, decay=[0.01 * (i % 3) for i in range(150)], lr_scale=[1.0 + i % 4 for i in range(150)], seed=3)
    before = m.values()
    norm = lib.loftq_adamw(m.tensors, t=5, max_norm=0.5, **HOW)
    want, clip = oracle.adamw_clip([b[1] for b in before], 0.5)
    assert abs(float(norm) - want) <= 2 * U * want
    m.check(before, 5, clip=clip)


@pytest.mark.parametrize("bits", [32, 8])
def test_from_nothing(lib, bits):
    """New states are zeros; a zero gradient leaves them so and the parameters but for the decay."""
    p, g = [torch.randn(700, device="cuda")], [torch.zeros(700, device="cuda")]
    t = lib.AdamWTensors(p, g, bits=bits, weight_decay=0.5)
    was = p[0].clone()
    lib.loftq_adamw(t, lr=0.1)
    assert torch.equal(p[0], was * np.float32(1 - 0.1 * 0.5))
    assert not host(t.m[0]).any() and not host(t.v[0]).any()
    if bits == 8:
        assert not t.m_scale[0].any() and not t.v_scale[0].any()
    g[0].copy_(torch.randn(700, device="cuda"))
    was = p[0].clone()
    lib.loftq_adamw(t, lr=0.1, t=1)
    # the first step from nothing: m / (1 - b1) = g and sqrt(v / (1 - b2)) = |g|, so lr g / (|g| + eps), which for a
    # gradient of 4e-5 is 2e-4 of lr less than lr
    want = was.double() * 0.95 - 0.1 * g[0].double() / (g[0].double().abs() + 1e-8)
    assert ((p[0] - want).abs() <= 1e-5 * (1 + want.abs())).all()


def test_small_second_moments_do_not_vanish(lib):
    """A block with one large gradient: the others' v is kept at the smallest code, so that a step stays a step."""
    p, g = [torch.zeros(256, device="cuda")], [torch.full((256,), 1e-6, device="cuda")]
    g[0][7] = 1e3
    t = lib.AdamWTensors(p, g, bits=8)
    lib.loftq_adamw(t, lr=0.1)
    codes = t.v[0].view(torch.uint8)
    assert codes[7] == 0x7B and (codes[torch.arange(256, device="cuda") != 7] == 1).all()
    g[0].zero_()
    was = p[0].clone()
    for k in range(2, 6):
        lib.loftq_adamw(t, lr=0.1, t=k)
    assert ((p[0] - was).abs() <= 4 * 0.1 * 10).all()


@pytest.mark.parametrize("small", [1e-22, 1e-19, 1e-12])
def test_second_moments_below_fp32_keep_the_smallest_code(lib, small):
    """A squared gradient that fp32 cannot hold is still a positive v, beside a block's large one and in a block that
    has no other at its size; where the whole block is below 2^-100 its scale is 0."""
    n = 3 * 256
    p, g = [torch.zeros(n, device="cuda")], [torch.full((n,), small, device="cuda")]
    g[0][7], g[0][300], g[0][511] = 1.0, 1e-3, 0.0
    t = lib.AdamWTensors(p, g, bits=8)
    lib.loftq_adamw(t, lr=0.1)
    codes, scale = t.v[0].view(torch.uint8).cpu(), t.v_scale[0].cpu()
    want = torch.ones(n, dtype=torch.uint8)
    want[7] = want[300] = 0x7B
    want[511] = 0
    if 1e-3 * small ** 2 < 2.0 ** -100:
        want[512:] = 0
        assert scale[2] == 0
    else:
        want[512:] = 0x7B
    assert torch.equal(codes, want) and (scale[:2] > 0).all()


def test_a_small_first_moment_is_divided_by_its_root(lib):
    """Gradients of 5e-6 of the block's largest: m / scale = 448 * 5e-6 = 2.2e-3 keeps a code (the smallest is 2^-9), v / scale
    = 57344 * 2.5e-11 = 1.4e-6 would round to zero (the smallest is 2^-16).  With no gradients afterwards a step is at
    most 0.1 * 0.67 (t = 2: b1 (1 - b1) / (1 - b1^2) sqrt(1 - b2^2) / sqrt(b2 (1 - b2))), times 2 where m's code is
    up to twice m and sqrt(1.5) where v's is down to v / 1.5; over eps alone it would be 0.1 * 200."""
    p, g = [torch.zeros(256, device="cuda")], [torch.full((256,), 1e-2, device="cuda")]
    g[0][7], g[0][8:64], g[0][64:128] = 1.0, 2e-3, 5e-6
    t = lib.AdamWTensors(p, g, bits=8)
    lib.loftq_adamw(t, lr=0.1)
    m, v = t.m[0].view(torch.uint8), t.v[0].view(torch.uint8)
    assert (m[64:128] == 1).all() and (v[64:128] == 1).all() and (m[:64] > 1).all() and (v[:64] > 1).all()
    g[0].zero_()
    for k in range(2, 6):
        was = p[0].clone()
        lib.loftq_adamw(t, lr=0.1, t=k)
        step = (p[0] - was).abs()
        assert (step > 0).all() and (step <= 0.1 * 0.67 * 2 * 1.23).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_gradients_that_are_not_finite(lib, bits, bad):
    m = Model(lib, [600, 300], bits, copies=True, seed=4)
    m.grads[0][300] = bad
    t = m.tensors
    states = [t.m, t.v, m.params, m.copies] + ([t.m_scale, t.v_scale] if bits == 8 else [])
    was = [[x.clone() for x in s] for s in states]
    norm = lib.loftq_adamw(t, max_norm=1.0, **HOW)   # a step that is clipped changes nothing
    assert not torch.isfinite(norm)
    for now, old in zip(states, was):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(now, old))
    lib.loftq_adamw(t, **HOW)                        # one that is not is spoilt where the formulas say
    at = torch.arange(600, device="cuda") != 300
    assert torch.isnan(m.params[0][300]) and torch.isfinite(m.params[0][at]).all() and torch.isfinite(m.params[1]).all()
    if bits == 8:
        assert torch.isnan(t.m_scale[0]).tolist() == [False, True, False] == torch.isnan(t.v_scale[0]).tolist()


def test_step_and_rate_from_the_device(lib):
    a, b = Model(lib, [1000, 77], seed=5), Model(lib, [1000, 77], seed=5)
    step, factor = torch.tensor([6], device="cuda"), torch.tensor([0.25], device="cuda")
    lib.loftq_adamw(a.tensors, t=1, step=step, lr_factor=factor, **HOW)
    lib.loftq_adamw(b.tensors, t=7, **dict(HOW, lr=HOW["lr"] / 4))
    for x, y in zip(a.params + a.tensors.m + a.tensors.v, b.params + b.tensors.m + b.tensors.v):
        # the bias corrections are formed by another library's power, off by an ulp of fp64
        assert torch.equal(x, y) or (x - y).abs().max() <= 2 * U * y.abs().max()


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps(lib, bits):
    """A step in a graph that counts itself, replayed with eager work between, against eager steps."""
    a, b = (Model(lib, [3000, 40, 256], bits, copies=True, seed=6) for _ in range(2))
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    norm = torch.empty((), device="cuda")

    def train(m):
        lib.loftq_adamw(m.tensors, t=1, step=step, max_norm=0.05, norm=norm, **HOW)

    for k in range(2):   # the capture's warm-up, on both
        step.fill_(k)
        train(a), train(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train(a)
        step.add_(1)
    step.fill_(2)
    for k in range(2, 6):
        for x, y in zip(a.grads, b.grads):
            x.copy_(torch.randn_like(x) * 0.01)
            y.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert step.item() == k + 1
        got = norm.clone()
        step.fill_(k)
        train(b)
        step.fill_(k + 1)
        assert torch.equal(got, norm)
        for x, y in zip(a.params + a.copies + a.tensors.m + a.tensors.v, b.params + b.copies + b.tensors.m + b.tensors.v):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_nothing_behind_the_tensors_is_touched(lib):
    for bits in (32, 8):
        sizes = [257, 5, 4099]
        want = Model(lib, sizes, bits, copies=True, seed=7)
        m = Model(lib, sizes, bits, copies=True, seed=7)
        t = m.tensors
        fences, lists = [], dict(params=m.params, grads=m.grads, m=t.m, v=t.v, copies=m.copies)
        if bits == 8:
            lists.update(m_scale=t.m_scale, v_scale=t.v_scale)
        moved = {}
        for k, ts in lists.items():
            moved[k] = []
            for x in ts:
                raw = x.view(torch.uint8)
                big = torch.full((raw.numel() + 4096,), 255, dtype=torch.uint8, device="cuda")
                big[: raw.numel()] = raw
                moved[k].append(big[: raw.numel()].view(x.dtype))
                fences.append(big[raw.numel():])
        fenced = lib.AdamWTensors(moved.pop("params"), moved.pop("grads"), weight_decay=0.1, **moved)
        for tensors in (want.tensors, fenced):
            lib.loftq_adamw(tensors, t=2, max_norm=0.01, **HOW)
        torch.cuda.synchronize()
        assert all((f == 255).all() for f in fences)
        for x, y in zip(fenced.params + fenced.m + fenced.v + fenced.copies,
                        want.params + want.tensors.m + want.tensors.v + want.copies):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_on_another_stream(lib):
    a, b = Model(lib, [100000, 33], seed=8), Model(lib, [100000, 33], seed=8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    norm = lib.loftq_adamw(a.tensors, t=2, max_norm=0.1, stream=side, **HOW)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(norm, lib.loftq_adamw(b.tensors, t=2, max_norm=0.1, **HOW))
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))


def test_binding_checks(lib):
    p, g = [torch.zeros(8, device="cuda")], [torch.zeros(8, device="cuda")]
    with pytest.raises(ValueError):
        lib.AdamWTensors([], [])
    with pytest.raises(ValueError):
        lib.AdamWTensors(p, [torch.zeros(9, device="cuda")])
    with pytest.raises(TypeError):
        lib.AdamWTensors(p, [torch.zeros(8, dtype=torch.float16, device="cuda")])
    with pytest.raises(TypeError):
        lib.AdamWTensors(p, g, copies=[torch.zeros(8, device="cuda")])
    with pytest.raises(lib.LoftqError):
        lib.AdamWTensors(p, g, bits=4)
    with pytest.raises(ValueError):
        lib.AdamWTensors(p, g, weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError):
        lib.AdamWTensors([torch.zeros(8)], g)
    t = lib.AdamWTensors(p, g)
    for how in (dict(t=0), dict(eps=0.0), dict(beta1=1.0), dict(beta2=-0.1), dict(lr=-1.0), dict(lr=float("nan")),
                dict(max_norm=-1.0), dict(max_norm=float("inf")), dict(norm=torch.zeros((), device="cuda"))):
        with pytest.raises(lib.LoftqError):
            lib.loftq_adamw(t, **{"lr": 0.1, **how})


def test_binding_refuses_lists_of_another_length(lib):
    p, g = ([torch.zeros(8, device="cuda") for _ in range(2)] for _ in range(2))
    for grads, more in ((g[:1], {}), ([], {}), (g, dict(m=[], v=g)), (g, dict(m=g[:1], v=g)), (g, dict(m=g, v=g[:1])),
                        (g, dict(copies=[]))):
        with pytest.raises(ValueError):
            lib.AdamWTensors(p, grads, **more)


@pytest.mark.parametrize("bits", [32, 8])
def test_states_made_on_another_stream(lib, bits):
    """The states that the tensors make for themselves, on a stream that is not the steps'."""
    p = [torch.ones(5000, device="cuda"), torch.ones(3, device="cuda")]
    q, g = [x.clone() for x in p], [torch.full_like(x, 0.5) for x in p]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = lib.AdamWTensors(p, g, bits=bits, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b = lib.AdamWTensors(q, g, bits=bits)
    for t in (1, 2):
        lib.loftq_adamw(a, lr=0.1, t=t)
        lib.loftq_adamw(b, lr=0.1, t=t)
    assert all(torch.equal(x, y) and not torch.equal(x, torch.ones_like(x)) for x, y in zip(p, q))


@pytest.mark.parametrize("max_norm", [0.0, 0.05])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_codes_are_the_nearest(lib, grad, max_norm):
    """Every code of the new states is the one nearest to the moment's quotient in fp64 (ties to the even code): what a
    rounding to fp32 in between would decide, a code in a million or so, is not left to it."""
    a = Model(lib, [300000, 4097], bits=8, grad=grad, seed=31)

    def whole(codes, scale, kind):   # the product of code and scale in fp64: 4 or 3 bits by 24
        ones = np.ones(scale.numel(), np.float32)
        return oracle.state_values(codes.view(torch.uint8).cpu().numpy(), ones, kind) * np.repeat(host(scale), 256)[:codes.numel()]

    t = a.tensors
    before = [(p, host(g), whole(t.m[i], t.m_scale[i], "m"), whole(t.v[i], t.v_scale[i], "v"))
              for i, (p, g) in enumerate(zip(a.params, a.grads))]
    norm, clip = oracle.adamw_clip([x[1] for x in before], max_norm) if max_norm else (0.0, 1.0)
    lib.loftq_adamw(a.tensors, t=3, max_norm=max_norm, **HOW)
    b1, b2 = HOW["beta1"], HOW["beta2"]
    for i, (_, g, m0, v0) in enumerate(before):
        want = dict(m=b1 * m0 + (1 - b1) * (clip * g), v=b2 * v0 + ((1 - b2) * (clip * g)) * (clip * g))
        for kind, codes, scale in (("m", t.m[i], t.m_scale[i]), ("v", t.v[i], t.v_scale[i])):
            levels = oracle.state_values(np.arange(127 if kind == "m" else 124, dtype=np.uint8), np.ones(1, np.float32), kind)
            x, s = want[kind], np.repeat(host(scale), 256)[:g.size]
            y = np.abs(x / s)
            at = np.clip(np.searchsorted(levels, y), 1, levels.size - 1)
            lo, hi = y - levels[at - 1], levels[at] - y
            code = np.where((lo < hi) | ((lo == hi) & (at % 2 == 1)), at - 1, at)
            if kind == "v":
                code = np.where(x > 0, np.maximum(code, 1), code)
            got = codes.view(torch.uint8).cpu().numpy()
            assert np.array_equal(got & 127, code)
            assert np.array_equal(got >= 128, np.signbit(x))


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_scales_are_the_products(lib, grad):
    """Every new scale, bit for bit: the block's largest moment (formed in fp64, rounded to fp32) times the rounded inverse
    of the format's top, 0 below 2^-100."""
    n = 256 * 700 + 33
    a = Model(lib, [n], bits=8, grad=grad, seed=33)
    t = a.tensors
    size = torch.exp2(-torch.arange(701, device="cuda") / 8.0)         # from 1 down to 2^-88, whose squares pass 2^-100
    a.grads[0].mul_(size.repeat_interleave(256)[:n].to(grad))
    t.m_scale[0].mul_(size), t.v_scale[0].mul_(size * size)

    def whole(codes, scale, kind):   # the product of code and scale in fp64
        ones = np.ones(scale.numel(), np.float32)
        return oracle.state_values(codes.view(torch.uint8).cpu().numpy(), ones, kind) * np.repeat(host(scale), 256)[:n]

    g, m, v = host(a.grads[0]), whole(t.m[0], t.m_scale[0], "m"), whole(t.v[0], t.v_scale[0], "v")
    lib.loftq_adamw(t, t=3, **HOW)
    b1, b2 = HOW["beta1"], HOW["beta2"]
    for x, scale, kind in ((b1 * m + (1 - b1) * g, t.m_scale[0], "m"), (b2 * v + ((1 - b2) * g) * g, t.v_scale[0], "v")):
        amax = np.abs(np.concatenate([x, np.zeros(-n % 256)])).reshape(-1, 256).max(1).astype(np.float32)
        want = np.where(amax < np.float32(2.0 ** -100), np.float32(0), amax * (np.float32(1) / np.float32(oracle.STATE_FORMATS[kind][3])))
        assert kind == "m" or ((want == 0).any() and (want > 0).any())
        assert np.array_equal(scale.cpu().numpy(), want.astype(np.float32))


@pytest.mark.parametrize("bits", [32, 8])
def test_offsets_past_32_bits(lib, bits):
    """The last elements of a tensor of more than 2^32 are stepped as those of a tensor of their own."""
    n, tail = (1 << 32) + 4096 + 77, 512 + 77
    g = torch.Generator(device="cuda").manual_seed(8)
    end = dict(params=torch.randn(tail, generator=g, device="cuda"), grads=torch.randn(tail, generator=g, device="cuda"))

    def large(x):
        out = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
        out[-tail:] = x
        return [out]

    big = {k: large(x) for k, x in end.items()}
    small = {k: [x.bfloat16()] for k, x in end.items()}
    a, b = (lib.AdamWTensors(x["params"], x["grads"], bits=bits) for x in (big, small))
    for t in (1, 2):
        norms = [lib.loftq_adamw(x, t=t, max_norm=0.5, **HOW) for x in (a, b)]
        assert torch.equal(*norms)
    assert torch.equal(big["params"][0][-tail:], small["params"][0]) and not big["params"][0][:-tail].any()
    for x, y in ((a.m, b.m), (a.v, b.v)):
        assert torch.equal(x[0][-tail:].view(torch.uint8), y[0].view(torch.uint8))
    if bits == 8:
        assert torch.equal(a.m_scale[0][-3:], b.m_scale[0]) and torch.equal(a.v_scale[0][-3:], b.v_scale[0])


def test_as_many_tensors_as_a_step_takes(lib):
    count = 65536
    p, g = (torch.randn(count, 4, generator=torch.Generator(device="cuda").manual_seed(k), device="cuda") for k in (1, 2))
    q, m, v, m1, v1 = p.clone(), *(torch.zeros_like(p) for _ in range(4))
    for tensors in (lib.AdamWTensors(list(p), list(g), m=list(m), v=list(v)), lib.AdamWTensors([q], [g], m=[m1], v=[v1])):
        norm = lib.loftq_adamw(tensors, max_norm=1.0, **HOW)
    assert abs(float(norm) - float(g.double().norm())) <= 2 * U * float(norm)
    # the norms may be added in another order, which an element's rounding can show
    for x, y in ((p, q), (m, m1), (v, v1)):
        assert ((x - y).abs() <= 8 * U * y.abs()).all()
    with pytest.raises(lib.LoftqError) as e:
        lib.AdamWTensors([*p, q[0]], [*g, g[0]])
    assert e.value.status == 2
