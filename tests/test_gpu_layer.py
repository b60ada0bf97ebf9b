"""The training and serving operators of an adapted layer on the GPU against the oracle's
formulas in fp64: dropout, MXFP4 quantization, the training forward and the gradient over
an NF4 and an MXFP4 base.

Bars.  Operands are the oracle's own bf16 (or FP4) values, so every product of two is exact
in fp32 and what differs is rounding of sums.  A sum of N terms added in fp32 in any order is
off by at most (N - 1) u sum |terms|, with u = 2^-23 per addition (nearest rounding has 2^-24;
the matrix cores may truncate), and a second product over the sums adds its own count:
    Y, dX:  (K + cols + 4 r + 16) u S,   K the base's sum, S the same formula on magnitudes
    dB, dA: (n + K' + 16) u S,           K' = cols for dB (through X A^T), rows for dA
where the 16 covers the joins of partial sums, the three-piece split of the inner sums
(2^-24 of each) and the last multiplications.  An output in bf16 adds half a step, 2^-8 |y|.
Errors of either sign mostly cancel, so the norm of an fp32 output's error must also stay
under 1e-6 of the output's norm."""
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


class Layer:
    """A random adapted layer on the host (fp64 values) and the device."""

    def __init__(self, n, rows, cols, r, base="nf", dq=False, bits=4, seed=0):
        g = np.random.default_rng(seed)
        self.shape, self.n, self.r, self.base = (rows, cols), n, r, base
        self.X, self.G = bf16(g.standard_normal((n, cols))), bf16(g.standard_normal((n, rows)))
        self.Xd, self.Gd = dev(self.X, torch.bfloat16), dev(self.G, torch.bfloat16)
        self.A = self.B = self.Ad = self.Bd = None
        if r:
            A, B = (0.1 * g.standard_normal(s).astype(np.float32) for s in ((r, cols), (rows, r)))
            self.A, self.B, self.Ad, self.Bd = bf16(A), bf16(B), dev(A), dev(B)
        if base == "mx":
            codes, byte = oracle.mx_quantize((0.05 * g.standard_normal((rows, cols))).astype(np.float32))
            packed, scales = oracle.mx_pack(codes, byte)
            self.W = oracle.mx_values(codes, byte, cols)
            self.kw = dict(packed=dev(packed, torch.uint8), scales=dev(scales, torch.uint8))
            return
        codes = g.integers(0, 1 << bits, rows * cols).astype(np.uint8)
        nb = rows * cols // 64
        self.kw = dict(packed=dev(oracle.pack_nibbles(codes), torch.uint8), bits=bits)
        if dq:
            qa = g.integers(1, 128, nb).astype(np.int8)
            dqs = (0.05 / 127 * (0.5 + g.random((nb + 255) // 256))).astype(np.float32)
            self.kw.update(qabsmax=dev(qa, torch.int8), dq_scale=dev(dqs))
            scale = oracle.dq_scales_expand(qa, dqs)
        else:
            scale = (0.05 * (0.25 + np.abs(g.standard_normal(nb)))).astype(np.float32)
            self.kw.update(absmax=dev(scale))
        self.W = bf16(oracle.dequantize(codes, scale, 64, codebook=oracle.nf_codebook(bits)).reshape(rows, cols))

    def keep(self, p, seed, offset):
        return oracle.keep_mask(self.X.shape, p, seed, offset) if p else None

    def forward(self, lib, alpha=1.5, p=0.0, seed=0, offset=0, **more):
        f = lib.loftq_mxfp4_forward if self.base == "mx" else lib.loftq_qlora_forward_dropout
        return f(self.Xd, shape=self.shape, B=self.Bd, A=self.Ad, alpha=alpha, p=p, seed=seed, offset=offset, **self.kw,
                 **more)

    def backward(self, lib, alpha=1.5, p=0.0, seed=0, offset=0, **more):
        f = lib.loftq_mxfp4_backward if self.base == "mx" else lib.loftq_qlora_backward
        return f(self.Gd, self.Xd, shape=self.shape, B=self.Bd, A=self.Ad, alpha=alpha, p=p, seed=seed, offset=offset,
                 **self.kw, **more)

    def xq(self):
        if self.base != "mx":
            return self.X
        codes, byte = oracle.mx_quantize(self.X.astype(np.float32))
        return oracle.mx_values(codes, byte, self.shape[1])

    def check_forward(self, Y, alpha=1.5, p=0.0, seed=0, offset=0):
        gain, keep, xq = alpha * oracle.drop_scale(p), self.keep(p, seed, offset), self.xq()
        mag = [None if v is None else np.abs(v) for v in (self.X, self.W, self.A, self.B)]
        ref = oracle.layer_forward(self.X, self.W, self.A, self.B, gain, keep, xq)
        S = oracle.layer_forward(*mag, abs(gain), keep, np.abs(xq))
        check(Y, ref, (2 * self.shape[1] + 4 * self.r + 16) * U * S)

    def check_backward(self, grads, alpha=1.5, p=0.0, seed=0, offset=0):
        gain, keep = alpha * oracle.drop_scale(p), self.keep(p, seed, offset)
        mag = [None if v is None else np.abs(v) for v in (self.G, self.X, self.W, self.A, self.B)]
        ref = oracle.layer_backward(self.G, self.X, self.W, self.A, self.B, gain, keep)
        S = oracle.layer_backward(*mag, abs(gain), keep)
        rows, cols = self.shape
        for got, want, s, k in zip(grads, ref, S or (), (2 * rows + 4 * self.r, self.n + cols, self.n + rows)):
            if got is not None:
                check(got, want, (k + 16) * U * s)


def check(got, ref, tol):
    y = host(got)
    assert y.shape == ref.shape
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(y - ref)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert np.all(err <= tol), (worst, y[worst], ref[worst], tol[worst])
    if got.dtype == torch.float32 and np.linalg.norm(ref) > 0:
        assert np.linalg.norm(err) <= 1e-6 * np.linalg.norm(ref)


# ---- dropout ----

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 3, 4, 7, 8, 9, 4096, 100003])
def test_dropout(lib, n, dtype):
    g = np.random.default_rng(n)
    X = dev(g.standard_normal(n).astype(np.float32), dtype)
    for p, seed, offset in ((0.1, 42, 0), (0.5, 2 ** 63 + 11, 9)):
        Y = lib.loftq_dropout(X, p, seed, offset)
        # the product with fl32(scale) in fp32, rounded once: exact to repeat on the host
        keep = oracle.keep_mask((n,), p, seed, offset)
        want = torch.where(torch.from_numpy(keep), (X.float() * oracle.drop_scale(p)).to(dtype).cpu(), torch.zeros((), dtype=dtype))
        assert torch.equal(Y.cpu(), want)


def test_dropout_ends_and_in_place(lib):
    X = torch.randn(33, 65, device="cuda")
    assert torch.equal(lib.loftq_dropout(X, 0.0, 1), X)
    assert torch.equal(lib.loftq_dropout(X, 1.0, 1), torch.zeros_like(X))
    want = lib.loftq_dropout(X, 0.3, 1, 2)
    assert lib.loftq_dropout(X, 0.3, 1, 2, out=X) is X and torch.equal(X, want)
    assert lib.loftq_dropout(X[:0], 0.3, 1).shape == (0, 65)


def test_dropout_drops_what_is_not_finite(lib):
    keep = torch.from_numpy(oracle.keep_mask((64, 64), 0.5, 5, 6)).cuda()
    for bad in (float("nan"), float("inf"), -torch.finfo(torch.float32).max):
        X = torch.where(keep, torch.ones((), device="cuda"), torch.full((), bad, device="cuda"))
        assert torch.equal(lib.loftq_dropout(X, 0.5, 5, 6), 2.0 * keep)
        Y = lib.loftq_dropout(torch.full((64, 64), bad, device="cuda"), 0.5, 5, 6)
        assert (Y[~keep] == 0).all() and not torch.isfinite(Y[keep]).any()


def test_dropout_step_and_stream(lib):
    X = torch.randn(1000, device="cuda")
    step = torch.tensor([3], device="cuda")
    assert torch.equal(lib.loftq_dropout(X, 0.2, 8, 4, step=step), lib.loftq_dropout(X, 0.2, 8, 7))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(X)
    lib.loftq_dropout(X, 0.2, 8, 7, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, lib.loftq_dropout(X, 0.2, 8, 7))


def test_dropout_past_32_bits(lib):
    n = (1 << 32) + 24
    X = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    lib.loftq_dropout(X, 0.5, 1, 2, out=X)
    for first in (0, (1 << 32) - 1000, n - 1000):
        keep = oracle.keep_mask((1000,), 0.5, 1, 2, first=first)
        assert np.array_equal(host(X[first:first + 1000]), 2.0 * keep)


# ---- MXFP4 ----

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 255), (4, 256), (3, 257), (17, 1000), (64, 4104)])
def test_mx_quantize(lib, rows, cols, dtype):
    g = np.random.default_rng(rows * 10000 + cols)
    # magnitudes over many binades, zeros, and one block of zeros
    R = g.standard_normal((rows, cols)) * 2.0 ** g.integers(-30, 30, (rows, cols))
    R[g.random((rows, cols)) < 0.1] = 0.0
    R[0, :32] = 0.0
    W = dev(R.astype(np.float32), dtype)
    packed, scales = lib.loftq_mxfp4_quantize(W)
    Wh = host(W).astype(np.float32)
    codes, byte = oracle.mx_quantize(Wh)
    want_packed, want_scales = oracle.mx_pack(codes, byte)
    assert np.array_equal(scales.cpu().numpy(), want_scales)
    assert np.array_equal(packed.cpu().numpy(), want_packed)
    v = oracle.mx_values(codes, byte, cols)
    for odt, half in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
        got = lib.loftq_mxfp4_dequantize(packed, scales, (rows, cols), out_dtype=odt)
        assert torch.equal(got.cpu(), torch.from_numpy(v).to(odt))
        E = host(lib.loftq_mxfp4_dequantize(packed, scales, (rows, cols), W=W, out_dtype=odt))
        ref = Wh.astype(np.float64) - v
        assert np.all(np.abs(E - ref) <= (half + 2.0 ** -24) * np.abs(ref))


def test_mx_every_code_and_border(lib):
    # each representable magnitude, each border between two and its neighbours, both signs, over many scales
    ulp = 2.0 ** -20
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    x = [v for m in mids for v in (m - ulp, m, m + ulp)] + list(oracle.E2M1) + [7.99]
    row = np.zeros(64)
    row[:len(x)] = x
    row[31] = row[63] = 6.0   # both blocks at scale 1
    R = np.stack([s * row * 2.0 ** e for e in (-120, -60, -3, 0, 1, 60, 120) for s in (1, -1)]).astype(np.float32)
    packed, scales = lib.loftq_mxfp4_quantize(dev(R))
    want_packed, want_scales = oracle.mx_pack(*oracle.mx_quantize(R))
    assert np.array_equal(scales.cpu().numpy(), want_scales) and np.array_equal(packed.cpu().numpy(), want_packed)


def test_mx_ends_of_the_range(lib):
    tiny, big = 2.0 ** -149, 3.4e38
    R = np.zeros((6, 32), dtype=np.float32)
    R[0, :3] = tiny, 2.0 ** -126, 2.0 ** -127
    R[1, :3] = big, -big, 1.0
    R[2, :2] = np.inf, 1.0
    R[3, :2] = 1.0, np.nan
    R[4, :2] = -0.0, 2.0 ** -128
    R[5, :2] = 2.0 ** -124, 2.0 ** -127
    packed, scales = lib.loftq_mxfp4_quantize(dev(R))
    codes, byte = oracle.mx_quantize(R)
    assert np.array_equal(scales.cpu().numpy(), oracle.mx_pack(codes, byte)[1])
    v = oracle.mx_values(codes, byte, 32)
    got = host(lib.loftq_mxfp4_dequantize(packed, scales, (6, 32)))
    assert np.array_equal(np.isnan(got), np.isnan(v)) and np.isnan(got[2:4]).all()
    fine = ~np.isnan(v)
    assert np.array_equal(got[fine], v[fine])


@pytest.mark.parametrize("r", [1, 16, 70])
def test_mx_quantize_residual(lib, r):
    """R = W - B A: codes may differ from the exact residual's only where fp32's rounding of R reaches a border."""
    g = np.random.default_rng(r)
    rows, cols = 24, 500
    W, B, A = (g.standard_normal(s).astype(np.float32) for s in ((rows, cols), (rows, r), (r, cols)))
    packed, scales = lib.loftq_mxfp4_quantize(dev(W), dev(B), dev(A))
    got = host(lib.loftq_mxfp4_dequantize(packed, scales, (rows, cols)))
    BA = B.astype(np.float64) @ A
    R = W - BA
    off = (r + 2) * 2.0 ** -24 * (np.abs(W) + np.abs(B).astype(np.float64) @ np.abs(A))
    # the value of R + d for every |d| <= off lies between those of R - off and R + off, at the block's scale or,
    # where the largest magnitude may cross a power of two, at a neighbouring one: half a step, at most amax / 6,
    # or what saturates, amax / 4
    amax = np.zeros((rows, 512))
    amax[:, :cols] = np.abs(R)
    amax = np.repeat(amax.reshape(rows, -1, 32).max(2), 32, axis=1)[:, :cols]
    assert np.all(np.abs(got - R) <= 0.25 * amax * (1 + 2.0 ** -10) + off)
    codes, byte = oracle.mx_quantize(R.astype(np.float32))
    same = got == oracle.mx_values(codes, byte, cols)
    assert same.mean() > 0.999


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,r", [(1, 1, 1), (2, 31, 3), (3, 256, 2), (4, 257, 5), (5, 40, 17), (6, 1000, 64),
                                         (7, 33, 4), (9, 300, 16)])
def test_mx_quantize_residual_exact(lib, rows, cols, r, dtype):
    """Small integers make R exact: every byte is the oracle's, with any number of rows, and the padding is zero also
    where B holds an infinity."""
    g = np.random.default_rng(rows * 1000 + cols)
    W = g.integers(-64, 65, (rows, cols)).astype(np.float32)
    B = g.integers(-3, 4, (rows, r)).astype(np.float32)
    A = g.integers(-3, 4, (r, cols)).astype(np.float32)
    for last in (2.0, np.inf):
        B[rows - 1, r - 1] = last
        with np.errstate(invalid="ignore"):
            codes, byte = oracle.mx_quantize((W - B @ A).astype(np.float32))
        want_packed, want_scales = oracle.mx_pack(codes, byte)
        packed, scales = lib.loftq_mxfp4_quantize(dev(W, dtype), dev(B), dev(A))
        assert np.array_equal(scales.cpu().numpy(), want_scales)
        packed = packed.cpu().numpy()
        finite = rows if last == 2.0 else rows - 1   # the codes beside a scale of 255 are free
        assert np.array_equal(packed[:finite], want_packed[:finite])
        assert not packed[:, (cols + 31) // 32 * 16:].any()


# ---- the layer's forward and gradient ----

SHAPES = [  # n, rows, cols, r, base, dq, bits
    (1, 1, 64, 1, "nf", False, 4), (1, 37, 64, 5, "nf", True, 4), (2, 64, 192, 16, "nf", False, 2),
    (31, 129, 320, 17, "nf", True, 3), (33, 100, 64, 0, "nf", False, 4), (65, 257, 640, 64, "nf", True, 4),
    (130, 384, 1024, 33, "nf", False, 4), (257, 260, 128, 48, "nf", True, 4),
    (1, 1, 32, 1, "mx", False, 4), (1, 48, 256, 16, "mx", False, 4), (3, 33, 96, 9, "mx", False, 4),
    (64, 130, 288, 64, "mx", False, 4), (70, 255, 544, 0, "mx", False, 4), (129, 512, 1056, 20, "mx", False, 4),
    (300, 333, 512, 64, "mx", False, 4), (16, 70, 416, 3, "mx", False, 4), (17, 129, 2080, 64, "mx", False, 4),
    (32, 48, 4128, 16, "mx", False, 4), (33, 48, 4128, 16, "mx", False, 4),
]


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_forward(lib, case, p):
    layer = Layer(*case, seed=sum(case[:4]))
    rng = dict(p=p, seed=77, offset=5)
    for dtype in (torch.float32, torch.bfloat16):
        layer.check_forward(layer.forward(lib, out_dtype=dtype, **rng), **rng)


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_backward(lib, case, p):
    layer = Layer(*case, seed=sum(case[:4]) + 1)
    rng = dict(p=p, seed=78, offset=6)
    for dtype in (torch.float32, torch.bfloat16):
        grads = layer.backward(lib, dx_dtype=dtype, **rng)
        assert (grads[1] is None) == (case[3] == 0)
        layer.check_backward(grads, **rng)


@pytest.mark.parametrize("base", ["nf", "mx"])
@pytest.mark.parametrize("n,rows,cols", [(1100, 1100, 1088), (2100, 512, 1024), (520, 2304, 512)])
def test_large_tiles(lib, base, n, rows, cols):
    layer = Layer(n, rows, cols, 24, base, seed=9)
    rng = dict(p=0.25, seed=3, offset=1)
    layer.check_forward(layer.forward(lib, **rng), **rng)
    layer.check_backward(layer.backward(lib, dx_dtype=torch.float32, **rng), **rng)


@pytest.mark.parametrize("base", ["nf", "mx"])
def test_everything_dropped(lib, base):
    layer = Layer(20, 64, 128, 8, base, seed=2)
    rng = dict(p=1.0, seed=3, offset=1)
    layer.check_forward(layer.forward(lib, **rng), **rng)
    dX, dB, dA = layer.backward(lib, **rng)
    layer.check_backward((dX, dB, dA), **rng)
    assert not dB.any() and not dA.any()


@pytest.mark.parametrize("base", ["nf", "mx"])
def test_gradient_against_differences(lib, base):
    """Y is linear in B (and in A) for the other at rest, and values that are bf16 already pass the factors' rounding:
    between B = 0 and B = step, <G, Y> changes by <dB, step>, up to the rounding of the sums."""
    layer = Layer(48, 96, 128, 16, base, seed=4)
    rng = dict(p=0.2, seed=1, offset=2)
    _, dB, dA = layer.backward(lib, **rng)
    for name, grad in (("Bd", dB), ("Ad", dA)):
        old = getattr(layer, name)
        step = torch.randn_like(old).bfloat16().float()
        # <G, Y(step) - Y(0)> = <grad, step>
        setattr(layer, name, step)
        moved = host(layer.forward(lib, **rng))
        setattr(layer, name, torch.zeros_like(step))
        still = host(layer.forward(lib, **rng))
        setattr(layer, name, old)
        change = (layer.G * (moved - still)).sum()
        size = (np.abs(layer.G) * (np.abs(moved) + np.abs(still))).sum()
        assert abs(change - (host(grad) * host(step)).sum()) <= 4 * (48 + 96 + 128) * U * size


def test_parts_of_the_gradient(lib):
    layer = Layer(40, 70, 128, 8, seed=5)
    rng = dict(p=0.1, seed=1, offset=2)
    dX, dB, dA = layer.backward(lib, **rng)
    only = layer.backward(lib, need_dx=False, **rng)
    assert only[0] is None and torch.equal(only[1], dB) and torch.equal(only[2], dA)
    out = torch.full_like(dX, 7.0)
    got = layer.backward(lib, out=(out, None, None), **rng)
    assert got[0] is out and torch.equal(out, dX)
    x, layer.Xd = layer.Xd, None   # the input is not needed for dX
    assert torch.equal(layer.backward(lib, out=(out, None, None), **rng)[0], dX)
    layer.Xd = x


def test_no_tokens(lib):
    layer = Layer(0, 64, 128, 8, seed=5)
    assert layer.forward(lib).shape == (0, 64)
    dX, dB, dA = layer.backward(lib)
    assert dX.shape == (0, 128) and not dB.any() and not dA.any()


def test_outputs_are_overwritten_and_nothing_else(lib):
    """Stale and unfinished contents of the workspace and of what lies behind the outputs do not matter, and stay."""
    layer = Layer(45, 99, 192, 8, seed=6)
    rng = dict(p=0.1, seed=1, offset=2)
    want = [t.clone() for t in layer.backward(lib, **rng)]
    need = lib.qlora_backward_workspace_bytes(45, 99, 192, 8)
    for fill in (0, 255):   # 255: NaN in every type
        ws = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
        bufs = [torch.full((t.numel() + 64,), float("nan"), dtype=t.dtype, device="cuda") for t in want]
        out = [b[: t.numel()].view(t.shape) for b, t in zip(bufs, want)]
        layer.backward(lib, out=out, ws=ws[:need], **rng)
        for o, b, t in zip(out, bufs, want):
            assert torch.equal(o, t) and torch.isnan(b[t.numel():]).all()
        assert (ws[need:] == fill).all()


@pytest.mark.parametrize("base,n,rows,cols", [("nf", 45, 100, 192), ("nf", 70, 128, 320), ("mx", 13, 96, 96), ("mx", 77, 130, 288)])
def test_nothing_behind_the_inputs_is_used(lib, base, n, rows, cols):
    """Inputs that end where NaN begins (every byte 255 behind each) give what they give by themselves."""
    layer = Layer(n, rows, cols, 20, base, seed=19)
    rng = dict(p=0.3, seed=9, offset=1)
    want = (layer.forward(lib, **rng), layer.forward(lib), *layer.backward(lib, **rng))

    def fenced(t):
        raw = t.contiguous().view(torch.uint8).reshape(-1)
        big = torch.full((raw.numel() + (1 << 16),), 255, dtype=torch.uint8, device="cuda")
        big[: raw.numel()] = raw
        return big[: raw.numel()].view(t.dtype).view(t.shape)

    for name in ("Xd", "Gd", "Ad", "Bd"):
        setattr(layer, name, fenced(getattr(layer, name)))
    layer.kw = {k: fenced(v) if torch.is_tensor(v) else v for k, v in layer.kw.items()}
    got = (layer.forward(lib, **rng), layer.forward(lib), *layer.backward(lib, **rng))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("n", [7, 300])
def test_mx_forward_of_what_is_not_finite(lib, n):
    """A NaN or an infinity makes its block of 32 columns NaN, and with it its token's results, and no other's."""
    layer = Layer(n, 96, 288, 8, "mx", seed=15)
    clean = layer.forward(lib)
    for bad in (float("nan"), float("inf")):
        X = layer.Xd
        layer.Xd = X.clone()
        layer.Xd[2, 287] = bad
        Y = layer.forward(lib)
        layer.Xd = X
        others = torch.arange(n, device="cuda") != 2
        assert torch.isnan(Y[2]).all() and torch.equal(Y[others], clean[others])
    layer.kw["scales"] = layer.kw["scales"].clone()
    layer.kw["scales"][1, 5, 0] = 255   # a NaN block of the weight's row 5
    Y = layer.forward(lib)
    rows = torch.arange(96, device="cuda") != 5
    assert torch.isnan(Y[:, 5]).all() and torch.equal(Y[:, rows], clean[:, rows])


@pytest.mark.parametrize("base", ["nf", "mx"])
def test_what_is_not_finite_stays_where_it_belongs(lib, base):
    layer = Layer(40, 64, 128, 8, base, seed=7)
    rng = dict(p=0.5, seed=1, offset=2)
    keep = oracle.keep_mask((40, 128), 0.5, 1, 2)
    clean = layer.backward(lib, **rng)
    X = layer.Xd
    layer.Xd = torch.where(torch.from_numpy(keep).cuda(), X, torch.full_like(X, float("nan")))
    got = layer.backward(lib, **rng)   # NaN only where X is dropped
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    layer.Xd = X.clone()
    layer.Xd[11] = float("nan")
    Y = layer.forward(lib, **rng)
    layer.Xd = X
    rows = torch.arange(40, device="cuda")
    assert torch.isnan(Y[11]).all() and torch.equal(Y[rows != 11], layer.forward(lib, **rng)[rows != 11])
    G = layer.Gd
    layer.Gd = G.clone()
    layer.Gd[3, 5] = float("inf")
    dX, dB, dA = layer.backward(lib, **rng)
    layer.Gd = G
    assert not torch.isfinite(dX[3]).any() and torch.equal(dX[rows != 3], clean[0][rows != 3])
    feat = torch.arange(64, device="cuda")
    assert torch.equal(dB[feat != 5], clean[1][feat != 5]) and not torch.isfinite(dB[5]).any()
    # dA: the columns that token 3 keeps
    kept = torch.from_numpy(keep[3]).cuda()
    assert torch.equal(dA[:, ~kept], clean[2][:, ~kept]) or torch.isnan(dA[:, ~kept]).any()


@pytest.mark.parametrize("base", ["nf", "mx"])
def test_same_results_again_and_on_a_stream(lib, base):
    layer = Layer(200, 320, 512, 16, base, dq=base == "nf", seed=8)
    rng = dict(p=0.1, seed=1, offset=2)
    Y, grads = layer.forward(lib, **rng), layer.backward(lib, **rng)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Y2, grads2 = layer.forward(lib, **rng), layer.backward(lib, **rng)
    side.synchronize()
    assert torch.equal(Y, Y2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    two = zero + 2
    assert torch.equal(layer.forward(lib, p=0.1, seed=1, step=two), Y)


def test_two_streams_at_once(lib):
    """Calls with workspaces of their own may overlap on two streams."""
    a, b = Layer(300, 512, 1024, 16, "nf", seed=16), Layer(280, 448, 992, 32, "mx", seed=17)
    rng = dict(p=0.2, seed=5, offset=1)
    want = [(x.forward(lib, **rng), *x.backward(lib, **rng)) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append((x.forward(lib, **rng), *x.backward(lib, **rng)))
    torch.cuda.synchronize()
    for i in range(2):
        for once in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(once, want[i]))


def test_captured_serving(lib):
    """The few-token and the tiled product over MXFP4 in one graph, sharing a workspace, replayed on new inputs."""
    layer = Layer(40, 192, 288, 16, "mx", seed=18)
    ws = torch.empty(lib.mxfp4_forward_workspace_bytes(40, 192, 288, 16), dtype=torch.uint8, device="cuda")
    X = layer.Xd.clone()
    one, many = torch.empty(1, 192, device="cuda"), torch.empty(40, 192, device="cuda")
    kw = dict(shape=layer.shape, B=layer.Bd, A=layer.Ad, alpha=0.5, ws=ws, **layer.kw)

    def serve():
        lib.loftq_mxfp4_forward(X, out=many, **kw)
        lib.loftq_mxfp4_forward(X[:1], out=one, **kw)

    serve()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        serve()
    for k in range(4):
        X.copy_(torch.randn(40, 288, device="cuda"))
        graph.replay()
        got = one.clone(), many.clone()
        serve()
        torch.cuda.synchronize()
        assert torch.equal(got[0], one) and torch.equal(got[1], many)
        layer.X, layer.Xd = X.double().cpu().numpy(), X
        layer.check_forward(many, alpha=0.5)
        layer.X = layer.X[:1]
        layer.check_forward(one, alpha=0.5)


def test_captured_training_step(lib):
    """Forward and gradient in one graph that counts its own step: each replay draws that step's mask."""
    layer = Layer(96, 192, 256, 16, dq=True, seed=10)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    nf = layer.shape
    wf = torch.empty(lib.qlora_forward_dropout_workspace_bytes(96, *nf, 16), dtype=torch.uint8, device="cuda")
    wb = torch.empty(lib.qlora_backward_workspace_bytes(96, *nf, 16), dtype=torch.uint8, device="cuda")
    Y = torch.empty(96, 192, device="cuda")
    out = (torch.empty(96, 256, dtype=torch.bfloat16, device="cuda"), torch.empty_like(layer.Bd), torch.empty_like(layer.Ad))

    def train():
        layer.forward(lib, p=0.3, seed=4, offset=0, step=step, out=Y, ws=wf)
        layer.backward(lib, p=0.3, seed=4, offset=0, step=step, out=out, ws=wb)
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
        want = [layer.forward(lib, p=0.3, seed=4, offset=k), *layer.backward(lib, p=0.3, seed=4, offset=k)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
    assert step.item() == 9


def test_offsets_past_32_bits(lib):
    """X, Y, dY and dX of more than 2^31 elements: the last tokens' results against the oracle, zeros before them."""
    n, rows, cols, r = 140000, 16448, 16384, 4
    layer = Layer(8, rows, cols, r, "mx", seed=11)
    tail, G8 = layer.Xd, layer.Gd
    layer.Xd = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
    layer.Xd[-8:] = tail
    Y = layer.forward(lib, out_dtype=torch.bfloat16)
    layer.check_forward(Y[-8:])
    assert not Y[:-8].any()
    del Y
    layer.Gd = torch.zeros(n, rows, dtype=torch.bfloat16, device="cuda")
    layer.Gd[-8:] = G8
    dX, dB, dA = layer.backward(lib)
    layer.check_backward((dX[-8:], dB, dA))
    assert not dX[:-8].any()


def test_lifecycle_over_mxfp4(lib):
    """The operators together, as they are used: LoftQ's alternation over MXFP4 (quantize W - B A, fit the adapter to
    the residual), a training step with dropout, and serving; each stage against the oracle on the same state."""
    g = np.random.default_rng(12)
    rows, cols, r, n = 160, 256, 16, 24
    W = dev((0.05 * g.standard_normal((rows, cols))).astype(np.float32))
    B = A = None
    errors = []
    for t in range(1, 4):
        packed, scales = lib.loftq_mxfp4_quantize(W, B, A)
        E = lib.loftq_mxfp4_dequantize(packed, scales, (rows, cols), W=W)
        B, A, _ = lib.loftq_lowrank_svd(E, r, t=t)
        errors.append(float(torch.linalg.norm(E - B @ A)))
    assert errors[-1] < errors[0]
    layer = Layer(n, rows, cols, r, "mx", seed=13)
    layer.kw = dict(packed=packed, scales=scales)
    layer.W = host(lib.loftq_mxfp4_dequantize(packed, scales, (rows, cols)))
    layer.Ad, layer.Bd, layer.A, layer.B = A, B, bf16(A.cpu().numpy()), bf16(B.cpu().numpy())
    rng = dict(p=0.1, seed=2, offset=0)
    layer.check_forward(layer.forward(lib, **rng), **rng)
    dX, dB, dA = layer.backward(lib, dx_dtype=torch.float32, **rng)
    layer.check_backward((dX, dB, dA), **rng)
    layer.Bd, layer.Ad = B - 1e-3 * dB, A - 1e-3 * dA
    layer.A, layer.B = bf16(layer.Ad.cpu().numpy()), bf16(layer.Bd.cpu().numpy())
    layer.check_forward(layer.forward(lib))
    x, layer.Xd, X, layer.X = layer.Xd, layer.Xd[:1].contiguous(), layer.X, layer.X[:1]
    layer.check_forward(layer.forward(lib))


def test_binding_checks_on_device(lib):
    layer = Layer(8, 64, 128, 8, seed=14)
    with pytest.raises(ValueError):
        layer.forward(lib, out=torch.empty(8, 65, device="cuda"))
    with pytest.raises(ValueError):
        layer.backward(lib, out=(None, torch.empty(64, 8, device="cuda"), torch.empty(8, 127, device="cuda")))
    with pytest.raises(TypeError):
        layer.forward(lib, out_dtype=torch.float16)
    with pytest.raises(lib.LoftqError):
        layer.forward(lib, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        lib.loftq_mxfp4_dequantize(torch.zeros(4, dtype=torch.uint8, device="cuda"),
                                   torch.zeros(8, dtype=torch.uint8, device="cuda"), (8, 64))
    strided = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")[:, ::2]
    layer.Xd = strided
    with pytest.raises(ValueError):
        layer.forward(lib)
