"""The tiled product of the training and serving calls in each of its tile shapes, and the few-token product with each
number of feature tiles, against the oracle in fp64 (bars as in test_gpu_layer.py).  Which tile runs is the planner's
choice: each case names the tile that it is there for and reads from the launch timing that it ran."""
import pytest
import torch

from test_gpu_layer import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture
def ran(lib):
    """f(call) -> (result, the names of the kernels that it launched)."""
    def f(call):
        lib.profile_collect()
        lib.profile_enable(True)
        try:
            out = call()
            torch.cuda.synchronize()
        finally:
            lib.profile_enable(False)
        return out, set(lib.profile_collect())
    return f


# base, tokens, features, K, r, tile.  The ring holds two steps or three (128 x 256): one step, fewer than the ring, the
# ring and more, of 64 columns (NormalFloat) or 256 (MXFP4).  Tokens and features end inside a tile.
WIDE = [("nf", 777, 14001, 64, 16, "256x256"), ("nf", 777, 14001, 320, 64, "256x256"),
        ("nf", 520, 14001, 64, 16, "192x256"), ("nf", 520, 14001, 128, 0, "192x256"), ("nf", 520, 14001, 320, 64, "192x256"),
        ("nf", 1000, 4099, 64, 16, "128x256"), ("nf", 1000, 4099, 128, 0, "128x256"), ("nf", 1000, 4099, 192, 33, "128x256"),
        ("nf", 1000, 4099, 320, 64, "128x256"),
        ("mx", 777, 14001, 96, 16, "256x256"), ("mx", 777, 14001, 544, 64, "256x256"),
        ("mx", 520, 14001, 256, 16, "192x256"), ("mx", 520, 14001, 544, 64, "192x256"),
        ("mx", 1000, 4099, 32, 16, "128x256"), ("mx", 1000, 4099, 512, 0, "128x256"), ("mx", 1000, 4099, 1056, 64, "128x256")]
# the product divided into K ranges
DEEP = [("nf", 1000, 4159, 6400, 16, "256x256"), ("nf", 200, 4161, 6400, 16, "128x256"),
        ("nf", 520, 4160, 16384, 16, "192x256"), ("nf", 520, 1100, 2048, 16, "64x128"),
        ("mx", 1000, 4160, 16384, 16, "256x256"), ("mx", 520, 4160, 25600, 16, "192x256"), ("mx", 1000, 2111, 12288, 16, "128x256"), ("mx", 520, 1100, 4096, 16, "64x128")]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(map(str, c)))
def test_forward_in_each_tile(lib, ran, case, dtype):
    base, n, rows, cols, r, tile = case
    layer = Layer(n, rows, cols, r, base, dq=base == "nf", seed=n + cols)
    rng = dict(p=0.2, seed=5, offset=3)
    Y, names = ran(lambda: layer.forward(lib, out_dtype=dtype, **rng))
    assert f"{'mx' if base == 'mx' else 'bf16'}_product_{tile}" in names and "join_product" not in names
    layer.check_forward(Y, **rng)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", [c[:2] + (-(-c[2] // 32) * 32 if c[0] == "mx" else -(-c[2] // 64) * 64,) + c[3:] for c in WIDE]
                         + [("nf", 1000, 4160, 100, 16, "128x256"), ("mx", 777, 14016, 130, 16, "256x256")],
                         ids=lambda c: "-".join(map(str, c)))
def test_gradient_in_each_tile(lib, ran, case, dtype):
    """dX's features are the layer's columns, its K the layer's rows (the mask is applied in the accumulators)."""
    base, n, cols, rows, r, tile = case
    layer = Layer(n, rows, cols, r, base, seed=n + cols)
    rng = dict(p=0.2, seed=6, offset=4)
    grads, names = ran(lambda: layer.backward(lib, dx_dtype=dtype, **rng))
    assert f"bf16_product_{tile}" in names and "join_product" not in names
    layer.check_backward(grads, **rng)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", DEEP, ids=lambda c: "-".join(map(str, c)))
def test_ranges_of_k_in_each_tile(lib, ran, case, dtype):
    base, n, rows, cols, r, tile = case
    layer = Layer(n, rows, cols, r, base, seed=n + cols)
    rng = dict(p=0.2, seed=7, offset=5)
    Y, names = ran(lambda: layer.forward(lib, out_dtype=dtype, **rng))
    assert f"{'mx' if base == 'mx' else 'bf16'}_product_{tile}" in names and "join_product" in names
    layer.check_forward(Y, **rng)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("r", [0, 3, 64])
@pytest.mark.parametrize("n", [1, 8, 16])
@pytest.mark.parametrize("rows", [8192 + 5, 16384 + 37])
def test_few_tokens_with_two_and_four_feature_tiles(lib, ran, rows, n, r, dtype):
    layer = Layer(n, rows, 288, r, "mx", seed=rows + n)
    Y, names = ran(lambda: layer.forward(lib, out_dtype=dtype))
    assert "mx_token_product" in names
    layer.check_forward(Y)


@pytest.mark.parametrize("rows,cols,r,n,few", [
    (4096, 4096, 64, 16, True), (8192, 4096, 64, 16, True), (4096, 4096, 16, 17, False), (11008, 4096, 16, 8, True),
    (11008, 4096, 16, 9, False), (11008, 4096, 64, 8, False), (16384, 8192, 16, 8, True), (16384, 8192, 64, 2, True),
    (22016, 4096, 64, 8, False), (11008, 11008, 0, 1, False), (11008, 11008, 64, 8, False), (28672, 8192, 16, 2, False),
    (1024, 11008, 16, 8, True), (64, 11008, 64, 1, False), (1024, 16384, 64, 8, False), (128, 65536, 0, 1, False)])
def test_which_product_takes_few_tokens(lib, ran, rows, cols, r, n, few):
    """The faster of the two, as measured at these sizes."""
    steps = -(-cols // 256)
    base = dict(packed=torch.zeros(rows, steps * 128, dtype=torch.uint8, device="cuda"),
                scales=torch.zeros(steps, rows, 8, dtype=torch.uint8, device="cuda"))
    ad = dict(B=torch.zeros(rows, r, device="cuda"), A=torch.zeros(r, cols, device="cuda")) if r else {}
    X = torch.ones(n, cols, dtype=torch.bfloat16, device="cuda")
    Y, names = ran(lambda: lib.loftq_mxfp4_forward(X, shape=(rows, cols), **base, **ad))
    assert ("mx_token_product" in names) == few and not Y.any()
