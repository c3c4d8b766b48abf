"""The operators (linear, gated, cross entropy) against their definitions in
64 bits, forward and backward, at the sizes and values where they can go
wrong.  Bounds: operator_reference.py."""
import math
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import operator_reference as ref  # noqa: E402
import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from software_pipelined_tiled_loop_gb300 import build
    build.build()
    pg.lib()
    assert pg.pgemm_get_device_status() == 0
    yield
    assert pg.pgemm_get_device_status() == 0


def rnd(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def nan_like(*shape, dtype=torch.bfloat16):
    """An output buffer that shows every element a kernel leaves unwritten."""
    return torch.full(shape, float("nan"), device="cuda", dtype=dtype)


# ---------------------------------------------------------------- linear ---
def linear_inputs(M, N, K, seed, bias=True, residual=True):
    return (rnd(seed, M, K), rnd(seed + 1, K, N, std=max(K, 1) ** -0.5),
            rnd(seed + 2, N) if bias else None, rnd(seed + 3, M, N) if residual else None)


# one element; a token; odd everything; whole tiles; tails of rows, columns and
# K; an empty K; rows whose pitch TMA cannot describe; a grid of CTA pairs; a
# long K over few tiles (parts along K)
LINEAR_SIZES = [(1, 1, 1), (1, 64, 64), (1, 1000, 520), (7, 33, 17), (16, 40, 2048), (24, 200, 1000), (33, 96, 72),
                (64, 512, 136), (65, 129, 200), (128, 128, 64), (129, 257, 130), (300, 520, 96),
                (5, 8, 0), (64, 4097, 40), (2500, 2600, 136), (96, 130, 4100), (200, 64, 8192),
                (1, 264, 9000)]


@pytest.mark.parametrize("i,size", list(enumerate(LINEAR_SIZES)))
@pytest.mark.parametrize("bias,residual", [(False, False), (True, True)])
def test_linear_forward(i, size, bias, residual):
    M, N, K = size
    X, W, b, R = linear_inputs(M, N, K, 100 + i, bias, residual)
    name = ACTS[i % len(ACTS)]
    Y, Z = nan_like(M, N), nan_like(M, N, dtype=torch.float32)
    pg.linear_bf16(M, N, K, X, W, b, name, R, Y, preact=Z)
    y, bound, z, ez = ref.linear(X, W, b, name, R)
    ref.check(Y, y, bound, "Y")
    ref.check(Z, z, ez + 1e-30, "preact")
    Y2 = nan_like(M, N)  # the same without keeping Z
    pg.linear_bf16(M, N, K, X, W, b, name, R, Y2)
    assert torch.equal(Y, Y2)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("M", [3, 130])
def test_linear_activations(name, M):
    X, W, b, _ = linear_inputs(M, 264, 96, 300)
    b = (b * 6).to(torch.bfloat16)  # arguments out to the flat parts
    Y = nan_like(M, 264)
    pg.linear_bf16(M, 264, 96, X, W, b, name, None, Y)
    y, bound, _, _ = ref.linear(X, W, b, name, None)
    ref.check(Y, y, bound, name)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("M,K", [(3, 96), (130, 96), (130, 0), (130, 1100)])
def test_activations_of_infinities_and_nan(name, M, K):
    # a column of each through the bias; its neighbours stay as they are
    X, W, b, _ = linear_inputs(M, 264, K, 310)
    special = {5: math.inf, 70: -math.inf, 263: math.nan}
    plain = nan_like(M, 264)
    pg.linear_bf16(M, 264, K, X, W, b, name, None, plain, preact=nan_like(
        M, 264, dtype=torch.float32))
    b = b.clone()
    for column, value in special.items():
        b[column] = value
    Y, Z = nan_like(M, 264), nan_like(M, 264, dtype=torch.float32)
    pg.linear_bf16(M, 264, K, X, W, b, name, None, Y, preact=Z)
    for column, value in special.items():
        want = ref.act(torch.full((M,), value, dtype=torch.float64, device="cuda"), name)
        assert torch.equal(Y[:, column].double().nan_to_num(7.0, 9.0, -9.0),
                           want.nan_to_num(7.0, 9.0, -9.0)), (name, value)
        plain[:, column] = Y[:, column] = 0
    assert torch.equal(Y, plain)


@pytest.mark.parametrize("M,N,K", [(3, 264, 96), (130, 264, 96), (130, 261, 96), (8, 128, 8192),
                                   (128, 128, 8192)])
def test_linear_residual_in_place(M, N, K):
    X, W, b, R = linear_inputs(M, N, K, 310)
    y, bound, _, _ = ref.linear(X, W, b, "silu", R)
    pg.linear_bf16(M, N, K, X, W, b, "silu", R, R)
    ref.check(R, y, bound, "Y")


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("i,size", list(enumerate(
    [(1, 1, 1), (1, 64, 72), (7, 33, 17), (129, 257, 130), (300, 520, 96), (777, 136, 520),
     (1500, 2600, 136), (64, 4096, 64), (4100, 128, 64)])))
def test_linear_backward(i, size, kept):
    M, N, K = size
    name = ACTS[(i + 3) % len(ACTS)]
    X, W, b, _ = linear_inputs(M, N, K, 400 + i)
    dY = rnd(450 + i, M, N, std=0.1)
    Z = None
    if kept:
        Z = nan_like(M, N, dtype=torch.float32)
        pg.linear_bf16(M, N, K, X, W, b, name, None, nan_like(M, N), preact=Z)
    dX, dW, db = nan_like(M, K), nan_like(K, N), nan_like(N)
    pg.linear_bf16_backward(M, N, K, X, W, b, name, dY, dX, dW, db, preact=Z)
    want = ref.linear_backward(X, W, b, name, dY)
    ref.check(dX, *want["dX"], "dX")
    ref.check(dW, *want["dW0"], "dW")
    ref.check(db, *want["db"], "dbias")


@pytest.mark.parametrize("name", ACTS)
def test_linear_backward_activations_and_absent_outputs(name):
    M, N, K = 70, 136, 96
    X, W, b, _ = linear_inputs(M, N, K, 500)
    dY = rnd(501, M, N)
    want = ref.linear_backward(X, W, b, name, dY)
    dX, dW, db = nan_like(M, K), nan_like(K, N), nan_like(N)
    pg.linear_bf16_backward(M, N, K, X, W, b, name, dY, dX, None, None)
    pg.linear_bf16_backward(M, N, K, X, W, b, name, dY, None, dW, None)
    pg.linear_bf16_backward(M, N, K, X, W, b, name, dY, None, None, db)
    ref.check(dX, *want["dX"], "dX")
    ref.check(dW, *want["dW0"], "dW")
    ref.check(db, *want["db"], "dbias")


# one CTA's tiles; pairs, and half-width units; parts along K
RELU_SIZES = [(150, 264, 1100), (2500, 1400, 1032), (260, 136, 4104)]


@pytest.mark.parametrize("M,N,K", RELU_SIZES)
def test_relu_pre_activations_are_summed_in_rounds(M, N, K):
    # rounds of 512 products, added with rounding: a chain of 32 steps and one
    # more for each round
    X, W, b, R = linear_inputs(M, N, K, 520)
    Y, Z = nan_like(M, N), nan_like(M, N, dtype=torch.float32)
    pg.linear_bf16(M, N, K, X, W, b, "relu", R, Y, preact=Z)
    y, bound, z, _ = ref.linear(X, W, b, "relu", R)
    ref.check(Y, y, bound, "Y")
    size = X.double().abs() @ W.double().abs() + b.double().abs()
    ref.check(Z, z, ref.step(512 + 16 * (K // 512 + 1)) * size, "preact")
    dY = rnd(521, M, N)
    want = ref.linear_backward(X, W, b, "relu", dY)
    for kept in (Z, None):
        dX, dW, db = nan_like(M, K), nan_like(K, N), nan_like(N)
        pg.linear_bf16_backward(M, N, K, X, W, b, "relu", dY, dX, dW, db, preact=kept)
        ref.check(dX, *want["dX"], "dX")
        ref.check(dW, *want["dW0"], "dW")
        ref.check(db, *want["db"], "dbias")


@pytest.mark.parametrize("M,F,K", RELU_SIZES)
def test_gated_relu_in_rounds(M, F, K):
    X, Wg, Wu = gated_inputs(M, F, K, 530)
    H, Z = nan_like(M, F), nan_like(2, M, F, dtype=torch.float32)
    pg.gated_bf16(M, F, K, X, Wg, Wu, "relu", H, preact=Z)
    h, bound, g, u, eg, eu, _, _ = ref.gated(X, Wg, Wu, "relu")
    ref.check(H, h, bound, "H")
    ref.check(Z[0], g, eg, "X Wg")
    ref.check(Z[1], u, eu, "X Wu")
    dH = rnd(531, M, F)
    want = ref.gated_backward(X, Wg, Wu, "relu", dH)
    for kept in (Z, None):
        dX, dWg, dWu = nan_like(M, K), nan_like(K, F), nan_like(K, F)
        pg.gated_bf16_backward(M, F, K, X, Wg, Wu, "relu", dH, dX, dWg, dWu, preact=kept)
        ref.check(dX, *want["dX"], "dX")
        ref.check(dWg, *want["dW0"], "dWg")
        ref.check(dWu, *want["dW1"], "dWu")


def test_linear_backward_of_nothing():
    dW, db, dX = nan_like(24, 40), nan_like(40), nan_like(5, 24)
    pg.linear_bf16_backward(0, 40, 24, None, rnd(1, 24, 40), None, "silu", None, None, dW, db)
    assert not dW.any() and not db.any()  # sums over no rows
    pg.linear_bf16_backward(5, 0, 24, rnd(2, 5, 24), None, None, "relu", None, dX, None, None)
    assert not dX.any()


# ----------------------------------------------------------------- gated ---
def gated_inputs(M, F, K, seed):
    return (rnd(seed, M, K), rnd(seed + 1, K, F, std=max(K, 1) ** -0.5),
            rnd(seed + 2, K, F, std=max(K, 1) ** -0.5))


GATED_SIZES = [(1, 1, 1), (1, 64, 64), (1, 1000, 520), (7, 33, 17), (16, 40, 2048), (24, 200, 1000), (33, 96, 72),
               (64, 512, 136), (65, 129, 200), (129, 257, 130), (300, 520, 96), (5, 8, 0),
               (2500, 1300, 136), (1, 136, 9000)]


@pytest.mark.parametrize("i,size", list(enumerate(GATED_SIZES)))
def test_gated_forward(i, size):
    M, F, K = size
    X, Wg, Wu = gated_inputs(M, F, K, 600 + i)
    name = ACTS[(i + 4) % len(ACTS)]
    H, Z = nan_like(M, F), nan_like(2, M, F, dtype=torch.float32)
    pg.gated_bf16(M, F, K, X, Wg, Wu, name, H, preact=Z)
    h, bound, g, u, eg, eu, _, _ = ref.gated(X, Wg, Wu, name)
    ref.check(H, h, bound, "H")
    ref.check(Z[0], g, eg + 1e-30, "X Wg")
    ref.check(Z[1], u, eu + 1e-30, "X Wu")
    H2 = nan_like(M, F)
    pg.gated_bf16(M, F, K, X, Wg, Wu, name, H2)
    assert torch.equal(H, H2)


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("i,size", list(enumerate(
    [(1, 1, 1), (1, 64, 72), (7, 33, 17), (129, 257, 130), (300, 520, 96), (777, 136, 520),
     (2500, 1300, 136), (64, 2048, 64)])))
def test_gated_backward(i, size, kept):
    M, F, K = size
    name = ACTS[(i + 1) % len(ACTS)]
    X, Wg, Wu = gated_inputs(M, F, K, 700 + i)
    dH = rnd(750 + i, M, F, std=0.1)
    Z = None
    if kept:
        Z = nan_like(2, M, F, dtype=torch.float32)
        pg.gated_bf16(M, F, K, X, Wg, Wu, name, nan_like(M, F), preact=Z)
    dX, dWg, dWu = nan_like(M, K), nan_like(K, F), nan_like(K, F)
    pg.gated_bf16_backward(M, F, K, X, Wg, Wu, name, dH, dX, dWg, dWu, preact=Z)
    want = ref.gated_backward(X, Wg, Wu, name, dH)
    ref.check(dX, *want["dX"], "dX")
    ref.check(dWg, *want["dW0"], "dWg")
    ref.check(dWu, *want["dW1"], "dWu")


def test_gated_backward_of_nothing():
    dWg, dWu, dX = nan_like(24, 40), nan_like(24, 40), nan_like(5, 24)
    pg.gated_bf16_backward(0, 40, 24, None, None, None, "silu", None, None, dWg, dWu)
    assert not dWg.any() and not dWu.any()
    pg.gated_bf16_backward(5, 0, 24, None, None, None, "silu", None, dX, None, None)
    assert not dX.any()


# ------------------------------------- few rows of weights at any pitch ---
# every alignment of a weight row, tiles that end in a row, short and long K
ODD_SIZES = [(1, 257, 64), (1, 1001, 700), (3, 130, 65), (16, 139, 200), (17, 517, 136),
             (33, 263, 1000), (64, 1294, 72), (65, 133, 520), (128, 407, 333), (100, 7, 4100),
             (128, 20003, 24)]


@pytest.mark.parametrize("i,size", list(enumerate(ODD_SIZES)))
def test_linear_few_rows_odd_pitch(i, size):
    M, N, K = size
    X, W, b, R = linear_inputs(M, N, K, 1400 + i)
    name = ACTS[i % len(ACTS)]
    Y = nan_like(M, N)
    pg.linear_bf16(M, N, K, X, W, b, name, R, Y)
    y, bound, _, _ = ref.linear(X, W, b, name, R)
    ref.check(Y, y, bound, "Y")
    dY = rnd(1450 + i, M, N)
    dX, dW, db = nan_like(M, K), nan_like(K, N), nan_like(N)
    pg.linear_bf16_backward(M, N, K, X, W, b, name, dY, dX, dW, db)
    want = ref.linear_backward(X, W, b, name, dY)
    for key, got in (("dX", dX), ("dW0", dW), ("db", db)):
        ref.check(got, *want[key], key)


@pytest.mark.parametrize("i,size", list(enumerate(ODD_SIZES)))
def test_gated_few_rows_odd_pitch(i, size):
    M, F, K = size
    X, Wg, Wu = gated_inputs(M, F, K, 1500 + i)
    name = ACTS[i % len(ACTS)]
    H = nan_like(M, F)
    pg.gated_bf16(M, F, K, X, Wg, Wu, name, H)
    h, bound = ref.gated(X, Wg, Wu, name)[:2]
    ref.check(H, h, bound, "H")
    dH = rnd(1550 + i, M, F)
    dX, dWg, dWu = nan_like(M, K), nan_like(K, F), nan_like(K, F)
    pg.gated_bf16_backward(M, F, K, X, Wg, Wu, name, dH, dX, dWg, dWu)
    want = ref.gated_backward(X, Wg, Wu, name, dH)
    for key, got in (("dX", dX), ("dW0", dWg), ("dW1", dWu)):
        ref.check(got, *want[key], key)


@pytest.mark.parametrize("N", [135, 136, 261])
def test_few_rows_keep_a_nan_in_its_column(N):
    # the first and last weights of rows lie beside their neighbours' in memory
    M, K = 5, 150
    X, W, _, _ = linear_inputs(M, N, K, 1600)
    dY = rnd(1601, M, N)
    Y, dX = nan_like(M, N), nan_like(M, K)
    pg.linear_bf16(M, N, K, X, W, None, "none", None, Y)
    pg.linear_bf16_backward(M, N, K, X, W, None, "none", dY, dX, None, None)
    bad = W.clone()
    bad[70, 0] = math.nan
    bad[149, N - 1] = math.inf
    Y2, dX2 = nan_like(M, N), nan_like(M, K)
    pg.linear_bf16(M, N, K, X, bad, None, "none", None, Y2)
    pg.linear_bf16_backward(M, N, K, X, bad, None, "none", dY, dX2, None, None)
    assert Y2[:, 0].isnan().all() and not Y2[:, N - 1].isfinite().any()
    assert dX2[:, 70].isnan().all() and not dX2[:, 149].isfinite().any()
    Y2[:, 0], Y2[:, N - 1], dX2[:, 70], dX2[:, 149] = Y[:, 0], Y[:, N - 1], dX[:, 70], dX[:, 149]
    assert torch.equal(Y, Y2) and torch.equal(dX, dX2)


# --------------------------- few tiles of many rows share their K in clusters ---
SHARED_SIZES = [(129, 520, 1100), (136, 40, 4100), (200, 1368, 2736), (300, 130, 1024),
                (257, 517, 1048), (513, 264, 1500), (777, 136, 3001), (1030, 130, 2050)]


@pytest.mark.parametrize("act", [0, 2])
@pytest.mark.parametrize("i,size", list(enumerate(SHARED_SIZES)))
def test_linear_few_tiles(i, size, act):
    M, N, K = size
    X, W, b, R = linear_inputs(M, N, K, 1700 + i)
    name = ACTS[(i + act) % len(ACTS)]
    Y, Z = nan_like(M, N), nan_like(M, N, dtype=torch.float32)
    pg.linear_bf16(M, N, K, X, W, b, name, R, Y, preact=Z)
    y, bound, z, ez = ref.linear(X, W, b, name, R)
    ref.check(Y, y, bound, "Y")
    ref.check(Z, z, ez + 1e-30, "preact")
    dY = rnd(1750 + i, M, N)
    want = ref.linear_backward(X, W, b, name, dY)
    for kept in (None, Z):
        dX, dW, db = nan_like(M, K), nan_like(K, N), nan_like(N)
        pg.linear_bf16_backward(M, N, K, X, W, b, name, dY, dX, dW, db, preact=kept)
        for key, got in (("dX", dX), ("dW0", dW), ("db", db)):
            ref.check(got, *want[key], key)
    # the reduction the other way round: M x K outputs from N columns
    X, W, b, _ = linear_inputs(M, K, N, 1780 + i)
    dY, dX = rnd(1790 + i, M, K), nan_like(M, N)
    pg.linear_bf16_backward(M, K, N, X, W, b, "silu", dY, dX, None, None)
    ref.check(dX, *ref.linear_backward(X, W, b, "silu", dY)["dX"], "dX of many columns")


@pytest.mark.parametrize("i,size", list(enumerate(SHARED_SIZES)))
def test_gated_few_tiles(i, size):
    M, F, K = size
    X, Wg, Wu = gated_inputs(M, F, K, 1800 + i)
    name = ACTS[(i + 2) % len(ACTS)]
    H, Z = nan_like(M, F), nan_like(2, M, F, dtype=torch.float32)
    pg.gated_bf16(M, F, K, X, Wg, Wu, name, H, preact=Z)
    h, bound, g, u, eg, eu, _, _ = ref.gated(X, Wg, Wu, name)
    ref.check(H, h, bound, "H")
    ref.check(Z[0], g, eg + 1e-30, "X Wg")
    ref.check(Z[1], u, eu + 1e-30, "X Wu")
    dH = rnd(1850 + i, M, F)
    want = ref.gated_backward(X, Wg, Wu, name, dH)
    for kept in (None, Z):
        dX, dWg, dWu = nan_like(M, K), nan_like(K, F), nan_like(K, F)
        pg.gated_bf16_backward(M, F, K, X, Wg, Wu, name, dH, dX, dWg, dWu, preact=kept)
        for key, got in (("dX", dX), ("dW0", dWg), ("dW1", dWu)):
            ref.check(got, *want[key], key)


# ----------------------------------------------------------------- xent ---
def xent_inputs(T, V, D, seed, padded=0.2):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y = torch.where(torch.rand((T,), generator=g, device="cuda") < padded, -100, y)
    return (rnd(seed + 1, T, D), rnd(seed + 2, V, D, std=2 * max(D, 1) ** -0.5), y,
            torch.rand((T,), generator=g, device="cuda"))


# one token of one; odd vocabularies; tails below and above a tile; pairs
XENT_SIZES = [(1, 1, 8), (1, 3, 1), (1, 1000, 64), (5, 129, 33), (33, 257, 40), (64, 4096, 64),
              (130, 1001, 72), (257, 515, 136), (3, 7, 0), (1100, 9000, 64), (2, 50257, 24),
              (65, 1001, 648), (1, 129, 1100), (40, 3000, 2500), (1100, 9001, 704),
              (200, 12001, 264)]


@pytest.mark.parametrize("i,size", list(enumerate(XENT_SIZES)))
def test_xent_forward(i, size):
    T, V, D = size
    X, W, y, _ = xent_inputs(T, V, D, 800 + i)
    loss, lse = nan_like(T, dtype=torch.float32), nan_like(T, dtype=torch.float32)
    pg.xent_bf16(T, V, D, X, W, y, loss, lse)
    want = ref.xent(X, W, y)
    ref.check(lse, *want["lse"], "lse")
    ref.check(loss, *want["loss"], "loss")
    alone = nan_like(T, dtype=torch.float32)
    pg.xent_bf16(T, V, D, X, W, y, alone, None)
    assert torch.equal(alone, loss)


# 0: the library's own workspace; 1: the smallest pieces of the vocabulary
@pytest.mark.parametrize("workspace", [0, 1])
@pytest.mark.parametrize("i,size", list(enumerate(XENT_SIZES)))
def test_xent_grad(i, size, workspace):
    T, V, D = size
    if workspace and V > 10000:
        V = 5001
    X, W, y, dl = xent_inputs(T, V, D, 900 + i)
    loss, lse = nan_like(T, dtype=torch.float32), nan_like(T, dtype=torch.float32)
    dX, dW = nan_like(T, D), nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, dl, loss, lse, dX, dW, workspace_bytes=workspace)
    want = ref.xent(X, W, y, dl)
    for name, got in (("lse", lse), ("loss", loss), ("dX", dX), ("dW", dW)):
        ref.check(got, *want[name], name)


# vocabularies a little beyond what one tile of every block of the few-token kernel covers
@pytest.mark.parametrize("i,size", list(enumerate([(1, 39001, 520), (20, 40003, 512),
                                                   (64, 20001, 776), (33, 60007, 520)])))
def test_xent_few_tokens_several_tiles(i, size):
    T, V, D = size
    X, W, y, dl = xent_inputs(T, V, D, 970 + i)
    y[0] = V - 1
    loss, lse = nan_like(T, dtype=torch.float32), nan_like(T, dtype=torch.float32)
    dX, dW = nan_like(T, D), nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, dl, loss, lse, dX, dW)
    want = ref.xent(X, W, y, dl)
    for name, got in (("lse", lse), ("loss", loss), ("dX", dX), ("dW", dW)):
        ref.check(got, *want[name], name)


@pytest.mark.parametrize("T", [3, 200, 700])
def test_xent_unlikely_tokens_beside_a_likely_one(T):
    # Token 0 takes all but exp(-20) of every row: the other rows of dW come from
    # probabilities of 2e-9 alone, which do not cancel: bf16's relative error twice (P's
    # rounding and the output's, 2^-8 each), 2^-11 of a kept exponential, and less than
    # 2^-12 from the logits' and sums' own errors.
    V, D = 96, 64
    X = torch.zeros(T, D, device="cuda", dtype=torch.bfloat16)
    X[:, 0] = 1
    X[:, 1:] = rnd(990, T, D - 1).abs()
    W = torch.zeros(V, D, device="cuda", dtype=torch.bfloat16)
    W[0, 0] = 20
    y = torch.zeros(T, device="cuda", dtype=torch.int64)
    dW = nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, None, None, None, None, dW)
    p = torch.softmax(X.double() @ W.double().t(), 1)
    want = p[:, 1:].t() @ X.double()
    assert ((dW[1:].double() - want).abs() <= (2.0 ** -7 + 2.0 ** -10) * want).all()


def test_xent_outputs_may_be_absent():
    T, V, D = 70, 1001, 72
    X, W, y, _ = xent_inputs(T, V, D, 1000)
    want = ref.xent(X, W, y, torch.ones(T, device="cuda"))
    dX, dW = nan_like(T, D), nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, None, None, None, dX, None)
    pg.xent_bf16_grad(T, V, D, X, W, y, None, None, None, None, dW)
    ref.check(dX, *want["dX"], "dX")
    ref.check(dW, *want["dW"], "dW")


def test_xent_rows_that_do_not_count():
    T, V, D = 200, 515, 64
    X, W, _, dl = xent_inputs(T, V, D, 1010)
    y = torch.full((T,), -100, device="cuda")
    y[::2] = V  # beyond the vocabulary: neither
    y[::3] = 2 ** 40
    loss = nan_like(T, dtype=torch.float32)
    dX, dW = nan_like(T, D), nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, dl, loss, None, dX, dW)
    assert not loss.any() and not dX.any() and not dW.any()


@pytest.mark.parametrize("scale", [30.0, -30.0])
def test_xent_large_logits(scale):
    # logits of some hundreds: exp alone would overflow (or vanish)
    T, V, D = 65, 1000, 64
    X, W, y, dl = xent_inputs(T, V, D, 1020, padded=0.0)
    X = (X.abs() * scale).to(torch.bfloat16)
    W = (W.abs() + 0.5).to(torch.bfloat16)
    loss, lse = nan_like(T, dtype=torch.float32), nan_like(T, dtype=torch.float32)
    dX, dW = nan_like(T, D), nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, dl, loss, lse, dX, dW)
    want = ref.xent(X, W, y, dl)
    for name, got in (("lse", lse), ("loss", loss), ("dX", dX), ("dW", dW)):
        ref.check(got, *want[name], name)


def test_xent_infinite_and_nan_logits():
    # a row of W is -inf where x > 0: its logits are -inf and its share zero;
    # a NaN in a row of X stays in that row
    T, V, D = 40, 300, 8
    X = rnd(1030, T, D).abs() + 0.1
    W = rnd(1031, V, D)
    W[7] = float("-inf")
    y = torch.arange(T, device="cuda") + 8
    lse = nan_like(T, dtype=torch.float32)
    loss = nan_like(T, dtype=torch.float32)
    pg.xent_bf16(T, V, D, X, W, y, loss, lse)
    logits = X.double() @ W.double().t()
    assert torch.allclose(lse.double(), torch.logsumexp(logits, 1), rtol=1e-5, atol=1e-5)
    X[3, 2] = float("nan")
    pg.xent_bf16(T, V, D, X, W, y, loss, lse)
    assert torch.isnan(lse[3]) and torch.isnan(loss[3])
    rest = torch.arange(T, device="cuda") != 3
    assert torch.isfinite(lse[rest]).all() and torch.isfinite(loss[rest]).all()


def test_xent_column_blocks_of_nothing_but_minus_infinity():
    # whole blocks of -inf logits beside a block of very negative ones
    T, V, D = 9, 1024, 8
    X = torch.ones(T, D, device="cuda", dtype=torch.bfloat16)
    W = torch.full((V, D), float("-inf"), device="cuda", dtype=torch.bfloat16)
    W[512:640] = -40.0
    y = torch.arange(T, device="cuda") + 512
    loss, lse = nan_like(T, dtype=torch.float32), nan_like(T, dtype=torch.float32)
    pg.xent_bf16(T, V, D, X, W, y, loss, lse)
    want = torch.full((T,), -320.0 + math.log(128), device="cuda")
    assert torch.allclose(lse, want, rtol=1e-6)
    assert torch.allclose(loss, torch.full_like(want, math.log(128)), rtol=1e-4)


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("weights", ["mean", "random", "signs", "wide"])
def test_xent_scale_of_the_loss(T, weights):
    # the products' operand is rounded after division by the largest weight of a
    # row that counts, so that a mean's common factor rounds nothing
    V, D = 1001, 72
    X, W, y, dl = xent_inputs(T, V, D, 1040)
    if weights == "mean":
        dl = torch.full((T,), 1.0 / 417, device="cuda")
    elif weights == "signs":
        dl = torch.where(dl > 0.5, dl, -dl)
    elif weights == "wide":
        dl = torch.pow(10.0, -30 * dl)
        dl[y < 0] = float("inf")  # a row that does not count may hold anything
    dX, dW = nan_like(T, D), nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, dl, None, None, dX, dW)
    want = ref.xent(X, W, y, torch.where(y < 0, torch.zeros_like(dl), dl))
    ref.check(dX, *want["dX"], "dX")
    ref.check(dW, *want["dW"], "dW")
    if weights == "mean":
        # -1 / 417 rounds to bf16 1.0e-3 off: unscaled, so would everything
        for got, key in ((dX, "dX"), (dW, "dW")):
            d, r = got.double(), want[key][0]
            assert abs((d * r).sum() / (r * r).sum() - 1) < 5e-4


def test_xent_no_tokens():
    dW = nan_like(40, 24)
    pg.xent_bf16_grad(0, 40, 24, None, rnd(1, 40, 24), None, None, None, None, None, dW)
    assert not dW.any()


# ------------------------------------------- gradients against differences ---
def directional(f, x, v, h):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_linear_gradient_against_differences(name):
    M, N, K = 40, 72, 48
    X, W, b, _ = linear_inputs(M, N, K, 1100)
    dY = rnd(1101, M, N)
    dX, dW, db = nan_like(M, K), nan_like(K, N), nan_like(N)
    pg.linear_bf16_backward(M, N, K, X, W, b, name, dY, dX, dW, db)
    bounds = ref.linear_backward(X, W, b, name, dY)
    Xd, Wd, bd, dYd = X.double(), W.double(), b.double(), dY.double()

    def f(x, w, c):
        return (ref.act(x @ w + c, name) * dYd).sum()

    for got, key, at in ((dX, "dX", 0), (dW, "dW0", 1), (db, "db", 2)):
        args = [Xd, Wd, bd]
        v = torch.randn(args[at].shape, device="cuda", dtype=torch.float64,
                        generator=torch.Generator(device="cuda").manual_seed(5))
        num = directional(lambda x: f(*args[:at], x, *args[at + 1:]), args[at], v, 1e-5)
        assert abs((got.double() * v).sum() - num) <= (bounds[key][1] * v.abs()).sum() + 1e-6 * abs(num)


@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_gated_gradient_against_differences(name):
    M, F, K = 40, 72, 48
    X, Wg, Wu = gated_inputs(M, F, K, 1110)
    dH = rnd(1111, M, F)
    dX, dWg, dWu = nan_like(M, K), nan_like(K, F), nan_like(K, F)
    pg.gated_bf16_backward(M, F, K, X, Wg, Wu, name, dH, dX, dWg, dWu)
    bounds = ref.gated_backward(X, Wg, Wu, name, dH)
    args = [X.double(), Wg.double(), Wu.double()]

    def f(x, wg, wu):
        return (ref.act(x @ wg, name) * (x @ wu) * dH.double()).sum()

    for got, key, at in ((dX, "dX", 0), (dWg, "dW0", 1), (dWu, "dW1", 2)):
        v = torch.randn(args[at].shape, device="cuda", dtype=torch.float64,
                        generator=torch.Generator(device="cuda").manual_seed(6))
        num = directional(lambda x: f(*args[:at], x, *args[at + 1:]), args[at], v, 1e-5)
        assert abs((got.double() * v).sum() - num) <= (bounds[key][1] * v.abs()).sum() + 1e-6 * abs(num)


def test_xent_gradient_against_differences():
    T, V, D = 50, 300, 40
    X, W, y, dl = xent_inputs(T, V, D, 1120)
    dX, dW = nan_like(T, D), nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, dl, None, None, dX, dW)
    bounds = ref.xent(X, W, y, dl)
    args = [X.double(), W.double()]

    def f(x, w):
        return (ref.xent(x, w, y)["loss"][0] * dl.double()).sum()

    for got, key, at in ((dX, "dX", 0), (dW, "dW", 1)):
        v = torch.randn(args[at].shape, device="cuda", dtype=torch.float64,
                        generator=torch.Generator(device="cuda").manual_seed(7))
        num = directional(lambda x: f(*args[:at], x, *args[at + 1:]), args[at], v, 1e-5)
        assert abs((got.double() * v).sum() - num) <= (bounds[key][1] * v.abs()).sum() + 1e-6 * abs(num)


# ------------------------------------------------ streams, graphs, repeats ---
def all_operators(stream=None):
    """Every operator once on fixed inputs; what they wrote."""
    M, N, K = 200, 264, 2056
    X, W, b, R = linear_inputs(M, N, K, 1200)
    out = []

    def new(*shape, dtype=torch.bfloat16):
        out.append(torch.zeros(shape, device="cuda", dtype=dtype))
        return out[-1]

    ins = (X, W, b, R, rnd(1204, M, N), *gated_inputs(M, N, K, 1205)[1:], rnd(1209, M, N),
           *xent_inputs(M, 3001, K, 1210))
    bufs = [new(M, N), new(M, K), new(K, N), new(N), new(M, N), new(M, K), new(K, N), new(K, N),
            new(M, dtype=torch.float32), new(M, K), new(3001, K), new(3, N)]

    def call():
        X, W, b, R, dY, Wg, Wu, dH, Xx, Wx, y, dl = ins
        pg.linear_bf16(M, N, K, X, W, b, "gelu", R, bufs[0], stream=stream)
        pg.linear_bf16_backward(M, N, K, X, W, b, "gelu", dY, *bufs[1:4], stream=stream)
        pg.gated_bf16(M, N, K, X, Wg, Wu, "silu", bufs[4], stream=stream)
        pg.gated_bf16_backward(M, N, K, X, Wg, Wu, "silu", dH, *bufs[5:8], stream=stream)
        pg.xent_bf16_grad(M, 3001, K, Xx, Wx, y, dl, bufs[8], None, *bufs[9:11],
                          workspace_bytes=1 << 20, stream=stream)
        pg.linear_bf16(3, N, K, X[:3], W, b, "gelu", R[:3], bufs[11], stream=stream)
    return call, bufs


def test_results_do_not_depend_on_timing_or_stream():
    call, bufs = all_operators()
    call()
    torch.cuda.synchronize()
    first = [t.clone() for t in bufs]
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, bufs))
    side = torch.cuda.Stream()
    call2, bufs2 = all_operators(stream=side)
    torch.cuda.synchronize()
    call2()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, bufs2))


def test_operators_from_several_threads():
    call, bufs = all_operators()
    call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    jobs = [all_operators(stream=st) for st in streams]
    torch.cuda.synchronize()
    errors = []

    def work(k):
        try:
            for _ in range(5):
                jobs[k][0]()
            streams[k].synchronize()
        except Exception as e:  # reported by the main thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for _, got in jobs:
        assert all(torch.equal(a, b) for a, b in zip(bufs, got))


def test_operators_in_a_captured_graph():
    call, bufs = all_operators()
    call()
    torch.cuda.synchronize()
    first = [t.clone() for t in bufs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in bufs:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, bufs))


def test_untouched_memory_around_outputs():
    # outputs as slices of larger buffers: not a byte beyond them is written
    M, N, K = 130, 261, 72
    X, W, b, _ = linear_inputs(M, N, K, 1300)
    pad = 64
    buf = torch.full((M * N + 2 * pad,), 7.0, device="cuda", dtype=torch.bfloat16)
    Y = buf[pad:pad + M * N].view(M, N)
    pg.linear_bf16(M, N, K, X, W, b, "none", None, Y)
    torch.cuda.synchronize()
    assert (buf[:pad] == 7).all() and (buf[pad + M * N:] == 7).all()
    y, bound, _, _ = ref.linear(X, W, b, "none", None)
    ref.check(Y, y, bound, "Y")
