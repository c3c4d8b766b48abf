"""Operators at the edges of their contracts: absent operands, ReLU sums of few
rows, losses near zero, infinite logits, far tails of activations, the scratch
that small workspaces take, memory around outputs.  Bounds: operator_reference.py,
unless a test derives its own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import operator_reference as ref  # noqa: E402
import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402


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
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def nan_like(*shape, dtype=torch.bfloat16):
    """An output buffer that shows every element a kernel leaves unwritten."""
    return torch.full(shape, float("nan"), device="cuda", dtype=dtype)


# --------------------------------------------------------- absent operands ---
@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("N", [261, 264])
@pytest.mark.parametrize("name", ["none", "silu"])
def test_linear_weight_gradients_without_weights(M, N, name):
    # dW and db need W only to compute Z again
    K = 72
    X, W, b, dY = rnd(1, M, K), rnd(2, K, N, std=K ** -0.5), rnd(3, N), rnd(4, M, N)
    Z = None
    if name != "none":
        Z = nan_like(M, N, dtype=torch.float32)
        pg.linear_bf16(M, N, K, X, W, b, name, None, nan_like(M, N), preact=Z)
    want = ref.linear_backward(X, W, b, name, dY)
    dW, db, db2 = nan_like(K, N), nan_like(N), nan_like(N)
    pg.linear_bf16_backward(M, N, K, X, None, None, name, dY, None, dW, db, preact=Z)
    pg.linear_bf16_backward(M, N, K, None, None, None, name, dY, None, None, db2, preact=Z)
    ref.check(dW, *want["dW0"], "dW")
    ref.check(db, *want["db"], "db")
    assert torch.equal(db, db2)


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("F,K", [(261, 72), (264, 77)])
def test_gated_gradients_without_what_they_do_not_read(M, F, K):
    X, Wg, Wu, dH = (rnd(11, M, K), rnd(12, K, F, std=K ** -0.5), rnd(13, K, F, std=K ** -0.5),
                     rnd(14, M, F))
    Z = nan_like(2, M, F, dtype=torch.float32)
    pg.gated_bf16(M, F, K, X, Wg, Wu, "silu", nan_like(M, F), preact=Z)
    want = ref.gated_backward(X, Wg, Wu, "silu", dH)
    dX, dWg, dWu = nan_like(M, K), nan_like(K, F), nan_like(K, F)
    pg.gated_bf16_backward(M, F, K, None, Wg, Wu, "silu", dH, dX, None, None, preact=Z)
    pg.gated_bf16_backward(M, F, K, X, None, None, "silu", dH, None, dWg, dWu, preact=Z)
    for key, got in (("dX", dX), ("dW0", dWg), ("dW1", dWu)):
        ref.check(got, *want[key], key)


# ------------------------------------------------------- cross entropy's scratch ---
def scratch_of(call):
    """Bytes that the library's pool holds after a call that found it empty."""
    torch.cuda.synchronize()
    pg.pgemm_trim_scratch()
    before = torch.cuda.mem_get_info()[0]
    call()
    torch.cuda.synchronize()
    return before - torch.cuda.mem_get_info()[0]


def test_xent_small_workspace_takes_little_scratch():
    # 256 pieces of the vocabulary: the statistics' 4 MB, P of one piece, a running sum
    # of dX and one piece's (8 MB each), dW's parts (4 MB at most); the pool grows by
    # blocks of some 32 MB.  A sum kept for every piece would be 2 GB.
    T, V, D = 1024, 65536, 2048
    X, W, dl = rnd(21, T, D), rnd(22, V, D, std=2 * D ** -0.5), torch.rand(T, device="cuda")
    y = torch.randint(0, V, (T,), device="cuda")
    dX, dW = nan_like(T, D), nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, dl, None, None, dX, dW)  # (code and tables loaded)
    took = {ws: scratch_of(lambda: pg.xent_bf16_grad(T, V, D, X, W, y, dl, None, None, dX, dW,
                                                     workspace_bytes=ws)) for ws in (0, 1)}
    assert took[1] < 128 << 20 and took[1] < took[0], took
    want = ref.xent(X, W, y, dl)
    ref.check(dX, *want["dX"], "dX")
    ref.check(dW, *want["dW"], "dW")


@pytest.mark.parametrize("workspace", [1 << 20, 3 << 20, 16 << 20])
def test_xent_sums_of_dx_taken_in_now_and_then(workspace):
    # room for 2, 6 and 32 partial sums of dX (512 KB each) beside 16, 5 and 1 pieces
    T, V, D = 256, 30001, 512
    X, W, dl = rnd(23, T, D), rnd(24, V, D, std=2 * D ** -0.5), torch.rand(T, device="cuda")
    y = torch.randint(0, V, (T,), device="cuda")
    dX, dW = nan_like(T, D), nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, dl, None, None, dX, dW, workspace_bytes=workspace)
    want = ref.xent(X, W, y, dl)
    ref.check(dX, *want["dX"], "dX")
    ref.check(dW, *want["dW"], "dW")


# ------------------------------------------------- ReLU sums of few rows ---
# A Z that decides a ReLU's derivative is summed in rounds of 512 products at any number
# of rows.  With all products positive every truncation falls short: half an ulp, at
# most 2^-24 of the running sum, on average over many outputs, 32 times a round, while
# the running sum grows evenly to the round's own: (32 + 1) / 2 * 2^-24 of it, and the
# rounds' additions round to nearest either way.  A tenth more for the sampling.  Chains
# of a block's whole share (K = 8192 of one block) fall 16 times as short.
RELU_MEAN = 1.1 * 16.5 * 2.0 ** -24
FEW_RELU = [(1, 20000, 8192), (17, 264, 8192), (64, 20000, 8192), (128, 264, 9001),
            (128, 39000, 4104), (3, 20001, 8192), (100, 20003, 4100)]


def positive(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(shape, generator=g, device="cuda") + 0.25).to(torch.bfloat16)


@pytest.mark.parametrize("M,N,K", FEW_RELU)
def test_few_rows_sum_relu_pre_activations_in_rounds(M, N, K):
    X, W = positive(31, M, K), positive(32, K, N)
    Y, Z = nan_like(M, N), nan_like(M, N, dtype=torch.float32)
    pg.linear_bf16(M, N, K, X, W, None, "relu", None, Y, preact=Z)
    z = X.double() @ W.double()
    assert ((Z.double() - z) / z).mean().abs().item() < RELU_MEAN
    G = nan_like(2, M, N, dtype=torch.float32)
    H = nan_like(M, N)
    pg.gated_bf16(M, N, K, X, W, W, "relu", H, preact=G)
    for g in G:
        assert ((g.double() - z) / z).mean().abs().item() < RELU_MEAN


@pytest.mark.parametrize("M,N,K", FEW_RELU)
def test_few_rows_compute_relu_pre_activations_alike(M, N, K):
    # what a backward pass computes again has the signs of what a forward pass kept
    X, W, b, dY = rnd(33, M, K), rnd(34, K, N, std=K ** -0.5), rnd(35, N), rnd(36, M, N)
    Y, Z = nan_like(M, N), nan_like(M, N, dtype=torch.float32)
    pg.linear_bf16(M, N, K, X, W, b, "relu", None, Y, preact=Z)
    y, bound, z, _ = ref.linear(X, W, b, "relu", None)
    ref.check(Y, y, bound, "Y")
    size = X.double().abs() @ W.double().abs() + b.double().abs()
    # the longest chain, an addition a round, and one a block of a shared tile
    ref.check(Z, z, ref.step(512 + 16 * (K // 512 + 9)) * size, "preact")
    del size, z, y, bound
    got = []
    for kept in (Z, None):
        dX, db = nan_like(M, K), nan_like(N)
        pg.linear_bf16_backward(M, N, K, X, W, b, "relu", dY, dX, None, db, preact=kept)
        got.append((dX, db))
    want = ref.linear_backward(X, W, b, "relu", dY)
    for dX, db in got:
        ref.check(dX, *want["dX"], "dX")
        ref.check(db, *want["db"], "db")
    if N % 8 == 0:
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


# ----------------------------------------------------------- losses near zero ---
@pytest.mark.parametrize("T", [1, 40, 300, 1300])
def test_xent_losses_of_certain_tokens_are_not_negative(T):
    # Logits of 24 at the targets beside others of at most some 4: losses of 1e-7, where
    # lse and the target's logit are off by up to the bound's 1e-5 each.
    V, D = 1001, 1024
    W = rnd(41, V, D)
    y = torch.randint(0, V, (T,), device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(42))
    X = (W[y].float() * (24.0 / D)).to(torch.bfloat16)
    want = ref.xent(X, W, y)["loss"]
    alone = nan_like(T, dtype=torch.float32)
    pg.xent_bf16(T, V, D, X, W, y, alone, None)
    loss, dX, dW = nan_like(T, dtype=torch.float32), nan_like(T, D), nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, None, loss, None, dX, dW)
    pieces = nan_like(T, dtype=torch.float32)
    pg.xent_bf16_grad(T, V, D, X, W, y, None, pieces, None, dX, dW, workspace_bytes=1)
    for got in (alone, loss, pieces):
        ref.check(got, *want, "loss")
        assert (got >= 0).all(), got.min().item()


# ------------------------------------------------------------ infinite logits ---
@pytest.mark.parametrize("T", [9, 100, 1300])
@pytest.mark.parametrize("workspace", [0, 1])
def test_xent_of_infinite_logits(T, workspace):
    # token 7's logits are +inf in every other row (a +inf weight times a positive or a
    # zero input would be NaN: those rows hold -1, whose product is -inf); row 3 holds a
    # NaN beside them
    V, D = 700, 40
    X, W = rnd(51, T, D), rnd(52, V, D, std=D ** -0.5)
    X[:, 5] = 1
    X[1::2, 5] = -1
    W[7, 5] = float("inf")
    y = torch.arange(T, device="cuda") % 300 + 8
    y[4] = 7  # the infinite one itself
    X[3, 2] = float("nan")
    rows = torch.arange(T, device="cuda")
    up = (rows % 2 == 0)
    fine = ~up & (rows != 3)
    loss, lse = nan_like(T, dtype=torch.float32), nan_like(T, dtype=torch.float32)
    pg.xent_bf16(T, V, D, X, W, y, loss, lse)
    loss2, lse2 = nan_like(T, dtype=torch.float32), nan_like(T, dtype=torch.float32)
    dX, dW = torch.zeros_like(X), torch.zeros_like(W)
    pg.xent_bf16_grad(T, V, D, X, W, y, None, loss2, lse2, dX, dW, workspace_bytes=workspace)
    # W without that token, for what is finite
    rest = torch.arange(V, device="cuda") != 7
    want = ref.xent(X[fine], W[rest], torch.where(y[fine] > 7, y[fine] - 1, y[fine]))
    for got, total in ((loss, lse), (loss2, lse2)):
        assert (total[up] == float("inf")).all() and total[3].isnan() and got[3].isnan()
        assert (got[up & (rows != 4)] == float("inf")).all() and got[4].isnan()
        ref.check(total[fine], *want["lse"], "lse")
        ref.check(got[fine], *want["loss"], "loss")
    # an infinite sum leaves the finite tokens nothing: their own rows take P = -1 at the
    # target alone, and only token 7's P is no number
    dW1 = torch.zeros_like(W)
    only = torch.where(up, y, -100)
    pg.xent_bf16_grad(T, V, D, X, W, only, None, None, None, None, dW1, workspace_bytes=workspace)
    p = torch.zeros(T, V, device="cuda", dtype=torch.float64)
    p[rows[up], y[up]] = -1.0
    finite = torch.where(X.isnan(), torch.zeros_like(X), X).double()
    # (row 3 does not count here, but its zeros meet the NaN of X: leave its column out)
    cols = torch.arange(D, device="cuda") != 2
    exact = (p.t() @ finite)[:, cols]
    keep = rest
    got = dW1[:, cols][keep].double()
    assert ((got - exact[keep]).abs() <= 2.0 ** -8 * exact[keep].abs()
            + ref.step(T) * (p.abs().t() @ finite.abs())[:, cols][keep]).all()
    assert dW1[7].isnan().all()


# -------------------------------------------------------- far tails of activations ---
def tails():
    """Every bf16 from 2^-6 to 13 and its negative, as one row."""
    z = torch.arange(0x3C80, 0x4150, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    return torch.cat([z, -z])


@pytest.mark.parametrize("M", [1, 200])
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_activations_are_right_relatively(M, name):
    # Z is one exact product.  The value: 2^-8 of itself by rounding to bf16 and 2^-13
    # for everything before, which bounds the documented 4.4e-5 of the tail with the
    # exponential's and the reciprocal's own errors (an argument of 2^7 carries 2^-18).
    # gelu_tanh's tail: its argument 0.8 (z + 0.045 z^3) is as large as 2^7.2 at -13, where
    # the 64-bit form needs its own way to the tail, z / (1 + exp(2 y)).
    z = tails()
    N = z.numel()
    X = torch.ones(M, 1, device="cuda", dtype=torch.bfloat16)
    Y, H = nan_like(M, N), nan_like(M, N)
    pg.linear_bf16(M, N, 1, X, z.view(1, N), None, name, None, Y)
    pg.gated_bf16(M, N, 1, X, z.view(1, N), torch.ones_like(z).view(1, N), name, H)
    zd = z.double()
    if name == "gelu_tanh":
        y = zd / (1 + torch.exp(2 * (2 / torch.pi) ** 0.5 * -(zd + 0.044715 * zd ** 3)))
    else:
        y = ref.act(zd, name)
    seen = y.abs() >= 2.0 ** -110  # (smaller ones may be flushed on the way)
    assert seen.sum() > 0.7 * N
    for got in (Y, H):
        over = (got.double() - y).abs() - (2.0 ** -8 + 2.0 ** -13) * y.abs()
        assert (over[:, seen] <= 0).all(), z[seen][over[:, seen].amax(0).argmax()].item()
        assert (got[:, ~seen].abs().double() <= 2.0 ** -100).all()


@pytest.mark.parametrize("kept", [False, True])
def test_gelu_gradient_of_the_tail(kept):
    # dbias of one row is gelu'(z) = Phi + z phi, whose terms differ in sign below zero:
    # 2^-13 of each, and two roundings to bf16
    z = tails()
    N = z.numel()
    X, ones = torch.ones(1, 1, device="cuda", dtype=torch.bfloat16), torch.ones_like(z).view(1, N)
    Z = z.float().view(1, N).contiguous() if kept else None
    db = nan_like(N)
    pg.linear_bf16_backward(1, N, 1, X, z.view(1, N), None, "gelu", ones, None, None, db, preact=Z)
    zd = z.double()
    phi = torch.exp(-zd * zd / 2) / (2 * torch.pi) ** 0.5
    Phi = 0.5 * torch.erfc(-zd / 2 ** 0.5)
    d = Phi + zd * phi
    bound = 2.0 ** -7 * (1 + 2.0 ** -8) * d.abs() + 2.0 ** -13 * (Phi + zd.abs() * phi) + 2.0 ** -110
    assert ((db.double() - d).abs() <= bound).all()


# ----------------------------------------------- P of pieces and the sums it divides by ---
@pytest.mark.parametrize("T", [40, 100, 1100])
@pytest.mark.parametrize("workspace", [0, 1])
def test_xent_probabilities_share_the_sums_of_their_statistics(T, workspace):
    # All products are positive, logits about 24 with a deviation of 0.2: a sum that the
    # tensor core truncates 512 times ends some 512 / 2 * 2^-24 * 24 = 3.7e-4 short, and a
    # probability taken from it against a log-sum-exp of shorter rounds as much of itself.
    # With the same rounds both shorten alike.  Rows of dW of tokens that are no target
    # are then off by roundings to nearest alone, which average out over 1e5 and more
    # probabilities (2^-9 / 300 = 6e-6), by lse's own in fp32 (2e-6, twice) and by 2^-11 of
    # kept exponentials, rounded to nearest too.
    V, D = 2500, 8192
    X = (positive(61, T, D).float() * (24 / (0.5625 * D))).to(torch.bfloat16)
    W = positive(62, V, D)
    y = torch.zeros(T, device="cuda", dtype=torch.int64)
    dW = nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, None, None, None, None, dW, workspace_bytes=workspace)
    p = torch.softmax(X.double() @ W.double().t(), 1)
    want = p[:, 1:].t() @ X.double()
    off = ((dW[1:].double() - want) / want).mean().item()
    assert abs(off) < 3e-5, off


@pytest.mark.parametrize("T", [100, 1100])
def test_xent_of_logits_in_the_millions_stays_finite(T):
    # a logit's own rounding is some units here, so that nothing but the order of
    # magnitude of a probability is left: at most e^16 of lse's rounding at 2^27
    V, D = 600, 8
    X = torch.zeros(T, D, device="cuda", dtype=torch.bfloat16)
    X[:, 0] = positive(71, T) * 2.0 ** 13
    W = torch.zeros(V, D, device="cuda", dtype=torch.bfloat16)
    W[:, 0] = 2.0 ** 13
    W[:, 1:] = rnd(72, V, D - 1)
    y = torch.randint(0, V, (T,), device="cuda")
    loss, lse = nan_like(T, dtype=torch.float32), nan_like(T, dtype=torch.float32)
    dX, dW = nan_like(T, D), nan_like(V, D)
    for sign in (1, -1):
        pg.xent_bf16_grad(T, V, D, sign * X, W, y, None, loss, lse, dX, dW)
        want = torch.logsumexp(sign * X.double() @ W.double().t(), 1)
        assert ((lse.double() - want).abs() <= 2.0 ** -22 * want.abs()).all()
        assert all(t.isfinite().all() for t in (loss, dX, dW))


@pytest.mark.parametrize("T", [9, 100, 1100])
@pytest.mark.parametrize("workspace", [0, 1])
def test_xent_gradient_beside_blocks_of_minus_infinity(T, workspace):
    # whole column blocks of -inf logits, whose tokens have no probability (dX is left
    # out: it would multiply their zeros by their infinite weights)
    V, D = 1024, 8
    X = torch.ones(T, D, device="cuda", dtype=torch.bfloat16)
    W = torch.full((V, D), float("-inf"), device="cuda", dtype=torch.bfloat16)
    W[512:640] = -40.0
    y = torch.arange(T, device="cuda") % 128 + 512
    loss, lse, dW = nan_like(T, dtype=torch.float32), nan_like(T, dtype=torch.float32), nan_like(V, D)
    pg.xent_bf16_grad(T, V, D, X, W, y, None, loss, lse, None, dW, workspace_bytes=workspace)
    log = torch.log(torch.tensor(128.0, dtype=torch.float64)).item()
    assert ((lse.double() - (log - 320)).abs() <= 2.0 ** -22 * 320).all()
    assert ((loss.double() - log).abs() <= 2.0 ** -21 * 320).all()
    p = torch.full((T, V), 0.0, device="cuda", dtype=torch.float64)
    p[:, 512:640] = 1 / 128
    p[torch.arange(T, device="cuda"), y] -= 1.0
    want = p.t() @ X.double()
    # P: two roundings to 2^-8 and what 2^-21 of 320 and 2^-11 make of an exponential
    bound = (2.0 ** -8 * 2 + 2.0 ** -10) * (p.abs().t() @ X.double()) + 2.0 ** -8 * want.abs()
    assert ((dW.double() - want).abs() <= bound).all()
