"""Operators whose outputs or scratch pass 2^31 elements: rows at the top, middle
and bottom (and gradients that sum over all rows) against 64 bits."""
import math

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
    yield
    assert pg.pgemm_get_device_status() == 0
    torch.cuda.empty_cache()
    pg.pgemm_trim_scratch()


def rnd(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    for part in out.view(-1).split(1 << 28):  # few fp32 temporaries
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * std)
    return out


def some_rows(M):
    return [*range(0, 40), *range(M // 2, M // 2 + 40), *range(M - 40, M)]


@pytest.mark.parametrize("N", [33024, 33001])  # TMA stores; plain stores
def test_linear_output_past_31_bits(N):
    M, K = 66000, 64
    X, W, b, R = rnd(1, M, K), rnd(2, K, N, std=0.125), rnd(3, N), rnd(4, M, N)
    rows = some_rows(M)
    y, bound, _, _ = ref.linear(X[rows], W, b, "silu", R[rows])
    pg.linear_bf16(M, N, K, X, W, b, "silu", R, R)
    ref.check(R[rows], y, bound, "Y")


def test_gated_pre_activations_past_31_bits():
    M, F, K = 40000, 33024, 64  # 2 M F > 2^31
    X, Wg, Wu = rnd(5, M, K), rnd(6, K, F, std=0.125), rnd(7, K, F, std=0.125)
    H = torch.empty(M, F, device="cuda", dtype=torch.bfloat16)
    Z = torch.empty(2, M, F, device="cuda")
    pg.gated_bf16(M, F, K, X, Wg, Wu, "silu", H, preact=Z)
    rows = some_rows(M)
    h, bound, g, u, eg, eu, _, _ = ref.gated(X[rows], Wg, Wu, "silu")
    ref.check(H[rows], h, bound, "H")
    ref.check(Z[0, rows], g, eg, "X Wg")
    ref.check(Z[1, rows], u, eu, "X Wu")
    # the elementwise gradient reads all of Z: dX of those rows
    dH = H  # any values
    dX = torch.empty_like(X)
    pg.gated_bf16_backward(M, F, K, X, Wg, Wu, "silu", dH, dX, None, None, preact=Z)
    want = ref.gated_backward(X[rows], Wg, Wu, "silu", dH[rows])
    ref.check(dX[rows], *want["dX"], "dX")


@pytest.mark.parametrize("D", [64, 648])
def test_xent_probabilities_past_31_bits(D):
    T, V = 9000, 240000  # P has 2.16e9 entries, kept in one piece
    X, W = rnd(8, T, D), rnd(9, V, D, std=2 * D ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(10)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    pg.xent_bf16_grad(T, V, D, X, W, y, None, loss, lse, dX, dW, workspace_bytes=6 << 30)
    rows = some_rows(T)
    want = ref.xent(X[rows], W, y[rows], torch.ones(len(rows), device="cuda"))
    for name, got in (("lse", lse), ("loss", loss), ("dX", dX)):
        ref.check(got[rows], *want[name], name)
    # the same gradient in pieces of the vocabulary
    dX2, dW2 = torch.empty_like(X), torch.empty_like(W)
    pg.xent_bf16_grad(T, V, D, X, W, y, None, None, None, dX2, dW2)
    for a, b in ((dX, dX2), (dW, dW2)):
        assert ((a.float() - b.float()).norm() / b.float().norm()).item() < 4e-3


# The largest sizes an int holds, where rounding up to whole tiles passes it.
LAST = 2 ** 31 - 1


@pytest.mark.parametrize("T", [1, 65])
def test_xent_largest_vocabulary(T):
    D = 8
    X = torch.ones(T, D, device="cuda", dtype=torch.bfloat16)
    W = torch.zeros(LAST, D, device="cuda", dtype=torch.bfloat16)
    W[LAST - 1] = 3  # its logit is 24, all others 0
    y = torch.full((T,), LAST - 1, device="cuda", dtype=torch.int64)
    loss = torch.empty(T, device="cuda")
    pg.xent_bf16(T, LAST, D, X, W, y, loss, None)
    want = math.log(math.exp(24.0) + LAST - 1) - 24.0
    # two logarithms near 24 subtracted, and the sums' own errors: 2^-20 of 24 is ample
    assert (loss - want).abs().max().item() <= 24 * 2.0 ** -20


@pytest.mark.parametrize("M,N", [(LAST, 8), (3, LAST), (200, 1 << 24)])
def test_linear_largest_extents(M, N):
    K = 8
    X, W = rnd(21, M, K), rnd(22, K, N)
    Y = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    pg.linear_bf16(M, N, K, X, W, None, "none", None, Y)
    rows, cols = (some_rows(M) if M > 1000 else range(M)), slice(None)
    if N > 1000:
        cols = torch.tensor(some_rows(N), device="cuda")
    rows = torch.tensor(list(rows), device="cuda")
    y, bound, _, _ = ref.linear(X[rows], W[:, cols], None, "none", None)
    ref.check(Y[rows][:, cols] if N <= 1000 else Y[:, cols], y, bound, "Y")
