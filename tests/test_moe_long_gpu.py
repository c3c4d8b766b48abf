"""The experts' products of long sums: weight gradients of many rows are as exact as of few, and
no wait runs out, up to 2^31 - 1 rows; forward and dX at the most columns that they take."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe_reference as moe  # noqa: E402
import operator_reference as ref  # noqa: E402
import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402

BF16 = torch.bfloat16
ROUND = 8256  # rows whose products the kernel adds in the tensor core


@pytest.fixture(autouse=True)
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


def positive(seed, R, n):
    """Values of one sign, whose sums lose most to truncation; columns of different sizes, so
    that the sums lie all over a binade."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = 1 + torch.arange(n, device="cuda") / n
    out = torch.empty(R, n, device="cuda", dtype=BF16)
    for part in out.split(1 << 24):
        part.copy_((0.5 + 0.5 * torch.rand(part.shape, generator=g, device="cuda")) * size)
    return out


def offsets_of(sizes):
    return torch.tensor([0] + sizes, device="cuda").cumsum(0).int()


def check_weights(dW, X, dY, sizes):
    a = 0
    for e, n in enumerate(sizes):
        want = torch.zeros(X.shape[1], dY.shape[1], dtype=torch.float64, device="cuda")
        for i in range(a, a + n, 1 << 23):
            j = min(i + (1 << 23), a + n)
            want += X[i:j].double().t() @ dY[i:j].double()
        a += n
        # Every term is positive, so the sum of magnitudes is the sum: 2^-23 of it for each
        # step of 16 rows of a round, 2^-24 for each addition of a round, and half of the
        # last of bf16's eight bits.
        err = want * ((ROUND / 16 + 4) * 2.0 ** -23 + n // ROUND * 2.0 ** -24)
        half = torch.exp2(torch.floor(torch.log2(want + err)) - 8)
        off = (dW[e].double() - want).abs()
        assert (off <= err + torch.where(want > 0, half, 0)).all(), \
            (e, n, float((off / (err + half)).max()))


def test_weights_of_long_groups_are_as_exact():
    sizes = [1_500_007, 300_000, 16, ROUND, ROUND + 1, 0, 2 * ROUND, 2 * ROUND + 15, 3 * ROUND - 1]
    R, K, N, E = sum(sizes), 72, 64, len(sizes)
    X, dY = positive(1, R, K), positive(2, R, N)
    for n in (N, N - 1):  # (by TMA, and by plain stores)
        d = dY[:, :n].contiguous()
        dW = torch.full((E, K, n), float("nan"), device="cuda", dtype=BF16)
        pg.experts_linear_bf16_backward(R, n, K, E, offsets_of(sizes), X, None, d, None, dW)
        check_weights(dW, X, d, sizes)


@pytest.mark.parametrize("sizes", [[ROUND + 1, 5, 2 * ROUND + 16], [40] * 60 + [3 * ROUND, 0, 33]])
def test_gated_weights_of_several_rounds(sizes):
    """(few rows a group on average, and many: both of the kernel's configurations)"""
    R, K, F, E = sum(sizes), 136, 72, len(sizes)
    g = torch.Generator(device="cuda").manual_seed(3)

    def rnd(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)

    X, dH = rnd(R, K), rnd(R, F)
    Wg, Wu = rnd(E, K, F, std=K ** -0.5), rnd(E, K, F, std=K ** -0.5)
    dX, dWg, dWu = torch.empty_like(X), torch.empty_like(Wg), torch.empty_like(Wu)
    offsets = offsets_of(sizes)
    pg.experts_gated_bf16_backward(R, F, K, E, offsets, X, Wg, Wu, "silu", dH, dX, dWg, dWu)
    want = moe.experts_gated_backward(offsets, X, Wg, Wu, "silu", dH)
    ref.check(dX, *want["dX"], "dX")
    ref.check(dWg, *want["dW0"], "dWg")
    ref.check(dWu, *want["dW1"], "dWu")


def test_weights_of_as_many_rows_as_an_int_counts():
    """Two groups of some 2^30 rows take seconds each, and the short groups behind them on the
    same CTAs wait that long for their last rows."""
    K = N = 8
    short = [7] * 88
    sizes = [2 ** 30, 2 ** 30 - 1 - sum(short)] + short
    R, E = sum(sizes), len(sizes)
    assert R == 2 ** 31 - 1
    X, dY = positive(4, R, K), positive(5, R, N)
    dW = torch.full((E, K, N), float("nan"), device="cuda", dtype=BF16)
    pg.experts_linear_bf16_backward(R, N, K, E, offsets_of(sizes), X, None, dY, None, dW)
    torch.cuda.synchronize()
    check_weights(dW, X, dY, sizes)


@pytest.mark.parametrize("sizes", [[1, 3], [41] * 40])  # (tiles of one CTA, and of a pair)
def test_sums_of_as_many_columns_as_there_may_be(sizes):
    K, N, E, R = 2 ** 19, 24, len(sizes), sum(sizes)
    offsets = offsets_of(sizes)
    X, W = positive(6, R, K), positive(7, E * K, N).view(E, K, N)
    Y, H = (torch.full((R, N), float("nan"), device="cuda", dtype=BF16) for _ in range(2))
    pg.experts_linear_bf16(R, N, K, E, offsets, X, W, Y)
    ref.check(Y, *moe.experts_linear(offsets, X, W)["Y"], "Y")
    pg.experts_gated_bf16(R, N, K, E, offsets, X, W, W, "none", H)
    ref.check(H, *moe.experts_gated(offsets, X, W, W, "none")["H"], "H")
    Wt, dX = positive(8, E * N, K).view(E, N, K), torch.full_like(Y, float("nan"))
    pg.experts_linear_bf16_backward(R, K, N, E, offsets, None, Wt, X, dX, None)  # X as dY
    want = moe.experts_linear_backward(offsets, Y.zero_(), Wt, X)
    ref.check(dX, *want["dX"], "dX")
    g = torch.Generator(device="cuda").manual_seed(9)
    F = K // 2
    Z = torch.rand(2, R, F, generator=g, device="cuda")
    pg.experts_gated_bf16_backward(R, F, N, E, offsets, None, Wt[..., :F].contiguous(),
                                   Wt[..., F:].contiguous(), "none", X[:, :F].contiguous(), dX,
                                   None, None, preact=Z)
    for e, a, b in moe.groups(offsets):
        d = X[a:b, :F].double()
        dz = torch.cat([d * Z[1, a:b], d * Z[0, a:b]], 1)  # dG, dU: act is the identity
        y = dz @ Wt[e].double().t()
        # of positive terms: their rounding to bf16 and 2^-23 for every 16 columns
        ref.check(dX[a:b], y, moe.bf16_out(y, y * (2.0 ** -8 + ref.step(K))), "gated dX")
