"""Rows of every width through the operators of a mixture-of-experts block that take them in
16-byte vectors: all alignments of a row, all ways its ends can fall, several rows a block; and
the zeros of experts without rows, wherever their matrices begin."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe_reference as moe  # noqa: E402
import operator_reference as ref  # noqa: E402
import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NAN, EPS = float("nan"), 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from software_pipelined_tiled_loop_gb300 import build
    build.build()
    pg.lib()
    yield
    assert pg.pgemm_get_device_status() == 0


def rnd(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def nan(*shape, dtype=BF16):
    return torch.full(shape, NAN, device="cuda", dtype=dtype)


def guarded(*shape):
    """A view of NaNs with 64 sevens before and behind it, and the whole."""
    n = 1
    for d in shape:
        n *= d
    whole = torch.full((n + 128,), 7.0, device="cuda", dtype=BF16)
    whole[64:64 + n] = NAN
    return whole[64:64 + n].view(shape), whole


def kept(whole):
    return bool((whole[:64] == 7).all() and (whole[-64:] == 7).all())


@pytest.mark.parametrize("T,k", [(23, 1), (19, 2), (11, 3), (9, 6)])
@pytest.mark.parametrize("D", list(range(1, 42)) + [255, 263, 2050, 2052, 4097])
def test_gather_and_combine(T, k, D):
    g = torch.Generator("cuda").manual_seed(D)
    rows = torch.randperm(T * k, device="cuda", generator=g).int().reshape(T, k)
    rows[4] = -1
    ok = rows >= 0
    X, Ys, R, dY = rnd(1, T, D), rnd(2, T * k, D), rnd(3, T, D), rnd(4, T, D)
    w = rnd(5, T, k, dtype=F32)
    Xs, whole = guarded(T * k, D)
    pg.expert_gather_bf16(T, k, D, X, rows, Xs)
    want = nan(T * k, D)
    want[rows[ok].long()] = X.unsqueeze(1).expand(T, k, D)[ok]
    assert torch.equal(Xs.view(torch.int16), want.view(torch.int16)) and kept(whole)
    for weights in (w, None):
        Y, whole = guarded(T, D)
        pg.expert_combine_bf16(T, k, D, Ys, rows, weights, R, Y)
        ref.check(Y, *moe.combine(Ys, rows, weights, R), "Y")
        assert kept(whole)
    d, ed, dw, ew = moe.combine_backward(Ys, rows, w, dY)
    dYs, whole = guarded(T * k, D)
    dweights = nan(T, k, dtype=F32)
    pg.expert_combine_bf16_backward(T, k, D, Ys, rows, w, dY, dYs, dweights)
    ref.check(dweights, dw, ew, "dweights")
    ref.check(dYs[rows[ok].long()], d[ok], ed[ok], "dYs")
    assert kept(whole)


def test_neighbours_do_not_leak():
    """A row's vectors hold its neighbours' ends: a NaN there reaches no other row."""
    T, k = 16, 2
    for D in (9, 12, 31, 130):
        rows = torch.randperm(T * k, device="cuda").int().view(T, k)
        Ys, dY, w = rnd(6, T * k, D), rnd(7, T, D), rnd(8, T, k, dtype=F32)
        Ys[rows[5].long()], dY[5] = NAN, NAN
        S, gain = rnd(9, T, D), rnd(10, D)
        S[5] = NAN
        rest = [t for t in range(T) if t != 5]
        Y, dYs, dw = nan(T, D), nan(T * k, D), nan(T, k, dtype=F32)
        pg.expert_combine_bf16(T, k, D, Ys, rows, w, None, Y)
        pg.expert_combine_bf16_backward(T, k, D, Ys, rows, w, dY, dYs, dw)
        assert torch.isfinite(Y[rest].float()).all() and Y[5].isnan().all()
        assert torch.isfinite(dw[rest]).all() and dw[5].isnan().all()
        assert torch.isfinite(dYs[rows[rest].long()].float()).all()
        Y, dX = nan(T, D), nan(T, D)
        pg.rmsnorm_bf16(T, D, S, None, gain, EPS, None, Y)
        pg.rmsnorm_bf16_backward(T, D, S, gain, EPS, rnd(11, T, D), None, dX, None)
        assert torch.isfinite(Y[rest].float()).all() and torch.isfinite(dX[rest].float()).all()


# more rows than blocks run at once: a block's rows all start at the same place of a vector
@pytest.mark.parametrize("T,D", [(20000, 9), (9001, 65), (6005, 129), (3007, 1001), (2003, 2046),
                                 (1300, 8201), (700, 16390), (400, 20487), (333, 32761), (700, 10241), (450, 12290), (400, 16363)])
def test_norm_of_odd_widths_in_many_rows(T, D):
    X, R, gain, dY = rnd(21, T, D), rnd(22, T, D), rnd(23, D), rnd(24, T, D)
    S, Y = nan(T, D), nan(T, D)
    pg.rmsnorm_bf16(T, D, X, R, gain, EPS, S, Y)
    assert torch.equal(S, (X.float() + R.float()).to(BF16))
    y, err, _, _ = moe.norm(S, gain, EPS)
    ref.check(Y, y, moe.bf16_out(y, err), "Y")
    Q, scale = torch.full((T, D), 99, device="cuda", dtype=torch.int8), nan(T, dtype=F32)
    pg.rmsnorm_i8(T, D, X, R, gain, EPS, None, Q, scale)
    step = y.abs().amax(1) / 127
    assert ((scale.double() - step).abs() <= step * (2 * moe.RSTD)).all()
    off = (Q.double() * step.unsqueeze(1) - y).abs()
    assert (off <= step.unsqueeze(1) * (0.5 + 127 * 4 * moe.RSTD)).all()
    del y, err, off, Q
    want = moe.norm_backward(S, gain, EPS, dY, R)
    dX, dg = nan(T, D), nan(D)
    pg.rmsnorm_bf16_backward(T, D, S, gain, EPS, dY, R, dX, dg)
    ref.check(dX, *want["dX"], "dX")
    ref.check(dg, *want["dgain"], "dgain")


@pytest.mark.parametrize("sizes", [[0], [0, 0, 3, 0], [0, 40, 0, 0, 17, 0]])
@pytest.mark.parametrize("N,K", [(1, 1), (1, 3), (3, 1), (5, 5), (8, 8), (257, 3), (129, 301),
                                 (520, 264)])
def test_zeros_of_experts_without_rows(N, K, sizes):
    """dW of odd sizes, whose matrices begin anywhere in a vector; and weights of experts
    without rows, which may hold anything."""
    E, R = len(sizes), sum(sizes) + 2
    offsets = torch.tensor([0] + sizes, device="cuda").cumsum(0).int()
    live = int(offsets[-1])
    X, dY, W = rnd(31, R, K), rnd(32, R, N), rnd(33, E, K, N)
    U = rnd(34, E, K, N)
    for e, n in enumerate(sizes):
        if n == 0:
            W[e], U[e] = NAN, NAN
    dW, whole = guarded(E, K, N)
    dX = nan(R, K)
    pg.experts_linear_bf16_backward(R, N, K, E, offsets, X, W, dY, dX, dW)
    assert kept(whole)
    want = moe.experts_linear_backward(offsets, X, W, dY)
    ref.check(dW, *want["dW0"], "dW")
    ref.check(dX[:live], *want["dX"], "dX")
    dG, whole_g = guarded(E, K, N)
    dU, whole_u = guarded(E, K, N)
    pg.experts_gated_bf16_backward(R, N, K, E, offsets, X, W, U, "silu", dY, dX, dG, dU)
    assert kept(whole_g) and kept(whole_u)
    want = moe.experts_gated_backward(offsets, X, W, U, "silu", dY)
    ref.check(dG, *want["dW0"], "dWg")
    ref.check(dU, *want["dW1"], "dWu")
