"""The operators of a mixture-of-experts block against their definitions in 64 bits: norm,
routing, sorting by expert and back, the experts' products, each forward and backward, at
the sizes, group shapes and masks where they can go wrong."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe_reference as moe  # noqa: E402
import operator_reference as ref  # noqa: E402
import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NAN, INF = float("nan"), float("inf")
EPS = 1e-6


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


# ------------------------------------------------------------------- norm ---
NORMS = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 255), (9, 257), (33, 512), (700, 513), (1, 4096),
         (400, 4096), (7, 4097), (311, 1000), (3, 8200), (330, 5121), (2, 16384), (2, 16390),
         (2, 32768), (3, 32767), (1500, 264)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,D", NORMS)
def test_norm(T, D, residual):
    X, R, gain = rnd(1, T, D), rnd(2, T, D, std=3.0) if residual else None, rnd(3, D)
    if T > 2:
        X[1] = 0  # a row of zeros, with or without the residual's
        if residual:
            R[1] = 0
    want = (X.float() + R.float()).to(BF16) if residual else X
    for g in (gain, None):
        S, Y = nan(T, D), nan(T, D)
        pg.rmsnorm_bf16(T, D, X, R, g, EPS, S, Y)
        assert torch.equal(S, want)
        y, err, _, _ = moe.norm(want, g, EPS)
        ref.check(Y, y, moe.bf16_out(y, err), "Y")
        Y2 = nan(T, D)
        pg.rmsnorm_bf16(T, D, X, R, g, EPS, None, Y2)
        assert torch.equal(Y, Y2)
    # in place: S over X, and over the residual
    for into in ("X", "R") if residual else ("X",):
        x, r = X.clone(), R.clone() if residual else None
        Y2 = nan(T, D)
        pg.rmsnorm_bf16(T, D, x, r, None, EPS, x if into == "X" else r, Y2)
        assert torch.equal(x if into == "X" else r, want) and torch.equal(Y, Y2)


@pytest.mark.parametrize("T,D", NORMS)
def test_norm_int8(T, D):
    X, R, gain = rnd(4, T, D), rnd(5, T, D), rnd(6, D)
    if T > 2:
        X[1], R[1] = 0, 0
    S, Q, scale = nan(T, D), torch.full((T, D), 99, device="cuda", dtype=torch.int8), nan(T, dtype=F32)
    pg.rmsnorm_i8(T, D, X, R, gain, EPS, S, Q, scale)
    assert torch.equal(S, (X.float() + R.float()).to(BF16))
    y, err, _, _ = moe.norm(S, gain, EPS)
    step = y.abs().amax(1) / 127
    assert ((scale.double() - step).abs() <= step * (2 * moe.RSTD)).all()
    # half a step, and the error of y and of the scale in steps (at most 127 of them)
    off = (Q.double() * step.unsqueeze(1) - y).abs()
    assert (off <= step.unsqueeze(1) * (0.5 + 127 * 4 * moe.RSTD)).all()
    some = step > 0
    assert (Q.abs().amax(1)[some] == 127).all() and (Q[~some] == 0).all()


def test_norm_not_finite_and_tiny():
    X = rnd(7, 6, 40)
    X[0, 3], X[1, 4], X[2] = INF, NAN, X[2] * 2.0 ** -120
    Y, Q, scale = nan(6, 40), torch.zeros(6, 40, device="cuda", dtype=torch.int8), nan(6, dtype=F32)
    pg.rmsnorm_bf16(6, 40, X, None, None, EPS, None, Y)
    assert Y[1].isnan().all() and Y[0, 3].isnan() and (Y[0, :3] == 0).all()
    assert torch.isfinite(Y[2:].float()).all()
    pg.rmsnorm_i8(6, 40, X, None, None, EPS, None, Q, scale)
    assert scale[:2].isnan().all() and (Q[:2] == 0).all()
    y, _, _, _ = moe.norm(X, None, EPS)
    step = y.abs().amax(1) / 127
    for t in range(2, 6):  # (a row 2^-120 times smaller is quantised as finely)
        assert ((Q[t].double() * step[t] - y[t]).abs() <= step[t] * (0.5 + 127 * 4 * moe.RSTD)).all()


@pytest.mark.parametrize("D", [40, 257, 4096, 8200])
def test_norm_int8_ends_of_the_range(D):
    """Rows whose S gain, or whose squares, lie near the ends of fp32's range while y does
    not: quantised as finely as others."""
    S, gain = rnd(8, 6, D), rnd(9, D)
    scales = [2.0 ** 50, 2.0 ** -50, 1.0, 2.0 ** 20, 2.0 ** -20, 1.0]
    S = (S.float() * torch.tensor(scales, device="cuda").unsqueeze(1)).to(BF16)
    S[5] = 0
    S[5, D // 2] = 2.0 ** -60  # one value
    for by in (2.0 ** 60, 2.0 ** -60, 2.0 ** 110, 2.0 ** -110):
        g = (gain.float() * by).to(BF16)
        Q, scale = torch.full((6, D), 99, device="cuda", dtype=torch.int8), nan(6, dtype=F32)
        pg.rmsnorm_i8(6, D, S, None, g, 1e-30, None, Q, scale)
        y, _, _, _ = moe.norm(S, g, 1e-30)
        step = y.abs().amax(1) / 127
        # (a scale below the normal range is off by half of 2^-149 in itself)
        assert ((scale.double() - step).abs() <= step * (2 * moe.RSTD) + 2.0 ** -150).all()
        off = (Q.double() * step.unsqueeze(1) - y).abs()
        assert (off <= step.unsqueeze(1) * (0.5 + 127 * 4 * moe.RSTD)).all()
        assert (Q.abs().amax(1) == 127).all()


@pytest.mark.parametrize("T,D", NORMS + [(5000, 136), (2500, 1030)])
def test_norm_backward(T, D):
    S, gain, dY, dS = rnd(11, T, D, std=2.0), rnd(12, D), rnd(13, T, D), rnd(14, T, D)
    if T > 2:
        S[1] = 0
    for g, ds in ((gain, dS), (None, None)):
        want = moe.norm_backward(S, g, EPS, dY, ds)
        dX, dg = nan(T, D), nan(D)
        pg.rmsnorm_bf16_backward(T, D, S, g, EPS, dY, ds, dX, dg)
        ref.check(dX, *want["dX"], "dX")
        ref.check(dg, *want["dgain"], "dgain")
        dX2, dg2 = nan(T, D), nan(D)
        pg.rmsnorm_bf16_backward(T, D, S, g, EPS, dY, ds, dX2, None)
        pg.rmsnorm_bf16_backward(T, D, S, g, EPS, dY, ds, None, dg2)
        assert torch.equal(dX, dX2) and torch.equal(dg, dg2)
    over = dS.clone()
    pg.rmsnorm_bf16_backward(T, D, S, gain, EPS, dY, over, over, None)
    pg.rmsnorm_bf16_backward(T, D, S, gain, EPS, dY, dS, dX, None)
    assert torch.equal(over, dX)


def test_norm_nothing():
    dg = nan(16)
    pg.rmsnorm_bf16(0, 16, None, None, None, EPS, None, None)
    pg.rmsnorm_i8(4, 0, None, None, None, EPS, None, None, None)
    pg.rmsnorm_bf16_backward(0, 16, None, None, EPS, None, None, None, dg)
    assert (dg == 0).all()


def test_norm_gradient_against_differences():
    T, D, h = 3, 24, 2.0 ** -6
    S, gain, dY = rnd(15, T, D, dtype=F32).to(BF16), rnd(16, D), rnd(17, T, D)
    dX = nan(T, D)
    pg.rmsnorm_bf16_backward(T, D, S, gain, EPS, dY, None, dX, None)

    def loss(s):
        return (moe.norm(s, gain, EPS)[0] * dY.double()).sum(1)

    s = S.double()
    for i in range(D):
        e = torch.zeros(D, dtype=torch.float64, device="cuda")
        e[i] = h
        diff = (loss(s + e) - loss(s - e)) / (2 * h)
        # central differences: off by h^2 / 6 of the third derivative, which is at most 15
        # times the gradient's size over the row's own scale here
        size = dX.double().abs() + dY.double().abs().amax(1, keepdim=True)
        assert ((dX[:, i].double() - diff).abs() <= size[:, i] * (2.0 ** -7 + 10 * h * h)).all()


# ---------------------------------------------------------------- routing ---
ROUTES = [(1, 1, 1), (1, 8, 2), (5, 31, 4), (7, 32, 32), (33, 33, 5), (64, 64, 8), (300, 100, 1),
          (1000, 128, 8), (17, 200, 6), (9, 500, 3), (3, 1024, 32), (20000, 16, 2)]


def logits(seed, T, E):
    z = rnd(seed, T, E, std=2.0, dtype=F32)
    if T > 4:
        z[1] = -INF                    # nothing open
        z[2, : E - 1] = -INF           # one open
        z[3] = 0.5                     # all equal
        z[4] = z[4].round()            # many equal
        z[torch.rand(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)) < 0.1] = -INF
    return z


@pytest.mark.parametrize("normalise", [False, True])
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route(T, E, k, normalise):
    z = logits(21, T, E)
    experts = torch.full((T, k), 77, device="cuda", dtype=I32)
    w = nan(T, k, dtype=F32)
    pg.route_topk(T, E, k, z, normalise, experts, w)
    want, ww, bound, _ = moe.route(z, k, normalise)
    assert torch.equal(experts, want)
    ref.check(w, ww, bound, "weights")
    dw, dz = rnd(22, T, k, dtype=F32), nan(T, E, dtype=F32)
    dw[experts < 0] = NAN  # what does not count is not read into anything
    pg.route_topk_backward(T, E, k, z, normalise, experts, dw, dz)
    ref.check(dz, *moe.route_backward(z, k, normalise, experts, dw.nan_to_num(0)), "dlogits")


@pytest.mark.parametrize("normalise", [False, True])
@pytest.mark.parametrize("T,E,k", [(200, 5, 5), (64, 40, 8), (300, 128, 32), (33, 300, 17)])
def test_route_backward_expert_twice(T, E, k, normalise):
    """Choices that route_topk would not make: an expert several times, none at all."""
    z, dw = logits(31, T, E), rnd(32, T, k, dtype=F32)
    g = torch.Generator("cuda").manual_seed(33)
    experts = torch.randint(-1, E + 1, (T, k), generator=g, device="cuda", dtype=I32)
    experts[1:T:3] = experts[1:T:3, :1].clone()  # one expert k times
    experts[2:T:3, ::2] = experts[2:T:3, :1].clone()
    if E == 40:
        z = torch.zeros_like(z)
    open_ = z.gather(1, experts.clamp(0, E - 1).long()) > -INF
    experts = torch.where(open_, experts, -1)
    dz = nan(T, E, dtype=F32)
    pg.route_topk_backward(T, E, k, z, normalise, experts, dw, dz)
    ref.check(dz, *moe.route_backward(z, k, normalise, experts, dw), "dlogits")
    again = nan(T, E, dtype=F32)
    pg.route_topk_backward(T, E, k, z, normalise, experts, dw, again)
    assert torch.equal(dz, again)


def test_route_zeros_and_extremes():
    z = torch.zeros(4, 40, device="cuda")
    z[0, 7], z[0, 3] = 0.0, -0.0           # a tie whatever the sign
    z[1, 5], z[1, 30] = 3e38, -3e38
    z[2, 11] = NAN
    z[3, 2] = 1e-45                        # below the normal range, above zero
    experts, w = torch.empty(4, 3, device="cuda", dtype=I32), torch.empty(4, 3, device="cuda")
    for normalise in (True, False):
        pg.route_topk(4, 40, 3, z, normalise, experts, w)
        assert experts.tolist() == [[0, 1, 2], [5, 0, 1], [11, 0, 1], [2, 0, 1]]
        assert w[2].isnan().all() and w[1].tolist() == [1.0, 0.0, 0.0]
        assert torch.isfinite(w[[0, 1, 3]]).all()


def test_route_gradient_against_autograd():
    T, E, k = 50, 24, 4
    z = rnd(23, T, E, dtype=F32)
    dw = rnd(24, T, k, dtype=F32)
    for normalise in (True, False):
        experts, w, dz = (torch.empty(T, n, device="cuda", dtype=t)
                          for n, t in ((k, I32), (k, F32), (E, F32)))
        pg.route_topk(T, E, k, z, normalise, experts, w)
        pg.route_topk_backward(T, E, k, z, normalise, experts, dw, dz)
        leaf = z.double().requires_grad_()
        p = torch.softmax(leaf, 1).gather(1, experts.long())
        p = p / p.sum(1, keepdim=True) if normalise else p
        want, = torch.autograd.grad(p, leaf, dw.double())
        # the bound of moe.route_backward, coarsely: 2^-17 of the row's largest weight gradient
        assert ((dz.double() - want).abs() <= 2.0 ** -17 * dw.abs().sum(1, keepdim=True)).all()


# ------------------------------------------------------------------- sort ---
SORTS = [(1, 1, 1), (1, 4, 2), (3, 5, 3), (24, 64, 8), (100, 1024, 7), (512, 8, 8), (4096, 3, 1),
         (4097, 60, 1), (3000, 33, 6), (40000, 128, 8), (33000, 1000, 9)]


@pytest.mark.parametrize("T,E,k", SORTS)
def test_sort(T, E, k):
    g = torch.Generator("cuda").manual_seed(31)
    experts = torch.randint(0, E, (T, k), device="cuda", generator=g).int()
    drop = torch.rand(T, k, device="cuda", generator=g)
    for dropped in (False, True):
        x = experts.clone()
        if dropped:
            x[drop < 0.2] = -1
            x[drop > 0.9] = E
            x[drop > 0.95] = 2 ** 31 - 1
            x[(x >= E // 3) & (x < E // 2)] = E - 1  # empty groups
        offsets = torch.full((E + 1,), 77, device="cuda", dtype=I32)
        rows = torch.full((T, k), 77, device="cuda", dtype=I32)
        pg.expert_sort(T, E, k, x, offsets, rows)
        want_offsets, want_rows = moe.sort(x, E)
        assert torch.equal(offsets.cpu(), want_offsets)
        assert torch.equal(rows.cpu(), want_rows)


def test_sort_all_to_one_or_none():
    T, E, k = 5000, 16, 2
    for value, count in ((11, T * k), (-1, 0)):
        x = torch.full((T, k), value, device="cuda", dtype=I32)
        offsets, rows = torch.empty(E + 1, device="cuda", dtype=I32), torch.empty_like(x)
        pg.expert_sort(T, E, k, x, offsets, rows)
        assert offsets.tolist() == [0] * 12 + [count] * 5
        assert torch.equal(rows.reshape(-1), torch.arange(T * k, device="cuda", dtype=I32)
                           if count else torch.full((T * k,), -1, device="cuda", dtype=I32))
    offsets.fill_(5)
    pg.expert_sort(0, E, k, None, offsets, None)
    assert (offsets == 0).all()


# ----------------------------------------------------- gather and combine ---
ROWS = [(1, 1, 1), (1, 8, 2048), (5, 3, 7), (24, 8, 256), (300, 2, 1000), (77, 5, 258), (9, 40, 64),
        (1000, 4, 4096), (3, 6, 5000), (130, 4, 33)]


def rows_of(T, k, drop=0.15):
    """A random placing of the slots, some of them dropped, in one of the rows behind."""
    g = torch.Generator("cuda").manual_seed(41)
    rows = torch.randperm(T * k, device="cuda", generator=g).int().reshape(T, k)
    out = torch.rand(T, k, device="cuda", generator=g) < drop
    if T > 2:
        out[1] = True
    unused = rows[out].long()
    rows[out] = -1
    if T > 2:
        rows[1, 0] = T * k  # beyond the last row
    return rows, unused


@pytest.mark.parametrize("T,k,D", ROWS)
def test_gather_and_combine(T, k, D):
    rows, unused = rows_of(T, k)
    ok = (rows >= 0) & (rows < T * k)
    seen = torch.where(ok, rows, -1)
    X, Ys, R, dY = rnd(42, T, D), rnd(43, T * k, D), rnd(44, T, D), rnd(45, T, D)
    w = rnd(46, T, k, dtype=F32)
    Xs = torch.full((T * k, D), 7.0, device="cuda", dtype=BF16)
    pg.expert_gather_bf16(T, k, D, X, rows, Xs)
    want = torch.full_like(Xs, 7.0)
    want[rows[ok].long()] = X.unsqueeze(1).expand(T, k, D)[ok]
    assert torch.equal(Xs, want)
    Ys[unused] = NAN  # rows of no slot, and weights of slots that do not count
    w[~ok] = NAN
    clean, wc = Ys.nan_to_num(0), w.nan_to_num(0)
    for weights, wanted in ((w, wc), (None, None)):
        for res in (R, None):
            Y = nan(T, D)
            pg.expert_combine_bf16(T, k, D, Ys, rows, weights, res, Y)
            ref.check(Y, *moe.combine(clean, seen, wanted, res), "Y")
            if res is not None:
                over = R.clone()
                pg.expert_combine_bf16(T, k, D, Ys, rows, weights, over, over)
                assert torch.equal(over, Y)
        d, ed, dw, ew = moe.combine_backward(clean, seen, wanted, dY)
        dYs, dweights = torch.full_like(Ys, 7.0), nan(T, k, dtype=F32)
        pg.expert_combine_bf16_backward(T, k, D, Ys, rows, weights, dY, dYs, dweights)
        ref.check(dweights, dw, ew, "dweights")
        ref.check(dYs[rows[ok].long()], d[ok], ed[ok], "dYs")
        assert (dYs[unused] == 7).all()
        other = torch.full_like(Ys, 7.0)
        pg.expert_combine_bf16_backward(T, k, D, None, rows, weights, dY, other, None)
        assert torch.equal(other, dYs)
        only = nan(T, k, dtype=F32)
        pg.expert_combine_bf16_backward(T, k, D, Ys, rows, weights, dY, None, only)
        assert torch.equal(only, dweights)


def test_combine_adds_one_row_twice():
    # the same row in two slots: allowed forward (the backward call refuses nothing, but has
    # one place for two gradients)
    Ys = rnd(47, 4, 16)
    rows = torch.tensor([[0, 0], [3, 1]], device="cuda", dtype=I32)
    w = torch.tensor([[0.25, 0.5], [1.0, 2.0]], device="cuda")
    Y = nan(2, 16)
    pg.expert_combine_bf16(2, 2, 16, Ys, rows, w, None, Y)
    ref.check(Y, *moe.combine(Ys, rows, w, None), "Y")


# ----------------------------------------------------------------- experts ---
# group sizes, for the kernel of many rows a group and that of few
GROUPS = {
    "ragged": [0, 1, 31, 32, 33, 255, 256, 257, 0, 300, 64],
    "one": [700],
    "few": [1, 0, 0, 2, 17, 0, 16, 33, 64, 65, 0, 1],
    "single": [0, 0, 1, 0],
    "none": [0, 0, 0],
    "large": [1030, 5, 2000],
}
SIZES = [(64, 64), (8, 8), (1, 1), (72, 136), (133, 72), (264, 1000), (1365, 520), (130, 2050),
         (2, 4104)]  # (N, K)


def grouped(name, N, K, behind=3):
    sizes = GROUPS[name]
    offsets = torch.tensor([0] + sizes, device="cuda").cumsum(0).int()
    R = sum(sizes) + behind
    X = rnd(51, R, K)
    X[R - behind:] = NAN  # rows behind the last group
    return R, len(sizes), offsets, X


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("N,K", SIZES)
def test_experts_linear(N, K, name):
    R, E, offsets, X = grouped(name, N, K)
    live = int(offsets[-1])
    W, dY = rnd(52, E, K, N, std=K ** -0.5), rnd(53, R, N)
    dY[live:] = NAN
    Y = torch.full((R, N), 7.0, device="cuda", dtype=BF16)
    pg.experts_linear_bf16(R, N, K, E, offsets, X, W, Y)
    want = moe.experts_linear(offsets, X, W)
    ref.check(Y[:live], *want["Y"], "Y")
    assert (Y[live:] == 7).all()
    dX, dW = torch.full((R, K), 7.0, device="cuda", dtype=BF16), nan(E, K, N)
    pg.experts_linear_bf16_backward(R, N, K, E, offsets, X, W, dY, dX, dW)
    want = moe.experts_linear_backward(offsets, X, W, dY)
    ref.check(dX[:live], *want["dX"], "dX")
    assert (dX[live:] == 7).all()
    ref.check(dW, *want["dW0"], "dW")
    dX2, dW2 = torch.full_like(dX, 7.0), nan(E, K, N)
    pg.experts_linear_bf16_backward(R, N, K, E, offsets, None, W, dY, dX2, None)
    pg.experts_linear_bf16_backward(R, N, K, E, offsets, X, None, dY, None, dW2)
    assert torch.equal(dX, dX2) and torch.equal(dW, dW2)


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("F,K", SIZES)
def test_experts_gated(F, K, name):
    act = ["silu", "gelu", "gelu_tanh", "none"][(F + K + len(name)) % 4]
    R, E, offsets, X = grouped(name, F, K)
    live = int(offsets[-1])
    Wg, Wu = rnd(54, E, K, F, std=K ** -0.5), rnd(55, E, K, F, std=K ** -0.5)
    dH = rnd(56, R, F)
    dH[live:] = NAN
    H, Z = torch.full((R, F), 7.0, device="cuda", dtype=BF16), torch.full((2, R, F), 7.0, device="cuda")
    pg.experts_gated_bf16(R, F, K, E, offsets, X, Wg, Wu, act, H, preact=Z)
    want = moe.experts_gated(offsets, X, Wg, Wu, act)
    ref.check(H[:live], *want["H"], "H")
    ref.check(Z[0, :live], *want["G"], "G")
    ref.check(Z[1, :live], *want["U"], "U")
    assert (H[live:] == 7).all() and (Z[:, live:] == 7).all()
    H2 = torch.full_like(H, 7.0)
    pg.experts_gated_bf16(R, F, K, E, offsets, X, Wg, Wu, act, H2)
    assert torch.equal(H, H2)
    want = moe.experts_gated_backward(offsets, X, Wg, Wu, act, dH)
    for kept in (Z, None):
        dX, dWg, dWu = torch.full((R, K), 7.0, device="cuda", dtype=BF16), nan(E, K, F), nan(E, K, F)
        pg.experts_gated_bf16_backward(R, F, K, E, offsets, X, Wg, Wu, act, dH, dX, dWg, dWu,
                                       preact=kept)
        ref.check(dX[:live], *want["dX"], "dX")
        assert (dX[live:] == 7).all()
        ref.check(dWg, *want["dW0"], "dWg")
        ref.check(dWu, *want["dW1"], "dWu")
        only = torch.full_like(dX, 7.0)
        pg.experts_gated_bf16_backward(R, F, K, E, offsets, None if kept is not None else X, Wg, Wu,
                                       act, dH, only, None, None, preact=kept)
        assert torch.equal(only, dX)


@pytest.mark.parametrize("sizes", [[3, 70, 200, 5], [3, 7, 20, 5, 1, 1, 1, 2]])
def test_one_experts_nan_stays_with_it(sizes):
    N, K, E = 136, 200, len(sizes)
    offsets = torch.tensor([0] + sizes, device="cuda").cumsum(0).int()
    R, bad = sum(sizes), 1
    a, b = int(offsets[bad]), int(offsets[bad + 1])
    X, W, dY = rnd(61, R, K), rnd(62, E, K, N), rnd(63, R, N)

    def run():
        Y, dX, dW = nan(R, N), nan(R, K), nan(E, K, N)
        pg.experts_linear_bf16(R, N, K, E, offsets, X, W, Y)
        pg.experts_linear_bf16_backward(R, N, K, E, offsets, X, W, dY, dX, dW)
        return Y, dX, dW

    clean = run()
    X[a:b], dY[a:b], W[bad] = NAN, INF, NAN
    Y, dX, dW = run()
    for got, was in ((Y, clean[0]), (dX, clean[1])):
        assert torch.equal(got[:a], was[:a]) and torch.equal(got[b:], was[b:])
        assert got[a:b].isnan().all()
    assert torch.equal(dW[:bad], clean[2][:bad]) and torch.equal(dW[bad + 1:], clean[2][bad + 1:])
    assert dW[bad].isnan().all()


def test_experts_offsets_beyond_the_rows():
    # what the offsets say beyond R counts as R, below 0 as 0: nothing outside is touched
    R, N, K, E = 70, 72, 64, 4
    X, W, dY = rnd(64, R, K), rnd(65, E, K, N), rnd(66, R, N)
    good = torch.tensor([0, 0, 30, 70, 70], device="cuda", dtype=I32)
    wild = torch.tensor([-5, 0, 30, 2 ** 31 - 1, 99], device="cuda", dtype=I32)
    got = []
    for offsets in (good, wild):
        Y, dX, dW = nan(R, N), nan(R, K), nan(E, K, N)
        pg.experts_linear_bf16(R, N, K, E, offsets, X, W, Y)
        pg.experts_linear_bf16_backward(R, N, K, E, offsets, X, W, dY, dX, dW)
        got.append((Y, dX, dW))
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_experts_many_experts():
    E, N, K = 1024, 40, 72
    g = torch.Generator("cuda").manual_seed(67)
    sizes = torch.randint(0, 4, (E,), device="cuda", generator=g)
    offsets = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).int()
    R = int(offsets[-1])
    X, W, dY = rnd(68, R, K), rnd(69, E, K, N), rnd(70, R, N)
    Y, dX, dW = nan(R, N), nan(R, K), nan(E, K, N)
    pg.experts_linear_bf16(R, N, K, E, offsets, X, W, Y)
    pg.experts_linear_bf16_backward(R, N, K, E, offsets, X, W, dY, dX, dW)
    ref.check(Y, *moe.experts_linear(offsets, X, W)["Y"], "Y")
    want = moe.experts_linear_backward(offsets, X, W, dY)
    ref.check(dX, *want["dX"], "dX")
    ref.check(dW, *want["dW0"], "dW")


def test_experts_empty_extents():
    offsets = torch.tensor([0, 2, 5], device="cuda", dtype=I32)
    X, W = rnd(71, 5, 16), rnd(72, 2, 16, 24)
    Y = nan(5, 24)
    pg.experts_linear_bf16(5, 24, 0, 2, offsets, None, None, Y)  # an empty product is zero
    assert (Y == 0).all()
    H = nan(5, 24)
    pg.experts_gated_bf16(5, 24, 0, 2, offsets, None, None, None, "silu", H)
    assert (H == 0).all()
    dX, dW = nan(5, 16), nan(2, 16, 24)
    pg.experts_linear_bf16_backward(5, 0, 16, 2, offsets, X, None, None, dX, None)
    assert (dX == 0).all()
    pg.experts_linear_bf16_backward(0, 24, 16, 2, offsets, None, None, None, None, dW)
    assert (dW == 0).all()
    dWg, dWu = nan(2, 16, 24), nan(2, 16, 24)
    pg.experts_gated_bf16_backward(0, 24, 16, 2, offsets, None, None, None, "silu", None, None, dWg,
                                   dWu)
    assert (dWg == 0).all() and (dWu == 0).all()
    pg.experts_linear_bf16(0, 24, 16, 2, None, None, None, None)
    pg.experts_linear_bf16(5, 0, 16, 2, None, None, None, None)
