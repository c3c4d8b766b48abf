"""A mixture-of-experts block's operators where operands pass 2^31 elements, and at the
largest sizes an int holds: rows at the top, middle and bottom against 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe_reference as moe  # noqa: E402
import operator_reference as ref  # noqa: E402
import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
LAST = 2 ** 31 - 1
EPS = 1e-6


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


def rnd(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, device="cuda", dtype=BF16)
    for part in out.view(-1).split(1 << 28):  # few fp32 temporaries
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * std)
    return out


def some(M):
    return torch.tensor([*range(0, 30), *range(M // 2, M // 2 + 30), *range(M - 30, M)],
                        device="cuda")


@pytest.mark.parametrize("T,D", [(70000, 32768), (70000, 32003), (LAST, 8), (LAST, 3)])
def test_norm(T, D):
    S, gain = rnd(1, T, D), rnd(2, D)
    Y, rows = torch.empty_like(S), some(T)
    pg.rmsnorm_bf16(T, D, S, None, gain, EPS, None, Y)
    y, err, _, _ = moe.norm(S[rows], gain, EPS)
    ref.check(Y[rows], y, moe.bf16_out(y, err), "Y")
    dX = torch.empty_like(S)  # Y as its own gradient
    pg.rmsnorm_bf16_backward(T, D, S, gain, EPS, Y, None, dX, None)
    ref.check(dX[rows], *moe.norm_backward(S[rows], gain, EPS, Y[rows], None)["dX"], "dX")
    Q, scale = Y.view(torch.int8).view(-1)[:T * D].view(T, D), torch.empty(T, device="cuda")
    pg.rmsnorm_i8(T, D, S, None, gain, EPS, None, Q, scale)
    step = y.abs().amax(1) / 127
    assert ((Q[rows].double() * step.unsqueeze(1) - y).abs()
            <= step.unsqueeze(1) * (0.5 + 127 * 4 * moe.RSTD)).all()


def test_norm_gain_gradient_over_many_rows():
    T, D = 300000, 8192  # 2.5e9 elements
    S, dY = rnd(3, T, D), rnd(4, T, D)
    dg = torch.empty(D, device="cuda", dtype=BF16)
    pg.rmsnorm_bf16_backward(T, D, S, None, EPS, dY, None, None, dg)
    total = torch.zeros(D, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(total)
    for a in range(0, T, 20000):
        _, _, n, _ = moe.norm(S[a:a + 20000], None, EPS)
        d = dY[a:a + 20000].double() * n
        total += d.sum(0)
        size += d.abs().sum(0)
    err = size * (2 * moe.RSTD + (T / 100 + 100) * moe.EPS24)  # a block's rows, then the blocks
    ref.check(dg, total, moe.bf16_out(total, err), "dgain")


def test_rows_past_31_bits():
    T, k, D = 40000, 4, 16392  # 2.6e9 elements of sorted rows
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = torch.randperm(T * k, device="cuda", generator=g).int().view(T, k)
    X, w = rnd(6, T, D), torch.rand(T, k, device="cuda", generator=g)
    Xs = torch.empty(T * k, D, device="cuda", dtype=BF16)
    pg.expert_gather_bf16(T, k, D, X, rows, Xs)
    at = some(T)
    assert torch.equal(Xs[rows[at].long()], X[at].unsqueeze(1).expand(-1, k, D))
    Y = torch.empty_like(X)
    pg.expert_combine_bf16(T, k, D, Xs, rows, w, X, Y)

    def sub(t):  # those tokens and their rows alone
        return t[rows[at].long()].view(-1, D)

    own = torch.arange(at.numel() * k, device="cuda", dtype=I32).view(-1, k)
    ref.check(Y[at], *moe.combine(sub(Xs), own, w[at], X[at]), "Y")
    dYs, dw = torch.empty_like(Xs), torch.empty(T, k, device="cuda")
    pg.expert_combine_bf16_backward(T, k, D, Xs, rows, w, Y, dYs, dw)
    d, ed, v, ev = moe.combine_backward(sub(Xs), own, w[at], Y[at])
    ref.check(dYs[rows[at].long()], d, ed, "dYs")
    ref.check(dw[at], v, ev, "dweights")


@pytest.mark.parametrize("T,k,D", [(1, 2, LAST), (LAST // 2, 2, 4), (1, 1, LAST - 1)])
def test_rows_largest_extents(T, k, D):
    rows = torch.arange(T * k, device="cuda", dtype=I32).view(T, k)
    X = rnd(7, T, D)
    Xs = torch.empty(T * k, D, device="cuda", dtype=BF16)
    pg.expert_gather_bf16(T, k, D, X, rows, Xs)
    at = slice(-30, None)
    assert torch.equal(Xs.view(T, k, D)[at, -1, -40:], X[at, -40:])
    assert torch.equal(Xs.view(T, k, D)[:30, 0, :40], X[:30, :40])
    Y = torch.empty_like(X)
    pg.expert_combine_bf16(T, k, D, Xs, rows, None, None, Y)
    assert torch.equal(Y[at, -40:], X[at, -40:] * k)


def test_sort_of_many_slots():
    T, E, k = 30_000_000, 64, 8
    g = torch.Generator(device="cuda").manual_seed(8)
    experts = torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=I32)
    offsets, rows = torch.empty(E + 1, device="cuda", dtype=I32), torch.empty_like(experts)
    pg.expert_sort(T, E, k, experts, offsets, rows)
    counts = torch.bincount(experts.view(-1), minlength=E)
    assert torch.equal(offsets[1:].long(), counts.cumsum(0)) and offsets[0] == 0
    # a stable sort: read in the rows' order, slots ascend within each expert
    slot = torch.empty(T * k, dtype=I32, device="cuda")
    slot[rows.view(-1).long()] = torch.arange(T * k, device="cuda", dtype=I32)
    sorted_experts = experts.view(-1)[slot.long()]
    up = sorted_experts[1:] - sorted_experts[:-1]
    assert (up >= 0).all()
    assert ((slot[1:] > slot[:-1]) | (up > 0)).all()


def test_route_many_tokens():
    T, E, k = 20_000_000, 120, 2
    z = torch.empty(T, E, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    for part in z.split(1 << 21):
        part.normal_(generator=g)
    experts = torch.empty(T, k, device="cuda", dtype=I32)
    w, dz = torch.empty(T, k, device="cuda"), torch.empty_like(z)
    pg.route_topk(T, E, k, z, True, experts, w)
    at = some(T)
    want, ww, bound, _ = moe.route(z[at], k, True)
    assert torch.equal(experts[at], want)
    ref.check(w[at], ww, bound, "weights")
    pg.route_topk_backward(T, E, k, z, True, experts, w, dz)
    ref.check(dz[at], *moe.route_backward(z[at], k, True, experts[at], w[at]), "dlogits")


def groups(sizes):
    return torch.tensor([0] + sizes, device="cuda").cumsum(0).int()


@pytest.mark.parametrize("N", [4104, 4099])
def test_experts_weights_past_31_bits(N):
    E, K = 130, 4104  # 2.2e9 elements of weights
    sizes = [(7 * e) % 23 for e in range(E)]
    sizes[0], sizes[-1] = 40, 55
    offsets, R = groups(sizes), sum(sizes)
    X, W, dY = rnd(10, R, K), rnd(11, E, K, N, std=K ** -0.5), rnd(12, R, N)
    Y, dX, dW = torch.empty_like(dY), torch.empty_like(X), torch.empty_like(W)
    pg.experts_linear_bf16(R, N, K, E, offsets, X, W, Y)
    pg.experts_linear_bf16_backward(R, N, K, E, offsets, X, W, dY, dX, dW)
    for e in (0, 1, 64, E - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        y, bound, _, _ = ref.linear(X[a:b], W[e], None, "none", None)
        ref.check(Y[a:b], y, bound, "Y")
        want = ref.linear_backward(X[a:b], W[e], None, "none", dY[a:b])
        ref.check(dX[a:b], *want["dX"], "dX")
        ref.check(dW[e], *want["dW0"], "dW")


@pytest.mark.parametrize("F", [33024, 33003])
def test_experts_rows_past_31_bits(F):
    K, E = 64, 2  # 2 R F > 2^31
    sizes = [30011, 10000]
    offsets, R = groups(sizes), sum(sizes)
    X, Wg, Wu = rnd(13, R, K), rnd(14, E, K, F, std=0.125), rnd(15, E, K, F, std=0.125)
    H, Z = torch.empty(R, F, device="cuda", dtype=BF16), torch.empty(2, R, F, device="cuda")
    pg.experts_gated_bf16(R, F, K, E, offsets, X, Wg, Wu, "silu", H, preact=Z)
    dX = torch.empty_like(X)
    pg.experts_gated_bf16_backward(R, F, K, E, offsets, X, Wg, Wu, "silu", H, dX, None, None,
                                   preact=Z)
    dX2 = torch.empty_like(X)
    pg.experts_gated_bf16_backward(R, F, K, E, offsets, X, Wg, Wu, "silu", H, dX2, None, None)
    for e, a in ((0, 0), (0, 29980), (1, 30011), (1, R - 30)):
        at = torch.arange(a, a + 30, device="cuda")
        h, bound, g, u, eg, eu, _, _ = ref.gated(X[at], Wg[e], Wu[e], "silu")
        ref.check(H[at], h, bound, "H")
        ref.check(Z[0, at], g, eg, "G")
        ref.check(Z[1, at], u, eu, "U")
        want = ref.gated_backward(X[at], Wg[e], Wu[e], "silu", H[at])
        ref.check(dX[at], *want["dX"], "dX kept")
        ref.check(dX2[at], *want["dX"], "dX")


@pytest.mark.parametrize("R,N", [(LAST, 8), (3, LAST)])
def test_experts_largest_extents(R, N):
    K, E = 8, 2
    first = R // 2 + 1
    offsets = groups([first, R - first])
    X, W = rnd(16, R, K), rnd(17, E, K, N, std=0.3) if N < 100 else rnd(17, 1, K, N).expand(E, K, N)
    W = W.contiguous() if N < 100 else W
    if N >= 100:
        # (one matrix for both experts would be 68 GB with a copy: one expert then)
        E, offsets, W = 1, groups([R]), W[:1].contiguous()
    Y = torch.empty(R, N, device="cuda", dtype=BF16)
    pg.experts_linear_bf16(R, N, K, E, offsets, X, W, Y)
    if N < 100:
        for e, a in ((0, 0), (0, first - 30), (1, first), (1, R - 30)):
            at = torch.arange(a, a + 30, device="cuda")
            y, bound, _, _ = ref.linear(X[at], W[e], None, "none", None)
            ref.check(Y[at], y, bound, "Y")
        dX = torch.empty_like(X)
        pg.experts_linear_bf16_backward(R, N, K, E, offsets, None, W, Y, dX, None)
        at = some(R)
        e = (at >= first).long()
        # each row against its own expert's matrix
        for i in (0, 1):
            rows = at[e == i]
            want = ref.linear_backward(X[rows], W[i], None, "none", Y[rows])
            ref.check(dX[rows], *want["dX"], "dX")
    else:
        cols = some(N)
        y, bound, _, _ = ref.linear(X, W[0][:, cols], None, "none", None)
        ref.check(Y[:, cols], y, bound, "Y")
