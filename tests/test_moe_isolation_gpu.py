"""What one expert's group holds stays with it, and offsets that no sort makes keep to the
rows and to the outputs, in each of the experts' products: linear and gated, forward and
gradients, from kept products and without, on single CTAs and on pairs.  And the norm's
gradients with several wide rows a block."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe_reference as moe  # noqa: E402
import operator_reference as ref  # noqa: E402
import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NAN, INF = float("nan"), float("inf")
PAD = 64
# N (or F) and K: tiles of single CTAs; of pairs, with rows that TMA reads and without
SIZES = [(136, 200), (1032, 2056), (1030, 2055)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from software_pipelined_tiled_loop_gb300 import build
    build.build()
    pg.lib()
    yield
    assert pg.pgemm_get_device_status() == 0


def rnd(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


class Out:
    """Outputs of NaNs within larger buffers of sevens."""

    def __init__(self):
        self.all = []

    def new(self, *shape, dtype=BF16):
        n = 1
        for d in shape:
            n *= d
        whole = torch.full((n + 2 * PAD,), 7.0, device="cuda", dtype=dtype)
        whole[PAD:PAD + n] = NAN
        self.all.append(whole)
        return whole[PAD:PAD + n].view(shape)

    def check(self):
        torch.cuda.synchronize()
        for whole in self.all:
            assert (whole[:PAD] == 7).all() and (whole[-PAD:] == 7).all()
        assert pg.pgemm_get_device_status() == 0


class Problem:
    """Operands, and a run through every product: rows' outputs and weights' by name."""

    def __init__(self, R, N, K, E):
        self.sizes = R, N, K, E
        self.X, self.dY = rnd(1, R, K), rnd(2, R, N)
        self.W = [rnd(3 + i, E, K, N, std=K ** -0.5) for i in range(2)]

    def run(self, offsets):
        R, N, K, E = self.sizes
        X, dY, (W, U), o = self.X, self.dY, self.W, Out()
        rows, weights = {}, {}
        rows["Y"] = o.new(R, N)
        pg.experts_linear_bf16(R, N, K, E, offsets, X, W, rows["Y"])
        rows["dX"], weights["dW"] = o.new(R, K), o.new(E, K, N)
        pg.experts_linear_bf16_backward(R, N, K, E, offsets, X, W, dY, rows["dX"], weights["dW"])
        rows["H"], Z = o.new(R, N), o.new(2, R, N, dtype=F32)
        pg.experts_gated_bf16(R, N, K, E, offsets, X, W, U, "silu", rows["H"], preact=Z)
        rows["G"], rows["U"] = Z
        for name, kept in (("kept", Z), ("again", None)):
            rows[f"dX {name}"] = o.new(R, K)
            dWg, dWu = o.new(E, K, N), o.new(E, K, N)
            pg.experts_gated_bf16_backward(R, N, K, E, offsets, X, W, U, "silu", dY,
                                           rows[f"dX {name}"], dWg, dWu, preact=kept)
            weights[f"dWg {name}"], weights[f"dWu {name}"] = dWg, dWu
        o.check()
        return rows, weights


@pytest.mark.parametrize("N,K", SIZES)
def test_what_is_not_finite_stays_with_its_expert(N, K):
    sizes = [53, 70, 200, 45]
    offsets = torch.tensor([0] + sizes, device="cuda").cumsum(0).int()
    p, bad = Problem(sum(sizes), N, K, len(sizes)), 1
    a, b = int(offsets[bad]), int(offsets[bad + 1])
    rows, weights = p.run(offsets)
    p.X[a:b], p.dY[a:b] = NAN, INF
    for w in p.W:
        w[bad] = NAN
    rows2, weights2 = p.run(offsets)
    for name, was in rows.items():
        got = rows2[name]
        assert torch.isfinite(was).all(), name
        assert torch.equal(got[:a], was[:a]) and torch.equal(got[b:], was[b:]), name
        assert got[a:b].isnan().all(), name
    for name, was in weights.items():
        got = weights2[name]
        assert torch.isfinite(was).all(), name
        assert torch.equal(got[:bad], was[:bad]) and torch.equal(got[bad + 1:], was[bad + 1:]), name
        assert got[bad].isnan().all(), name


@pytest.mark.parametrize("N,K", SIZES)
def test_offsets_beyond_the_rows_end_with_them(N, K):
    R = 380
    p = Problem(R, N, K, 4)
    good = torch.tensor([0, 0, 190, R, R], device="cuda", dtype=I32)
    wild = torch.tensor([-5, -1, 190, 2 ** 31 - 1, 99], device="cuda", dtype=I32)
    for x, y in zip(p.run(good), p.run(wild)):
        for name in x:
            assert torch.equal(x[name], y[name]), name


@pytest.mark.parametrize("N,K", SIZES)
def test_offsets_that_decrease_stay_within_the_rows(N, K):
    """Expert 1 has no rows; 0 and 2 share some, whose outputs may be either's."""
    R = 380
    p = Problem(R, N, K, 4)
    offsets = torch.tensor([0, 200, 61, 300, R], device="cuda", dtype=I32)
    rows, weights = p.run(offsets)
    spans = {0: (0, 200), 2: (61, 300), 3: (300, R)}
    for e, (a, b) in {0: (0, 61), 2: (200, 300), 3: (300, R)}.items():
        for name, pair in (("Y", moe.experts_linear(torch.tensor([0, b - a]), p.X[a:b],
                                                    p.W[0][e:e + 1])["Y"]),
                           *((n, moe.experts_gated(torch.tensor([0, b - a]), p.X[a:b],
                                                   p.W[0][e:e + 1], p.W[1][e:e + 1],
                                                   "silu")[n]) for n in "HGU")):
            ref.check(rows[name][a:b], *pair, name)
        one = torch.tensor([0, b - a])
        want = moe.experts_linear_backward(one, p.X[a:b], p.W[0][e:e + 1], p.dY[a:b])
        ref.check(rows["dX"][a:b], *want["dX"], "dX")
        want = moe.experts_gated_backward(one, p.X[a:b], p.W[0][e:e + 1], p.W[1][e:e + 1], "silu",
                                          p.dY[a:b])
        for name in ("dX kept", "dX again"):
            ref.check(rows[name][a:b], *want["dX"], name)
    for e, (a, b) in spans.items():
        want = moe.experts_linear_backward(torch.tensor([0, b - a]), p.X[a:b], p.W[0][e:e + 1],
                                           p.dY[a:b])
        ref.check(weights["dW"][e:e + 1], *want["dW0"], "dW")
    for name, got in weights.items():
        assert (got[1] == 0).all() and torch.isfinite(got).all(), name
    for name, got in rows.items():
        assert torch.isfinite(got).all(), name
    # every expert with all rows, or none
    p.run(torch.tensor([R, 0, R, -9, 2 ** 31 - 1], device="cuda", dtype=I32))


@pytest.mark.parametrize("T,D", [(330, 9000), (700, 12288), (330, 16384), (330, 16376)])
def test_norm_backward_of_several_wide_rows_a_block(T, D):
    S, gain, dY, dS = rnd(11, T, D, std=2.0), rnd(12, D), rnd(13, T, D), rnd(14, T, D)
    S[1] = 0
    for g, ds in ((gain, dS), (None, None)):
        want = moe.norm_backward(S, g, 1e-6, dY, ds)
        o = Out()
        dX, dg, dX2, dg2 = o.new(T, D), o.new(D), o.new(T, D), o.new(D)
        pg.rmsnorm_bf16_backward(T, D, S, g, 1e-6, dY, ds, dX, dg)
        pg.rmsnorm_bf16_backward(T, D, S, g, 1e-6, dY, ds, dX2, None)
        pg.rmsnorm_bf16_backward(T, D, S, g, 1e-6, dY, ds, None, dg2)
        o.check()
        ref.check(dX, *want["dX"], "dX")
        ref.check(dg, *want["dgain"], "dgain")
        assert torch.equal(dX, dX2) and torch.equal(dg, dg2)
