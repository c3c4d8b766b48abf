"""Not a byte beyond the outputs of a mixture-of-experts block's operators is written, and
every one within: outputs are slices of larger buffers of a known pattern."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402

PAD = 64  # elements before and behind; outputs start on 16-byte boundaries
BF16, F32, I32, I8 = torch.bfloat16, torch.float32, torch.int32, torch.int8


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from software_pipelined_tiled_loop_gb300 import build
    build.build()
    pg.lib()
    yield
    assert pg.pgemm_get_device_status() == 0


class Guards:
    """Outputs full of a value that no right result has, in buffers of another."""

    def __init__(self):
        self.all = []

    def out(self, *shape, dtype=BF16, unset=float("nan")):
        n = 1
        for d in shape:
            n *= d
        if not dtype.is_floating_point:
            unset = -77
        buf = torch.full((n + 2 * PAD,), 7, device="cuda", dtype=dtype)
        buf[PAD:PAD + n] = unset
        self.all.append((buf, n, unset))
        return buf[PAD:PAD + n].view(shape)

    def check(self):
        torch.cuda.synchronize()
        for i, (buf, n, unset) in enumerate(self.all):
            assert (buf[:PAD] == 7).all(), f"output {i}: written before it"
            assert (buf[PAD + n:] == 7).all(), f"output {i}: written behind it"
            left = buf[PAD:PAD + n]
            left = left.isnan() if unset != unset else left == unset
            assert not left.any(), f"output {i}: elements left out"


def rnd(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


@pytest.mark.parametrize("T", [1, 7, 400])
@pytest.mark.parametrize("D", [1, 3, 8, 250, 511, 4104, 9001, 16385])
def test_norm(T, D):
    X, R, gain, dY = rnd(1, T, D), rnd(2, T, D), rnd(3, D), rnd(4, T, D)
    g = Guards()
    pg.rmsnorm_bf16(T, D, X, R, gain, 1e-6, g.out(T, D), g.out(T, D))
    Q = g.out(T, D, dtype=I8)
    Q.fill_(-128)  # (never a result)
    g.all[-1] = (*g.all[-1][:2], -128)
    pg.rmsnorm_i8(T, D, X, R, gain, 1e-6, g.out(T, D), Q, g.out(T, dtype=F32))
    pg.rmsnorm_bf16_backward(T, D, X, gain, 1e-6, dY, R, g.out(T, D), g.out(D))
    g.check()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 33, 5), (130, 64, 8), (77, 1000, 31)])
def test_route(T, E, k):
    z, dw = torch.randn(T, E, device="cuda"), torch.randn(T, k, device="cuda")
    g = Guards()
    for normalise in (True, False):
        experts = g.out(T, k, dtype=I32)
        pg.route_topk(T, E, k, z, normalise, experts, g.out(T, k, dtype=F32))
        pg.route_topk_backward(T, E, k, z, normalise, experts, dw, g.out(T, E, dtype=F32))
        rows = g.out(T, k, dtype=I32)
        pg.expert_sort(T, E, k, experts, g.out(E + 1, dtype=I32), rows)
    g.check()


@pytest.mark.parametrize("T,k", [(1, 1), (50, 3), (300, 9)])
@pytest.mark.parametrize("D", [1, 6, 40, 515, 2056])
def test_rows(T, k, D):
    rows = torch.randperm(T * k, device="cuda").int().view(T, k)
    X, Ys, w = rnd(5, T, D), rnd(6, T * k, D), torch.rand(T, k, device="cuda")
    g = Guards()
    pg.expert_gather_bf16(T, k, D, X, rows, g.out(T * k, D))
    pg.expert_combine_bf16(T, k, D, Ys, rows, w, X, g.out(T, D))
    pg.expert_combine_bf16_backward(T, k, D, Ys, rows, w, X, g.out(T * k, D), g.out(T, k, dtype=F32))
    g.check()


@pytest.mark.parametrize("sizes", [[1], [3, 0, 17, 16, 1], [33, 200, 0, 65, 300, 5]])
@pytest.mark.parametrize("N,K", [(8, 8), (1, 130), (132, 72), (133, 65), (264, 136), (261, 2056)])
def test_experts(N, K, sizes):
    E, R = len(sizes), sum(sizes)
    offsets = torch.tensor([0] + sizes, device="cuda").cumsum(0).int()
    X, W, W2 = rnd(7, R, K), rnd(8, E, K, N, std=K ** -0.5), rnd(9, E, K, N, std=K ** -0.5)
    dY = rnd(10, R, N)
    g = Guards()
    pg.experts_linear_bf16(R, N, K, E, offsets, X, W, g.out(R, N))
    pg.experts_linear_bf16_backward(R, N, K, E, offsets, X, W, dY, g.out(R, K), g.out(E, K, N))
    Z = g.out(2, R, N, dtype=F32)
    pg.experts_gated_bf16(R, N, K, E, offsets, X, W, W2, "silu", g.out(R, N), preact=Z)
    for kept in (Z, None):
        pg.experts_gated_bf16_backward(R, N, K, E, offsets, X, W, W2, "silu", dY, g.out(R, K),
                                       g.out(E, K, N), g.out(E, K, N), preact=kept)
    g.check()
