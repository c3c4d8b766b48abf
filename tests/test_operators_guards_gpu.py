"""Not a byte beyond an operator's outputs is written, and every one within: outputs are
slices of larger buffers of a known pattern.  Few rows by the streaming kernel (weights
at any pitch), one CTA's tiles and pairs, short reductions and ones split into parts or
shared by clusters, rows that TMA can and cannot describe."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402

PAD = 64  # elements before and behind; outputs start on 16-byte boundaries


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
    def __init__(self):
        self.all = []

    def out(self, *shape, dtype=torch.bfloat16):
        n = 1
        for d in shape:
            n *= d
        buf = torch.full((n + 2 * PAD,), 7.0, device="cuda", dtype=dtype)
        buf[PAD:PAD + n] = float("nan")
        self.all.append((buf, n))
        return buf[PAD:PAD + n].view(shape)

    def check(self):
        torch.cuda.synchronize()
        for i, (buf, n) in enumerate(self.all):
            assert (buf[:PAD] == 7).all(), f"output {i}: written before it"
            assert (buf[PAD + n:] == 7).all(), f"output {i}: written behind it"
            assert not buf[PAD:PAD + n].isnan().any(), f"output {i}: elements left out"


def rnd(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


SIZES = [(M, N, K) for M in (1, 17, 130) for N in (132, 133, 136, 261) for K in (72, 2050)]
SIZES += [(513, 1301, 136), (2500, 1301, 68), (2500, 1304, 70), (130, 5, 3), (3, 7, 8200)]


@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(M, N, K, act):
    X, W, b, R, dY = rnd(1, M, K), rnd(2, K, N, std=K ** -0.5), rnd(3, N), rnd(4, M, N), rnd(5, M, N)
    g = Guards()
    pg.linear_bf16(M, N, K, X, W, b, act, R, g.out(M, N))
    Z = g.out(M, N, dtype=torch.float32)
    pg.linear_bf16(M, N, K, X, W, b, act, None, g.out(M, N), preact=Z)
    for kept in (Z, None):
        pg.linear_bf16_backward(M, N, K, X, W, b, act, dY, g.out(M, K), g.out(K, N), g.out(N),
                                preact=kept)
    pg.linear_bf16_backward(M, N, K, X, W, b, "none", dY, g.out(M, K), g.out(K, N), g.out(N))
    g.check()


@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_gated(M, F, K, act):
    X, Wg, Wu = rnd(11, M, K), rnd(12, K, F, std=K ** -0.5), rnd(13, K, F, std=K ** -0.5)
    dH = rnd(14, M, F)
    g = Guards()
    pg.gated_bf16(M, F, K, X, Wg, Wu, act, g.out(M, F))
    Z = g.out(2, M, F, dtype=torch.float32)
    pg.gated_bf16(M, F, K, X, Wg, Wu, act, g.out(M, F), preact=Z)
    for kept in (Z, None):
        pg.gated_bf16_backward(M, F, K, X, Wg, Wu, act, dH, g.out(M, K), g.out(K, F), g.out(K, F),
                               preact=kept)
    g.check()


@pytest.mark.parametrize("workspace", [0, 1])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_xent(T, V, D, workspace):
    X, W, dl = rnd(21, T, D), rnd(22, V, D, std=2 * D ** -0.5), torch.rand(T, device="cuda")
    y = torch.randint(0, V, (T,), device="cuda")
    f32 = torch.float32
    g = Guards()
    pg.xent_bf16(T, V, D, X, W, y, g.out(T, dtype=f32), g.out(T, dtype=f32))
    for dloss in (dl, None):
        pg.xent_bf16_grad(T, V, D, X, W, y, dloss, g.out(T, dtype=f32), g.out(T, dtype=f32),
                          g.out(T, D), g.out(V, D), workspace_bytes=workspace)
    g.check()
