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
