"""How many columns the experts' products sum over at most: more are refused on the host,
before a GPU is touched.  A call whose last checked operand is misaligned shows that the
checks before that one passed."""
import pytest

import software_pipelined_tiled_loop_gb300 as pg
from software_pipelined_tiled_loop_gb300 import build as pgbuild

MISALIGNED, LARGE = 2, 7
G = 1 << 20  # an aligned address that is never dereferenced
MOST = 1 << 19
SILU = pg.ACTIVATIONS["silu"]


@pytest.fixture(scope="module")
def L():
    pgbuild.build()
    return pg.lib()


def test_linear(L):
    def forward(K, N=8):
        return L.experts_linear_bf16(40, N, K, 1, G, G, G, G + 2, None)
    assert forward(MOST) == MISALIGNED and forward(MOST + 1) == LARGE
    assert forward(2 ** 31 - 1) == LARGE and forward(8, N=2 ** 31 - 1) == MISALIGNED

    def backward(N, K=8, dX=G, dW=G + 2):
        return L.experts_linear_bf16_backward(40, N, K, 1, G, G, G, G, dX, dW, None)
    assert backward(MOST) == MISALIGNED and backward(MOST + 1) == LARGE
    assert backward(MOST + 1, dX=G + 2, dW=None) == LARGE
    # dW sums over rows
    assert backward(MOST + 1, dX=None) == MISALIGNED and backward(8, K=MOST + 1) == MISALIGNED


def test_gated(L):
    def forward(K, F=8):
        return L.experts_gated_bf16(40, F, K, 1, G, G, G, G, SILU, G + 2, None, None)
    assert forward(MOST) == MISALIGNED and forward(MOST + 1) == LARGE
    assert forward(8, F=2 ** 31 - 1) == MISALIGNED

    def backward(F, K=8, preact=G, dX=G, dWg=G, dWu=G + 2):
        return L.experts_gated_bf16_backward(40, F, K, 1, G, G, G, G, SILU, G, preact, dX, dWg, dWu,
                                             None)
    # dX sums over both products' columns
    assert backward(MOST // 2) == MISALIGNED and backward(MOST // 2 + 1) == LARGE
    assert backward(MOST // 2 + 1, dX=None) == MISALIGNED
    # products computed again
    assert backward(8, K=MOST, preact=None) == MISALIGNED
    assert backward(8, K=MOST + 1, preact=None) == LARGE
    assert backward(8, K=MOST + 1) == MISALIGNED
