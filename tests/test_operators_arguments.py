"""Further argument checks of the operators, made on the host before a GPU is
touched.  A call whose last operand is misaligned shows that the checks before that
one passed."""
import pytest

import software_pipelined_tiled_loop_gb300 as pg
from software_pipelined_tiled_loop_gb300 import build as pgbuild

INVALID, MISALIGNED = 1, 2
G = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    pgbuild.build()
    return pg.lib()


def test_gated_backward_asks_only_for_what_it_reads(L):
    def call(X=G, Wg=G, Wu=G, pre=G, dX=G, dWg=G, dWu=G):
        return L.gated_bf16_backward(200, 261, 77, X, Wg, Wu, 4, G + 2, pre, dX, dWg, dWu, None)

    assert call(X=None, dWg=None, dWu=None) == MISALIGNED
    assert call(Wg=None, Wu=None, dX=None) == MISALIGNED
    for kw in ({"X": None}, {"Wg": None}, {"Wu": None},
               {"X": None, "dWg": None, "dWu": None, "pre": None},
               {"Wg": None, "Wu": None, "dX": None, "pre": None},
               {"Wu": None, "dWg": None, "dWu": None}, {"X": None, "dX": None}):
        assert call(**kw) == INVALID, kw


def test_linear_backward_asks_only_for_what_it_reads(L):
    def call(X=G, W=G, pre=G, dX=G, dW=G, db=G):
        return L.linear_bf16_backward(200, 261, 77, X, W, None, 4, G + 2, pre, dX, dW, db, None)

    assert call(X=None, dW=None) == MISALIGNED
    assert call(W=None, dX=None) == MISALIGNED
    assert call(X=None, W=None, dX=None, dW=None) == MISALIGNED
    for kw in ({"X": None}, {"W": None}, {"X": None, "dW": None, "pre": None},
               {"W": None, "dX": None, "pre": None}):
        assert call(**kw) == INVALID, kw
