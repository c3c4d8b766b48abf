"""The operators' argument checks, made on the host before a GPU is touched,
and the binding's own."""
import pytest

import software_pipelined_tiled_loop_gb300 as pg
from software_pipelined_tiled_loop_gb300 import build as pgbuild

OK, INVALID, MISALIGNED = 0, 1, 2
G = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    pgbuild.build()
    return pg.lib()


def test_linear_refusals(L):
    f = L.linear_bf16
    for dims in ((-1, 4, 4), (4, -1, 4), (4, 4, -1)):
        assert f(*dims, G, G, None, 0, None, G, None, None) == INVALID
    for act in (-1, 5):
        assert f(4, 4, 4, G, G, None, act, None, G, None, None) == INVALID
    assert f(0, 4, 4, None, None, None, 0, None, None, None, None) == OK
    assert f(4, 0, 4, None, None, None, 0, None, None, None, None) == OK
    assert f(4, 4, 4, None, G, None, 0, None, G, None, None) == INVALID
    assert f(4, 4, 4, G, None, None, 0, None, G, None, None) == INVALID
    assert f(4, 4, 4, G, G, None, 0, None, None, None, None) == INVALID
    good = [G, G, G, 1, G, G, G]  # X, W, bias, act, residual, Y, preact
    for i in (0, 1, 2, 4, 5, 6):
        bad = list(good)
        bad[i] = G + 8
        assert f(4, 4, 4, *bad, None) == MISALIGNED


def test_linear_backward_refusals(L):
    f = L.linear_bf16_backward

    def call(M=4, N=4, K=4, X=G, W=G, bias=None, act=1, dY=G, pre=None, dX=G, dW=G, db=G):
        return f(M, N, K, X, W, bias, act, dY, pre, dX, dW, db, None)

    for kw in ({"M": -1}, {"N": -1}, {"K": -1}, {"act": 9}, {"dY": None}, {"X": None},
               {"W": None}, {"W": None, "dX": None}, {"X": None, "dW": None}):
        assert call(**kw) == INVALID, kw
    assert call(dX=None, dW=None, db=None) == OK
    assert call(M=0, dW=None, db=None) == OK
    for name in ("X", "W", "bias", "dY", "pre", "dX", "dW", "db"):
        assert call(**{name: G + 2}) == MISALIGNED, name


def test_gated_refusals(L):
    f = L.gated_bf16
    for dims in ((-1, 4, 4), (4, -1, 4), (4, 4, -1)):
        assert f(*dims, G, G, G, 4, G, None, None) == INVALID
    assert f(4, 4, 4, G, G, G, 7, G, None, None) == INVALID
    assert f(0, 4, 4, None, None, None, 4, None, None, None) == OK
    for i in range(3):
        ops = [G, G, G]
        ops[i] = None
        assert f(4, 4, 4, *ops, 4, G, None, None) == INVALID
        ops[i] = G + 4
        assert f(4, 4, 4, *ops, 4, G, None, None) == MISALIGNED
    assert f(4, 4, 4, G, G, G, 4, None, None, None) == INVALID
    assert f(4, 4, 4, G, G, G, 4, G + 8, None, None) == MISALIGNED
    assert f(4, 4, 4, G, G, G, 4, G, G + 8, None) == MISALIGNED


def test_gated_backward_refusals(L):
    f = L.gated_bf16_backward

    def call(M=4, F=4, K=4, X=G, Wg=G, Wu=G, act=4, dH=G, pre=None, dX=G, dWg=G, dWu=G):
        return f(M, F, K, X, Wg, Wu, act, dH, pre, dX, dWg, dWu, None)

    for kw in ({"M": -1}, {"F": -1}, {"K": -1}, {"act": -1}, {"dH": None}, {"X": None},
               {"Wg": None}, {"Wu": None}, {"dWg": None}, {"dWu": None}):
        assert call(**kw) == INVALID, kw
    assert call(dX=None, dWg=None, dWu=None) == OK
    for name in ("X", "Wg", "Wu", "dH", "pre", "dX", "dWg", "dWu"):
        assert call(**{name: G + 2}) == MISALIGNED, name


def test_xent_refusals(L):
    def call(T=4, V=9, D=8, X=G, W=G, y=G, dl=G, loss=G, lse=G, dX=G, dW=G, ws=0):
        return L.xent_bf16_grad(T, V, D, X, W, y, dl, loss, lse, dX, dW, ws, None)

    for kw in ({"T": -1}, {"V": 0}, {"V": -1}, {"D": -1}, {"ws": -1}, {"X": None}, {"W": None},
               {"y": None}):
        assert call(**kw) == INVALID, kw
    assert call(T=0, dW=None) == OK
    for name in ("X", "W", "y", "dl", "loss", "lse", "dX", "dW"):
        assert call(**{name: G + 4}) == MISALIGNED, name
    f = L.xent_bf16
    assert f(4, 0, 8, G, G, G, G, G, None) == INVALID
    assert f(4, 9, 8, G, G, None, G, G, None) == INVALID
    assert f(4, 9, 8, G, G, G, G + 4, G, None) == MISALIGNED
    assert f(0, 9, 8, None, None, None, None, None, None) == OK


class FakeTensor:
    """What the binding looks at, without a GPU."""
    is_cuda = True

    def __init__(self, numel, itemsize=2, contiguous=True):
        self.n, self.size, self.c = numel, itemsize, contiguous

    def is_contiguous(self):
        return self.c

    def data_ptr(self):
        return G

    def numel(self):
        return self.n

    def element_size(self):
        return self.size


def test_binding_checks_operands(L):
    ok = FakeTensor(16)
    for bad in (FakeTensor(15), FakeTensor(16, 4), FakeTensor(16, contiguous=False)):
        with pytest.raises(ValueError):
            pg.linear_bf16(4, 4, 4, bad, ok, None, "none", None, ok)
        with pytest.raises(ValueError):
            pg.gated_bf16(4, 4, 4, ok, ok, bad, "silu", ok)
    with pytest.raises(ValueError):  # int32 token ids
        pg.xent_bf16(4, 4, 4, ok, ok, FakeTensor(4, 4), None, None)
    with pytest.raises(ValueError):
        pg.linear_bf16(4, 4, 4, ok, ok, None, "swish", None, ok)
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        pg.linear_bf16(4, 4, 4, torch.zeros(16, dtype=torch.bfloat16), ok, None, "none", None, ok)


def test_activation_names_match_the_header(L):
    import os
    import re
    header = open(os.path.join(os.path.dirname(pgbuild.INCLUDE), "include", "pgemm.h")).read()
    found = {n.lower(): int(v) for n, v in re.findall(r"PGEMM_ACT_(\w+) = (\d+)", header)}
    assert found == pg.ACTIVATIONS


def test_binding_refuses_sizes_beyond_32_bits(L):
    # ctypes would pass their low 32 bits on
    big = 1 << 32
    for call in (lambda: pg.linear_bf16(big + 4, 4, 4, G, G, None, "none", None, G),
                 lambda: pg.linear_bf16_backward(4, big, 4, G, G, None, "silu", G, G, G, None),
                 lambda: pg.gated_bf16(4, 4, 1 << 31, G, G, G, "silu", G),
                 lambda: pg.gated_bf16_backward(big + 1, 4, 4, G, G, G, "silu", G, G, G, G),
                 lambda: pg.xent_bf16(4, big + 4, 4, G, G, G, G, G),
                 lambda: pg.xent_bf16_grad(4, 4, big + 4, G, G, G, None, G, G, G, G)):
        with pytest.raises(ValueError, match="sizes are at most"):
            call()
