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


class FakeCuda:
    """A contiguous CUDA tensor as the binding looks at it."""
    is_cuda = True

    def __init__(self, dtype, numel=16):
        self.dtype, self.n = dtype, numel

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return G

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize


def test_binding_checks_element_types(L):
    torch = pytest.importorskip("torch")
    ok, short = FakeCuda(torch.bfloat16), FakeCuda(torch.bfloat16, 15)
    f16, i32, f64 = (FakeCuda(t) for t in (torch.float16, torch.int32, torch.float64))
    f32, i64 = FakeCuda(torch.float32, 32), FakeCuda(torch.int64)
    for bad, call in (
            ("X", lambda: pg.linear_bf16(4, 4, 4, f16, ok, None, "none", None, ok)),
            ("bias", lambda: pg.linear_bf16(4, 4, 4, ok, ok, f16, "none", None, ok)),
            ("preact", lambda: pg.linear_bf16(4, 4, 4, ok, ok, None, "relu", None, ok, preact=i32)),
            ("dY", lambda: pg.linear_bf16_backward(4, 4, 4, ok, ok, None, "relu", f16, ok, ok, ok)),
            ("Wu", lambda: pg.gated_bf16(4, 4, 4, ok, ok, f16, "silu", ok)),
            ("preact", lambda: pg.gated_bf16_backward(4, 4, 2, ok, ok, ok, "silu", ok, ok, ok, ok,
                                                      preact=FakeCuda(torch.int32, 32))),
            ("target", lambda: pg.xent_bf16(4, 4, 4, ok, ok, f64, f32, f32)),
            ("loss", lambda: pg.xent_bf16(4, 4, 4, ok, ok, i64, i32, f32)),
            ("dloss", lambda: pg.xent_bf16_grad(4, 4, 4, ok, ok, i64, i32, f32, f32, ok, ok)),
            ("dW", lambda: pg.xent_bf16_grad(4, 4, 4, ok, ok, i64, f32, f32, f32, ok, f16))):
        for _ in range(2):  # (the second call finds the right types met before)
            with pytest.raises(ValueError, match=f"^{bad}: elements of type"):
                call()
    # right types pass on to the next check; so do bf16 bit patterns as integers
    for t in (torch.bfloat16, torch.int16):
        with pytest.raises(ValueError, match="^W: 15 elements"):
            pg.linear_bf16(4, 4, 4, FakeCuda(t), short, None, "none", None, ok)


def test_binding_refuses_sizes_below_32_bits(L):
    # ctypes would pass their low 32 bits on: -(1 << 32) + 4 as 4
    low = -(1 << 32)
    for call in (lambda: pg.linear_bf16(low + 4, 4, 4, G, G, None, "none", None, G),
                 lambda: pg.linear_bf16_backward(4, low, 4, G, G, None, "silu", G, G, G, None),
                 lambda: pg.gated_bf16(4, 4, low + 8, G, G, G, "silu", G),
                 lambda: pg.gated_bf16_backward(low + 1, 4, 4, G, G, G, "silu", G, G, G, G),
                 lambda: pg.xent_bf16(4, low + 4, 4, G, G, G, G, G),
                 lambda: pg.xent_bf16_grad(4, 4, 3 * low + 4, G, G, G, None, G, G, G, G)):
        with pytest.raises(ValueError, match="sizes are at most"):
            call()
    for small in (-1, -(1 << 31)):  # what 32 bits hold is refused by the C function
        with pytest.raises(pg.PgemmError):
            pg.linear_bf16(small, 4, 4, G, G, None, "none", None, G)


def test_no_size_beyond_32_bits_reaches_the_library():
    # every mixture of sizes around the powers of two, against what ctypes would make of it
    import ctypes
    import itertools
    edge = [k * (1 << 31) + d for k in range(-4, 5) for d in (-1, 0, 1, 5)]
    for dims in itertools.product(edge, repeat=3):
        try:
            pg._sizes("f", dims[0] | dims[1] | dims[2])
        except ValueError:
            assert any(d != ctypes.c_int(d).value for d in dims), dims
        else:  # all pass unchanged, or the C function refuses one for being negative
            seen = [ctypes.c_int(d).value for d in dims]
            assert list(dims) == seen or min(seen) < 0, dims
