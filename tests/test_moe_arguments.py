"""What the operators of a mixture-of-experts block refuse, on the host before a GPU is
touched.  A call whose last checked operand is misaligned shows that the checks before that
one passed."""
import pytest

import software_pipelined_tiled_loop_gb300 as pg
from software_pipelined_tiled_loop_gb300 import build as pgbuild

OK, INVALID, MISALIGNED, LARGE = 0, 1, 2, 7
G = 1 << 20  # an aligned address that is never dereferenced
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    pgbuild.build()
    return pg.lib()


def table(call, rows):
    """rows: (expected status, changed arguments)."""
    for want, kw in rows:
        assert call(**kw) == want, (want, kw)


def test_rmsnorm(L):
    for fn, last in ((L.rmsnorm_bf16, ()), (L.rmsnorm_i8, (G,))):
        def call(T=4, D=8, X=G, R=G, g=G, eps=1e-6, S=G, Y=G + 2):
            return fn(T, D, X, R, g, eps, S, Y, *last, None)
        table(call, [
            (MISALIGNED, {}), (MISALIGNED, {"R": None, "g": None, "S": None}),
            (MISALIGNED, {"Y": G, "X": G + 2}), (MISALIGNED, {"Y": G, "S": G + 8}),
            (MISALIGNED, {"eps": 0.0}),
            (INVALID, {"X": None}), (INVALID, {"Y": None}), (INVALID, {"T": -1}),
            (INVALID, {"D": -1}), (INVALID, {"eps": -1e-9}), (INVALID, {"eps": float("nan")}),
            (LARGE, {"D": 32769}), (MISALIGNED, {"D": 32768}),
            (OK, {"T": 0, "X": None, "Y": None}), (OK, {"D": 0, "X": None, "Y": None})])
    assert L.rmsnorm_i8(4, 8, G, G, G, 1e-6, G, G, None, None) == INVALID
    assert L.rmsnorm_i8(4, 8, G, G, G, 1e-6, G, G, G + 4, None) == MISALIGNED


def test_rmsnorm_backward(L):
    def call(T=4, D=8, S=G, g=G, eps=1e-6, dY=G, dS=G, dX=G, dg=G + 2):
        return L.rmsnorm_bf16_backward(T, D, S, g, eps, dY, dS, dX, dg, None)
    table(call, [
        (MISALIGNED, {}), (MISALIGNED, {"g": None, "dS": None, "dX": None}),
        (INVALID, {"S": None}), (INVALID, {"dY": None}), (INVALID, {"T": -1}),
        (INVALID, {"eps": -1.0}), (LARGE, {"D": BIG}),
        (OK, {"dX": None, "dg": None}), (OK, {"T": 0, "dg": None}), (OK, {"D": 0}),
        (MISALIGNED, {"T": 0, "S": None, "dY": None})])


def test_route(L):
    def call(T=4, E=8, k=2, z=G, e=G, w=G + 4):
        return L.route_topk(T, E, k, z, 1, e, w, None)
    sizes = [(INVALID, {"T": -1}), (INVALID, {"E": 0}), (INVALID, {"k": 0}), (INVALID, {"k": 9}),
             (LARGE, {"E": 1025}), (LARGE, {"E": 64, "k": 33}), (MISALIGNED, {"E": 1024, "k": 32}),
             (OK, {"T": 0}), (INVALID, {"z": None}), (INVALID, {"e": None}), (INVALID, {"w": None}),
             (MISALIGNED, {})]
    table(call, sizes)

    def back(T=4, E=8, k=2, z=G, e=G, w=G, d=G + 4):
        return L.route_topk_backward(T, E, k, z, 0, e, w, d, None)
    table(back, sizes + [(INVALID, {"d": None}), (MISALIGNED, {"d": G, "e": G + 4})])


def test_sort_gather_combine(L):
    def sort(T=4, E=8, k=2, x=G, o=G, r=G + 4):
        return L.expert_sort(T, E, k, x, o, r, None)
    table(sort, [
        (MISALIGNED, {}), (INVALID, {"T": -1}), (INVALID, {"E": 0}), (INVALID, {"k": 0}),
        (LARGE, {"E": 1025}), (LARGE, {"T": 1 << 30}), (MISALIGNED, {"T": (1 << 30) - 1}),
        (INVALID, {"x": None}), (INVALID, {"o": None}), (INVALID, {"r": None}),
        (INVALID, {"T": 0, "o": None})])

    def gather(T=4, k=2, D=8, X=G, r=G, Xs=G + 2):
        return L.expert_gather_bf16(T, k, D, X, r, Xs, None)
    sizes = [(INVALID, {"T": -1}), (INVALID, {"k": 0}), (INVALID, {"D": -1}), (LARGE, {"T": 1 << 30}),
             (INVALID, {"r": None}), (MISALIGNED, {})]
    table(gather, sizes + [(INVALID, {"X": None}), (INVALID, {"Xs": None}), (OK, {"T": 0}),
                           (OK, {"D": 0})])

    def combine(T=4, k=2, D=8, Ys=G, r=G, w=G, res=G, Y=G + 2):
        return L.expert_combine_bf16(T, k, D, Ys, r, w, res, Y, None)
    table(combine, sizes + [(INVALID, {"Ys": None}), (INVALID, {"Y": None}), (OK, {"T": 0}),
                            (OK, {"D": 0}), (MISALIGNED, {"w": None, "res": None})])

    def back(T=4, k=2, D=8, Ys=G, r=G, w=G, dY=G, dYs=G, dw=G + 4):
        return L.expert_combine_bf16_backward(T, k, D, Ys, r, w, dY, dYs, dw, None)
    table(back, sizes + [(INVALID, {"Ys": None}), (INVALID, {"dY": None}), (OK, {"T": 0}),
                         (OK, {"dYs": None, "dw": None}), (MISALIGNED, {"dYs": None, "w": None}),
                         (MISALIGNED, {"dw": None, "Ys": None, "dYs": G + 2})])


def test_experts_linear(L):
    def call(R=40, N=8, K=16, E=4, o=G, X=G, W=G, Y=G + 2):
        return L.experts_linear_bf16(R, N, K, E, o, X, W, Y, None)
    sizes = [(INVALID, {"R": -1}), (INVALID, {"N": -1}), (INVALID, {"K": -1}), (INVALID, {"E": 0}),
             (LARGE, {"E": 1025}), (LARGE, {"E": 1024, "K": 1 << 21}), (INVALID, {"o": None}),
             (MISALIGNED, {})]
    table(call, sizes + [(INVALID, {"X": None}), (INVALID, {"W": None}), (INVALID, {"Y": None}),
                         (OK, {"R": 0}), (OK, {"N": 0}), (MISALIGNED, {"K": 0, "X": None, "W": None})])

    def back(R=40, N=8, K=16, E=4, o=G, X=G, W=G, dY=G, dX=G, dW=G + 2):
        return L.experts_linear_bf16_backward(R, N, K, E, o, X, W, dY, dX, dW, None)
    table(back, sizes + [
        (INVALID, {"X": None}), (INVALID, {"W": None}), (INVALID, {"dY": None}),
        (MISALIGNED, {"X": None, "dW": None, "dX": G + 2}), (MISALIGNED, {"W": None, "dX": None}),
        (OK, {"dX": None, "dW": None}), (OK, {"R": 0, "dW": None}), (OK, {"K": 0}),
        (INVALID, {"dX": None, "X": None}), (INVALID, {"dW": None, "W": None, "dX": G + 2})])


def test_experts_gated(L):
    def call(R=40, F=8, K=16, E=4, o=G, X=G, Wg=G, Wu=G, act=4, H=G + 2, z=G):
        return L.experts_gated_bf16(R, F, K, E, o, X, Wg, Wu, act, H, z, None)
    sizes = [(INVALID, {"R": -1}), (INVALID, {"F": -1}), (INVALID, {"K": -1}), (INVALID, {"E": -3}),
             (LARGE, {"E": 1025}), (LARGE, {"E": 2, "K": 1 << 30}), (INVALID, {"o": None}),
             (INVALID, {"act": 5}), (INVALID, {"act": -1}), (INVALID, {"act": 1}),  # (relu)
             (MISALIGNED, {"act": 0}), (MISALIGNED, {})]
    table(call, sizes + [(INVALID, {"X": None}), (INVALID, {"Wg": None}), (INVALID, {"Wu": None}),
                         (INVALID, {"H": None}), (MISALIGNED, {"z": None}),
                         (MISALIGNED, {"H": G, "z": G + 8}), (OK, {"R": 0}), (OK, {"F": 0})])

    def back(R=40, F=8, K=16, E=4, o=G, X=G, Wg=G, Wu=G, act=4, dH=G, z=G, dX=G, dWg=G, dWu=G + 2):
        return L.experts_gated_bf16_backward(R, F, K, E, o, X, Wg, Wu, act, dH, z, dX, dWg, dWu, None)
    no_w = {"dWg": None, "dWu": None}
    table(back, sizes + [
        (INVALID, {"dWg": None}), (INVALID, {"dWu": None}), (INVALID, {"dH": None}),
        (INVALID, {"X": None}), (INVALID, {"Wg": None}), (INVALID, {"Wu": None}),
        (MISALIGNED, {"X": None, "dX": G + 2, **no_w}),
        (INVALID, {"X": None, "dX": G + 2, "z": None, **no_w}),
        (MISALIGNED, {"Wg": None, "Wu": None, "dX": None}),
        (INVALID, {"Wg": None, "Wu": None, "dX": None, "z": None}),
        (OK, {"dX": None, **no_w}), (OK, {"K": 0}), (OK, {"R": 0, **no_w})])


class Fake:
    """A contiguous CUDA tensor as the binding looks at it."""
    is_cuda = True

    def __init__(self, dtype, numel):
        self.dtype, self.n = dtype, numel

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return G

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize


def test_binding_checks_types_and_counts(L):
    torch = pytest.importorskip("torch")
    b, f, i, q = (Fake(t, 512) for t in (torch.bfloat16, torch.float32, torch.int32, torch.int8))
    half, i64, short = Fake(torch.float16, 512), Fake(torch.int64, 512), Fake(torch.bfloat16, 31)
    few = Fake(torch.int32, 4)
    wrong_type = (
        ("X", lambda: pg.rmsnorm_bf16(4, 8, half, b, b, 1e-6, b, b)),
        ("gain", lambda: pg.rmsnorm_bf16(4, 8, b, b, f, 1e-6, b, b)),
        ("Q", lambda: pg.rmsnorm_i8(4, 8, b, b, b, 1e-6, b, b, f)),
        ("scale", lambda: pg.rmsnorm_i8(4, 8, b, b, b, 1e-6, b, q, b)),
        ("dS", lambda: pg.rmsnorm_bf16_backward(4, 8, b, b, 1e-6, b, f, b, b)),
        ("logits", lambda: pg.route_topk(4, 8, 2, b, True, i, f)),
        ("experts", lambda: pg.route_topk(4, 8, 2, f, True, i64, f)),
        ("dlogits", lambda: pg.route_topk_backward(4, 8, 2, f, True, i, f, b)),
        ("offsets", lambda: pg.expert_sort(4, 8, 2, i, i64, i)),
        ("slot_row", lambda: pg.expert_gather_bf16(4, 2, 8, b, i64, b)),
        ("weights", lambda: pg.expert_combine_bf16(4, 2, 8, b, i, b, b, b)),
        ("dweights", lambda: pg.expert_combine_bf16_backward(4, 2, 8, b, i, f, b, b, b)),
        ("offsets", lambda: pg.experts_linear_bf16(4, 8, 8, 2, i64, b, b, b)),
        ("dW", lambda: pg.experts_linear_bf16_backward(4, 8, 8, 2, i, b, b, b, b, f)),
        ("Wu", lambda: pg.experts_gated_bf16(4, 8, 8, 2, i, b, b, f, "silu", b)),
        ("preact", lambda: pg.experts_gated_bf16_backward(4, 8, 8, 2, i, b, b, b, "silu", b, b, b,
                                                          b, preact=b)))
    for name, call in wrong_type:
        with pytest.raises(ValueError, match=f"^{name}: elements of"):
            call()
    too_few = (
        ("Y", lambda: pg.rmsnorm_bf16(4, 8, b, b, b, 1e-6, b, short)),
        ("experts", lambda: pg.route_topk(4, 8, 2, f, True, few, f)),
        ("offsets", lambda: pg.expert_sort(2, 4, 1, i, few, i)),
        ("Xs", lambda: pg.expert_gather_bf16(2, 2, 8, b, i, short)),
        ("Ys", lambda: pg.expert_combine_bf16(2, 2, 8, short, i, f, b, b)),
        ("offsets", lambda: pg.experts_linear_bf16(4, 8, 8, 4, few, b, b, b)),
        ("X", lambda: pg.experts_linear_bf16(4, 8, 8, 2, i, short, b, b)),
        ("W", lambda: pg.experts_linear_bf16(2, 8, 8, 9, i, b, b, b)),
        ("preact", lambda: pg.experts_gated_bf16(4, 65, 1, 1, i, b, b, b, "silu", b, preact=f)))
    for name, call in too_few:
        with pytest.raises(ValueError, match=f"^{name}: \\d+ elements, at least"):
            call()
    with pytest.raises(ValueError, match="unknown activation"):
        pg.experts_gated_bf16(4, 8, 8, 2, i, b, b, b, "swish", b)
    with pytest.raises(pg.PgemmError, match="INVALID_VALUE"):
        pg.experts_gated_bf16(4, 8, 8, 2, i, b, b, b, "relu", b)


def test_binding_refuses_sizes_beyond_32_bits(L):
    over = 1 << 32
    for call in (lambda: pg.rmsnorm_bf16(over, 8, G, G, G, 1e-6, G, G),
                 lambda: pg.rmsnorm_i8(4, over, G, G, G, 1e-6, G, G, G),
                 lambda: pg.rmsnorm_bf16_backward(-over, 8, G, G, 1e-6, G, G, G, G),
                 lambda: pg.route_topk(over + 1, 8, 2, G, True, G, G),
                 lambda: pg.route_topk_backward(4, 8, over + 2, G, True, G, G, G),
                 lambda: pg.expert_sort(4, over + 8, 2, G, G, G),
                 lambda: pg.expert_gather_bf16(4, 2, over, G, G, G),
                 lambda: pg.expert_combine_bf16(over, 2, 8, G, G, G, G, G),
                 lambda: pg.expert_combine_bf16_backward(4, over + 2, 8, G, G, G, G, G, G),
                 lambda: pg.experts_linear_bf16(over, 8, 8, 2, G, G, G, G),
                 lambda: pg.experts_linear_bf16_backward(4, 8, 8, over + 2, G, G, G, G, G, G),
                 lambda: pg.experts_gated_bf16(4, over, 8, 2, G, G, G, G, "silu", G),
                 lambda: pg.experts_gated_bf16_backward(4, 8, over, 2, G, G, G, G, "silu", G, G, G,
                                                        G)):
        with pytest.raises(ValueError, match="sizes are at most"):
            call()
