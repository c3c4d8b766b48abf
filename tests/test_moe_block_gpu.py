"""The operators of a mixture-of-experts block run together as a model runs them: norm,
router, sort, gather, experts, combine, and back; eager, captured into graphs whose routing
changes from replay to replay, on several streams and from several threads at once.  Each
operator's outputs are held to its definition for the inputs that it was given."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe_reference as moe  # noqa: E402
import operator_reference as ref  # noqa: E402
import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from software_pipelined_tiled_loop_gb300 import build
    build.build()
    pg.lib()
    yield
    assert pg.pgemm_get_device_status() == 0


class Block:
    """Weights, inputs and every buffer of one block, forward and backward."""

    def __init__(self, T, D, F, E, k, normalise, seed, kept=True):
        self.dims = T, D, F, E, k
        self.normalise, self.kept = normalise, kept
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        n = self.new
        self.gain, self.Wr = 1 + n(D, std=0.1), n(D, E, std=2 * D ** -0.5)
        self.Wg, self.Wu = n(E, D, F, std=D ** -0.5), n(E, D, F, std=D ** -0.5)
        self.Wd = n(E, F, D, std=F ** -0.5)
        self.X, self.R, self.dY = n(T, D), n(T, D), n(T, D, std=1 / T)
        R = T * k

        def e(*s, t=BF16):
            return torch.zeros(s, dtype=t, device="cuda")

        self.S, self.N, self.Y = e(T, D), e(T, D), e(T, D)
        self.z, self.w = e(T, E, t=F32), e(T, k, t=F32)
        self.experts, self.rows, self.offsets = e(T, k, t=I32), e(T, k, t=I32), e(E + 1, t=I32)
        self.Xs, self.H, self.Ys = e(R, D), e(R, F), e(R, D)
        self.Z = e(2, R, F, t=F32) if kept else None
        self.dYs, self.dw, self.dH, self.dXs = e(R, D), e(T, k, t=F32), e(R, F), e(R, D)
        self.dWd, self.dWg, self.dWu = e(E, F, D), e(E, D, F), e(E, D, F)
        self.dz, self.dN, self.dS, self.dgain = e(T, E, t=F32), e(T, D), e(T, D), e(D)

    def new(self, *shape, std=1.0):
        return (torch.randn(shape, generator=self.g, device="cuda") * std).to(BF16)

    def refill(self):
        for t, std in ((self.X, 1.0), (self.R, 1.0), (self.dY, 1 / self.dims[0])):
            t.copy_(self.new(*t.shape, std=std))

    def forward(self, stream=None):
        T, D, F, E, k = self.dims
        R, s = T * k, {"stream": stream}
        pg.rmsnorm_bf16(T, D, self.X, self.R, self.gain, EPS, self.S, self.N, **s)
        pg.gemm_bf16(T, E, D, 1.0, self.N, self.Wr, 0.0, self.z, **s)
        pg.route_topk(T, E, k, self.z, self.normalise, self.experts, self.w, **s)
        pg.expert_sort(T, E, k, self.experts, self.offsets, self.rows, **s)
        pg.expert_gather_bf16(T, k, D, self.N, self.rows, self.Xs, **s)
        pg.experts_gated_bf16(R, F, D, E, self.offsets, self.Xs, self.Wg, self.Wu, "silu", self.H,
                              preact=self.Z, **s)
        pg.experts_linear_bf16(R, D, F, E, self.offsets, self.H, self.Wd, self.Ys, **s)
        pg.expert_combine_bf16(T, k, D, self.Ys, self.rows, self.w, self.S, self.Y, **s)

    def backward(self, stream=None):
        T, D, F, E, k = self.dims
        R, s = T * k, {"stream": stream}
        pg.expert_combine_bf16_backward(T, k, D, self.Ys, self.rows, self.w, self.dY, self.dYs,
                                        self.dw, **s)
        pg.experts_linear_bf16_backward(R, D, F, E, self.offsets, self.H, self.Wd, self.dYs,
                                        self.dH, self.dWd, **s)
        pg.experts_gated_bf16_backward(R, F, D, E, self.offsets, self.Xs, self.Wg, self.Wu, "silu",
                                       self.dH, self.dXs, self.dWg, self.dWu, preact=self.Z, **s)
        pg.expert_combine_bf16(T, k, D, self.dXs, self.rows, None, None, self.dN, **s)
        pg.route_topk_backward(T, E, k, self.z, self.normalise, self.experts, self.dw, self.dz, **s)
        # (the residual's dY flows into S beside the norm's own gradient)
        pg.rmsnorm_bf16_backward(T, D, self.S, self.gain, EPS, self.dN, self.dY, self.dS,
                                 self.dgain, **s)

    OUTPUTS = ("S N z w experts rows offsets Xs H Ys Y dYs dw dH dXs dWd dWg dWu dz dN dS "
               "dgain").split()

    def outputs(self):
        return {n: getattr(self, n).clone() for n in self.OUTPUTS}

    def check(self):
        T, D, F, E, k = self.dims
        assert torch.equal(self.S, (self.X.float() + self.R.float()).to(BF16))
        y, err, _, _ = moe.norm(self.S, self.gain, EPS)
        ref.check(self.N, y, moe.bf16_out(y, err), "N")
        experts, w, bound, _ = moe.route(self.z, k, self.normalise)
        assert torch.equal(self.experts, experts)
        ref.check(self.w, w, bound, "w")
        offsets, rows = moe.sort(experts, E)
        assert torch.equal(self.offsets.cpu(), offsets) and torch.equal(self.rows.cpu(), rows)
        assert torch.equal(self.Xs[self.rows.long()], self.N.unsqueeze(1).expand(T, k, D))
        ref.check(self.H, *moe.experts_gated(self.offsets, self.Xs, self.Wg, self.Wu, "silu")["H"],
                  "H")
        ref.check(self.Ys, *moe.experts_linear(self.offsets, self.H, self.Wd)["Y"], "Ys")
        ref.check(self.Y, *moe.combine(self.Ys, self.rows, self.w, self.S), "Y")
        d, ed, dw, ew = moe.combine_backward(self.Ys, self.rows, self.w, self.dY)
        ref.check(self.dYs[self.rows.long()], d, ed, "dYs")
        ref.check(self.dw, dw, ew, "dw")
        want = moe.experts_linear_backward(self.offsets, self.H, self.Wd, self.dYs)
        ref.check(self.dH, *want["dX"], "dH")
        ref.check(self.dWd, *want["dW0"], "dWd")
        want = moe.experts_gated_backward(self.offsets, self.Xs, self.Wg, self.Wu, "silu", self.dH)
        ref.check(self.dXs, *want["dX"], "dXs")
        ref.check(self.dWg, *want["dW0"], "dWg")
        ref.check(self.dWu, *want["dW1"], "dWu")
        ref.check(self.dN, *moe.combine(self.dXs, self.rows, None, None), "dN")
        ref.check(self.dz, *moe.route_backward(self.z, k, self.normalise, self.experts, self.dw),
                  "dz")
        want = moe.norm_backward(self.S, self.gain, EPS, self.dN, self.dY)
        ref.check(self.dS, *want["dX"], "dS")
        ref.check(self.dgain, *want["dgain"], "dgain")


@pytest.mark.parametrize("T,D,F,E,k,normalise,kept", [
    (1, 64, 96, 8, 2, True, True), (24, 256, 136, 16, 4, False, False),
    (300, 200, 264, 6, 2, True, False), (777, 513, 130, 5, 3, False, True),
    (2000, 256, 512, 8, 2, True, True)])
def test_block(T, D, F, E, k, normalise, kept):
    b = Block(T, D, F, E, k, normalise, 1, kept)
    b.forward()
    b.backward()
    b.check()
    first = b.outputs()
    b.forward()
    b.backward()
    for name, was in first.items():  # nothing hangs on timing
        assert torch.equal(getattr(b, name), was), name


def capture(b):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.forward()
        b.backward()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward()
        b.backward()
    return graph


def test_graphs_replay_with_other_routing():
    # two captured blocks of different shapes, one with odd pitches (relayouts in scratch),
    # replayed in turn and beside eager calls of the same library
    blocks = [Block(400, 256, 128, 8, 2, True, 2), Block(90, 251, 133, 12, 3, False, 3, False)]
    graphs = [capture(b) for b in blocks]
    seen = []
    for _ in range(3):
        for b, graph in zip(blocks, graphs):
            b.refill()
            graph.replay()
            torch.cuda.synchronize()
            b.check()
            seen.append(b.offsets.tolist())
            got = b.outputs()
            b.forward()
            b.backward()
            for name, was in got.items():
                assert torch.equal(getattr(b, name), was), name
    assert len({tuple(s) for s in seen}) == len(seen)  # the groups did change


def test_graphs_on_two_streams_at_once():
    blocks = [Block(300, 256, 264, 8, 2, True, 4), Block(500, 133, 200, 6, 2, True, 5, False)]
    graphs = [capture(b) for b in blocks]
    alone = []
    for b, graph in zip(blocks, graphs):
        graph.replay()
        torch.cuda.synchronize()
        alone.append(b.outputs())
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for b, want in zip(blocks, alone):
        for name, was in want.items():
            assert torch.equal(getattr(b, name), was), name


def test_another_stream():
    b = Block(200, 128, 72, 8, 2, True, 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.forward(stream=s)
    b.backward(stream=s.cuda_stream)
    s.synchronize()
    b.check()


def test_threads_on_streams_of_their_own():
    blocks = [Block(150 + 70 * i, 128 + 5 * i, 72 + 8 * i, 8, 2, True, 10 + i, i % 2 == 0)
              for i in range(4)]
    want = []
    for b in blocks:
        b.forward()
        b.backward()
        want.append(b.outputs())
    torch.cuda.synchronize()
    failed = []

    def work(b):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    b.forward()
                    b.backward()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(b,)) for b in blocks]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for b, outs in zip(blocks, want):
        for name, was in outs.items():
            assert torch.equal(getattr(b, name), was), name


def test_norm_feeds_the_int8_product():
    # y W from int8 rows with their scales and an int8 W with a scale a column
    T, D, N = 200, 512, 136
    g = torch.Generator(device="cuda").manual_seed(7)
    X = torch.randn((T, D), generator=g, device="cuda").to(BF16)
    W = torch.randn((D, N), generator=g, device="cuda") * D ** -0.5
    wscale = W.abs().amax(0) / 127
    Wq = torch.round(W / wscale).to(torch.int8)
    Q, scale = torch.empty((T, D), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    C = torch.empty((T, N), dtype=I32, device="cuda")
    pg.rmsnorm_i8(T, D, X, None, None, EPS, None, Q, scale)
    pg.gemm_i8(T, N, D, 1, Q, Wq, 0, C)
    assert torch.equal(C.double(), Q.double() @ Wq.double())
    got = C.double() * scale.double().unsqueeze(1) * wscale.double()
    y, err, _, _ = moe.norm(X, None, EPS)
    deq = Wq.double() * wscale.double()
    # Q is off by half a step, and by the error of y and of the scale in steps
    bound = (scale.double().unsqueeze(1) * (0.5 + 127 * 4 * moe.RSTD)) @ \
        deq.abs().sum(0, keepdim=True)
    assert ((got - y @ deq).abs() <= bound).all()
