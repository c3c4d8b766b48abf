"""The norm of rows whose squares leave fp32's range: at either end with an eps of less than
2^-100, below with any."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe_reference as moe  # noqa: E402
import operator_reference as ref  # noqa: E402
import software_pipelined_tiled_loop_gb300 as pg  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
WIDTHS = [1, 40, 257, 4096, 4097, 8200, 12288, 16390, 20488, 32768]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from software_pipelined_tiled_loop_gb300 import build
    build.build()
    pg.lib()
    yield
    assert pg.pgemm_get_device_status() == 0


def rnd(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def nan(*shape, dtype=BF16):
    return torch.full(shape, NAN, device="cuda", dtype=dtype)


def rows(D, eps):
    """A row of each size, ordinary ones between them: what one needs must not reach the next."""
    large = [62, 64, 100, 120] if eps < 2.0 ** -100 else []
    sizes = [2.0 ** e for e in (0, -60, 0, -75, -100, -120, 0, -45, -55, 0, 50, *large, 0)]
    S = (rnd(1, len(sizes), D, dtype=F32).clamp(-60, 60)
         * torch.tensor(sizes, device="cuda").unsqueeze(1)).to(BF16)
    S[6] = S[6] * 2.0 ** -10
    if large:
        S[6, 0] = 2.0 ** 90  # one value
    S[2] = 0
    S[2, D // 2] = 2.0 ** -110
    return torch.where((S == 0) & (D == 1), 2.0 ** -90, S)  # (no row of zeros)


def check_int8(S, g, eps, got):
    Q, scale = got
    y, _, _, _ = moe.norm(S, g, eps)
    step = y.abs().amax(1) / 127
    assert ((scale.double() - step).abs() <= step * (2 * moe.RSTD) + 2.0 ** -150).all()
    off = (Q.double() * step.unsqueeze(1) - y).abs()
    assert (off <= step.unsqueeze(1) * (0.5 + 127 * 4 * moe.RSTD)).all()
    assert (Q.abs().amax(1)[step > 0] == 127).all()


@pytest.mark.parametrize("eps", [0.0, 1e-38, 2.0 ** -101, 2.0 ** -100, 1e-6])
@pytest.mark.parametrize("D", WIDTHS)
def test_forward(D, eps):
    S = rows(D, eps)
    T = S.shape[0]
    gain = rnd(2, D)
    gain[gain == 0] = 1
    for g in (gain, None):
        Y, kept = nan(T, D), nan(T, D)
        pg.rmsnorm_bf16(T, D, S, None, g, eps, kept, Y)
        assert torch.equal(kept, S)
        y, err, _, _ = moe.norm(S, g, eps)
        ref.check(Y, y, moe.bf16_out(y, err), "Y")
        R = torch.zeros_like(S)
        Y2 = nan(T, D)
        pg.rmsnorm_bf16(T, D, S, R, g, eps, None, Y2)
        assert torch.equal(Y, Y2)
        Q, scale = torch.full((T, D), 99, device="cuda", dtype=torch.int8), nan(T, dtype=F32)
        pg.rmsnorm_i8(T, D, S, None, g, eps, kept, Q, scale)
        assert torch.equal(kept, S)
        check_int8(S, g, eps, (Q, scale))


@pytest.mark.parametrize("eps", [0.0, 1e-38, 2.0 ** -100, 1e-6])
@pytest.mark.parametrize("D", WIDTHS)
def test_backward(D, eps):
    S = rows(D, eps)
    T = S.shape[0]
    gain, dY, dS = rnd(3, D), rnd(4, T, D, std=2.0 ** -10), rnd(5, T, D)
    for g, ds in ((gain, dS), (None, None)):
        want = moe.norm_backward(S, g, eps, dY, ds)
        dX, dg = nan(T, D), nan(D)
        pg.rmsnorm_bf16_backward(T, D, S, g, eps, dY, ds, dX, dg)
        ref.check(dX, *want["dX"], "dX")
        ref.check(dg, *want["dgain"], "dgain")
        dX2 = nan(T, D)
        pg.rmsnorm_bf16_backward(T, D, S, g, eps, dY, ds, dX2, None)
        assert torch.equal(dX, dX2)


def test_many_rows_of_every_size():
    """Several rows a block."""
    T, D = 9000, 264
    S = rnd(6, T, D, dtype=F32)
    S = (S * torch.exp2(torch.randint(-120, 120, (T, 1), device="cuda").float())).to(BF16)
    S[(S == 0).all(1)] = 1
    gain, dY = rnd(7, D), rnd(8, T, D, std=2.0 ** -10)
    Y, dX, dg = nan(T, D), nan(T, D), nan(D)
    pg.rmsnorm_bf16(T, D, S, None, gain, 0.0, None, Y)
    y, err, _, _ = moe.norm(S, gain, 0.0)
    ref.check(Y, y, moe.bf16_out(y, err), "Y")
    Q, scale = torch.full((T, D), 99, device="cuda", dtype=torch.int8), nan(T, dtype=F32)
    pg.rmsnorm_i8(T, D, S, None, gain, 0.0, None, Q, scale)
    check_int8(S, gain, 0.0, (Q, scale))
    pg.rmsnorm_bf16_backward(T, D, S, gain, 0.0, dY, None, dX, dg)
    want = moe.norm_backward(S, gain, 0.0, dY, None)
    ref.check(dX, *want["dX"], "dX")
    ref.check(dg, *want["dgain"], "dgain")


def test_squares_past_the_range_give_zeros_with_an_ordinary_eps():
    S, Y = rnd(10, 3, 200), nan(3, 200)
    S[1] = S[1] * 2.0 ** 70
    pg.rmsnorm_bf16(3, 200, S, None, None, 1e-6, None, Y)
    assert (Y[1] == 0).all()
    y, err, _, _ = moe.norm(S[::2], None, 1e-6)
    ref.check(Y[::2], y, moe.bf16_out(y, err), "Y")


def test_what_has_no_norm():
    S = rnd(9, 4, 40)
    S[0], S[1, 3], S[2, 5] = 0, INF, NAN
    Y, Q, scale = nan(4, 40), torch.full((4, 40), 99, device="cuda", dtype=torch.int8), nan(4, dtype=F32)
    pg.rmsnorm_bf16(4, 40, S, None, None, 0.0, None, Y)
    assert Y[0].isnan().all() and Y[2].isnan().all()  # 0 / 0
    assert Y[1, 3].isnan() and (Y[1, :3] == 0).all() and (Y[1, 4:] == 0).all()
    assert torch.isfinite(Y[3].float()).all()
    pg.rmsnorm_i8(4, 40, S, None, None, 0.0, None, Q, scale)
    assert scale[:3].isnan().all() and (Q[:3] == 0).all() and scale[3] > 0
