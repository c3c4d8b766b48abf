"""The example with a mixture of experts: it runs, and its gradients are those of the
function that it computes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_train_step_example_gpu import load  # noqa: E402


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from software_pipelined_tiled_loop_gb300 import build
    build.build()
    return load()


def test_example_runs(example):
    losses, _ = example.main(steps=3, quiet=True, experts=8)
    assert len(losses) == 3 and all(l == l and l > 0 for l in losses)


def test_gradients(example):
    m = example.SparseBlock(vocab=150, width=96, hidden=80, experts=6, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    T = 220
    ids = torch.randint(0, m.V, (T, m.C), generator=g, device="cuda")
    target = torch.randint(0, m.V, (T,), generator=g, device="cuda")
    target[::9] = -100
    loss, valid, grads = m.gradients(ids, target)
    experts = m.body(ids, keep=True)[2][2].long()  # as they were chosen

    p = {k: v.double().requires_grad_() for k, v in m.p.items()}
    f = torch.nn.functional
    h0 = p["E"][ids].mean(1)
    h1 = f.silu(h0 @ p["Wa"] + p["ba"]) + h0
    n = f.rms_norm(h1, (m.D,), p["gain"], m.EPS)
    w = torch.softmax(n @ p["Wr"], 1).gather(1, experts)
    up = f.silu(torch.einsum("td,tkdf->tkf", n, p["Wg"][experts]))
    up = up * torch.einsum("td,tkdf->tkf", n, p["Wu"][experts])
    h2 = h1 + torch.einsum("tkf,tkfd,tk->td", up, p["Wd"][experts], w)
    want = f.cross_entropy(h2 @ p["E"].t(), target, ignore_index=-100, reduction="none")
    mean = want.sum() / valid
    # Between the weights and a gradient lie at most twelve tensors rounded to bf16 (h0, h1,
    # n, g, y, h2 forward; dh2, dy, dg, dG or dU, dn, dh1 backward), each off by 2^-9 of its
    # norm (half a step, and the half of that on average), with the result's own rounding
    # thirteen: 2^-9 * 13 = 0.025 if all add up, the loss by half as many
    assert abs((loss.sum() / valid).item() - mean.item()) <= 0.0125 * mean.item()
    assert set(grads) == set(p)
    for name, ref in zip(p, torch.autograd.grad(mean, list(p.values()))):
        err = ((grads[name].double() - ref).norm() / ref.norm()).item()
        assert err <= 0.025, (name, err)
