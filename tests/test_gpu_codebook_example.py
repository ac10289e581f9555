"""The codebook-training example: its gradients against autograd in fp64 with
the labels it chose, and its loss over a few steps.

Bounds: every intermediate is rounded to bf16 (relative 2^-8 at most), at most
six such roundings in a row reach a gradient, and they average out over the
sums, so a gradient differs from the exact one by at most 6 * 2^-8 = 0.024 of
its norm; 0.03 leaves room for the second order."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
km = pytest.importorskip("means_nearest_centroid_amd")

_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples",
                     "codebook_training.py")
_spec = importlib.util.spec_from_file_location("codebook_training", _path)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a visible GPU")
    km.load_library()


@pytest.mark.parametrize("N,width,code,K", [(3000, 96, 64, 40), (517, 40, 32, 300)])
def test_gradients(N, width, code, K):
    X = example.synthetic(N, width, 16, seed=1)
    p = {n: t.to(torch.bfloat16) for n, t in example.parameters(width, code, K, seed=2).items()}
    loss, grads = example.gradients(p, X)

    x = X.double().cpu()
    q = {n: t.double().cpu().requires_grad_() for n, t in p.items()}
    H = torch.nn.functional.gelu(x @ q["W1"].T + q["b1"])
    h = km.kmeans_linear(X, p["W1"], p["b1"], activation="gelu")
    labels, _ = km.kmeans_assign(h, p["C"], km.kmeans_centroid_norms(p["C"]))
    Q = q["C"][labels.long().cpu()]
    through = Q + H - H.detach()              # Q's value, gradients to both
    Y = through @ q["W2"].T + q["b2"]
    exact = ((Y - x).square().sum() + (Q - H).square().sum()) / (2 * N)
    exact.backward()
    assert abs(loss.item() - exact.item()) <= 0.03 * exact.item()
    for n, g in grads.items():
        e = q[n].grad
        assert (g.double().cpu() - e).norm() <= 0.03 * e.norm(), n


def test_loss_falls():
    X = example.synthetic(4096, 64, 32)
    losses = example.train(X, example.parameters(64, 32, 128), 60)
    assert all(b == b for b in losses)
    assert losses[-1] < 0.7 * losses[0]
