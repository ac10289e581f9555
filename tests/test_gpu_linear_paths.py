"""The linear operators (HIP, through the public binding) at shapes chosen for
the code path they take, against the definitions in fp64: rows of few values,
and every kernel that the plan chooses between.  Bounds and their derivation:
``codebook_reference``."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
km = pytest.importorskip("means_nearest_centroid_amd")
import codebook_reference as ref  # noqa: E402
from linear_paths import PATHS  # noqa: E402

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a visible GPU")
    km.load_library()
    return torch.device("cuda:0")


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


# ---- rows of less than eight values ----------------------------------------

@pytest.mark.parametrize("D", [1, 2, 3, 7])
@pytest.mark.parametrize("N,F", [(65, 66), (66, 65), (70, 129), (129, 70), (321, 386), (391, 5)])
def test_gradients_of_narrow_rows(N, D, F):
    """Points of a few coordinates: the rows of X and W are shorter than one
    load, over one tile of the summed index and over several."""
    X, W = rand((N, D), BF, N), rand((F, D), BF, F)
    dY, Z = rand((N, F), BF, 5, 0.25), rand((N, F), BF, 6, 2.0)
    want = ref.linear_grad(dY, X, W, Z, "silu")
    for name, got in zip(("dX", "dW", "db"), km.kmeans_linear_grad(dY, X, W, Z, "silu")):
        ref.check(got, *want[name], name)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("N,D,F", [(40, 3, 50), (200, 7, 130), (321, 1, 17), (129, 2, 1)])
def test_forward_of_narrow_rows(N, D, F, dtype):
    X, W, b = rand((N, D), dtype, N), rand((F, D), dtype, F), rand((F,), dtype, 3)
    y, z, yb, zb = ref.linear(X, W, b, None, "relu")
    Y, Z = km.kmeans_linear(X, W, bias=b, activation="relu", save_pre=True)
    ref.check(Y, y, yb, "Y")
    ref.check(Z, z, zb, "Z")


# ---- every kernel of the plan ----------------------------------------------

def rows(t, extra):
    """The same values, `extra` more (NaN) between rows."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype,
                      device="cuda")
    v = wide[:, :t.shape[1]]
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("N,D,F,extra", [p[:4] for p in PATHS])
def test_forward_of_every_kernel(N, D, F, extra, dtype):
    X, W = rand((N, D), dtype, 1), rand((F, D), dtype, 2, D ** -0.5)
    b, R = rand((F,), dtype, 3), rand((N, F), dtype, 4)
    y, z, yb, zb = ref.linear(X, W, b, R, "gelu_tanh")
    Y, Z = km.kmeans_linear(rows(X, extra), rows(W, extra), bias=b, residual=R,
                            activation="gelu_tanh", save_pre=True)
    ref.check(Y, y, yb, "Y")
    ref.check(Z, z, zb, "Z")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("N,D,F,extra", [p[:4] for p in PATHS])
def test_gradients_of_every_kernel(N, D, F, extra, dtype):
    X, W = rand((N, D), dtype, 1), rand((F, D), dtype, 2, D ** -0.5)
    dY, Z = rand((N, F), dtype, 3, 0.25), rand((N, F), dtype, 4, 2.0)
    want = ref.linear_grad(dY, X, W, Z, "silu")
    got = km.kmeans_linear_grad(dY, rows(X, extra), rows(W, extra), Z, "silu")
    for name, g in zip(("dX", "dW", "db"), got):
        ref.check(g, *want[name], name)
