"""The linear operators' activations and slopes (HIP, through the public
binding) far from zero: each pre-activation goes through a one-feature layer of
weight 1, so it is exact."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
km = pytest.importorskip("means_nearest_centroid_amd")
import codebook_reference as ref  # noqa: E402

BF, FP = torch.bfloat16, torch.float16
SMOOTH = ["gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a visible GPU")
    km.load_library()
    return torch.device("cuda:0")


def column(values, dtype):
    return torch.tensor(values, dtype=torch.float64).to(dtype).cuda().reshape(-1, 1)


def slopes(z, a, dY):
    """dY act'(z) as dX of a layer of weight 1, and the bias's sum of it."""
    one = torch.ones(1, 1, dtype=z.dtype, device="cuda")
    dX, _, db = km.kmeans_linear_grad(dY, torch.zeros_like(z), one, z, a)
    return dX.float().cpu().flatten(), float(db)


@pytest.mark.parametrize("a", ["relu"] + SMOOTH)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_slopes_where_they_are_one_or_zero(a, dtype):
    far = [200.0, 1000.0, 60000.0, float("inf")]
    if dtype == BF:
        far += [1e10, 5e19, 1e20, 3e38]
    z = column(far + [-v for v in far], dtype)
    dY = torch.full_like(z, 0.75)
    got, db = slopes(z, a, dY)
    assert got[:len(far)].tolist() == [0.75] * len(far), got
    assert got[len(far):].tolist() == [0.0] * len(far), got
    assert db == 0.75 * len(far)


@pytest.mark.parametrize("a", SMOOTH)
def test_slopes_of_nan_are_nan(a):
    z = column([float("nan"), 1.0], BF)
    got, db = slopes(z, a, torch.ones_like(z))
    assert math.isnan(float(got[0])) and math.isfinite(float(got[1])) and math.isnan(db)


@pytest.mark.parametrize("a", SMOOTH)
def test_a_pre_activation_past_fp16_leaves_its_gradients_finite(a):
    """-90000 is kept as -inf in fp16, but Y = act(-90000) is zero, and so is
    the slope: its row of dX, its part of dW and db are those of the others."""
    X = torch.tensor([[300.0, 1.0], [1.0, 0.5]], dtype=FP, device="cuda")
    W = torch.tensor([[-300.0, 0.0], [0.25, 1.0]], dtype=FP, device="cuda")
    Y, Z = km.kmeans_linear(X, W, activation=a, save_pre=True)
    assert float(Z[0, 0]) == float("-inf") and float(Y[0, 0]) == 0.0
    dY = torch.ones(2, 2, dtype=FP, device="cuda")
    got = km.kmeans_linear_grad(dY, X, W, Z, a)
    Z = Z.clone()
    Z[0, 0] = -65504.0
    want = ref.linear_grad(dY, X, W, Z, a)
    for name, g in zip(("dX", "dW", "db"), got):
        ref.check(g, *want[name], name)
