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


# ---- relative accuracy in the tails ----------------------------------------
#
# The smooth activations are products, so their error is relative: the
# exponential's argument is off by at most 2^-23 of itself (two roundings),
# v_exp_f32 and v_rcp_f32 by a unit each, gelu's quotient of polynomials by
# 4e-7 and its roundings; tanh-gelu's argument takes three roundings more.
# 1.5e-6 and 5e-7 per unit of the exponent cover them.  Y is rounded once.

# |z| up to which neither exp(-exponent) nor the result leaves fp32's range
REACH = {"gelu": 12.5, "gelu_tanh": 9.5, "silu": 80.0}


def every_value(dtype, reach):
    """Every fourth value of the type with a magnitude up to `reach`."""
    bits = torch.arange(0, 1 << 15, 4, dtype=torch.int32).to(torch.int16)
    v = bits.view(dtype).double()
    v = v[(v <= reach) & (v > 1e-3)]
    return column(torch.cat([v, -v]).tolist(), dtype)


def exponent(z, a):
    """The exponent whose exponential the formula takes."""
    if a == "gelu":
        return 0.5 * z * z
    if a == "gelu_tanh":
        return (2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)).abs()
    return z.abs()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("a", SMOOTH)
def test_activations_keep_their_digits(a, dtype):
    z = every_value(dtype, REACH[a])
    Y = km.kmeans_linear(z, torch.ones(1, 1, dtype=dtype, device="cuda"), activation=a)
    z = ref.cpu64(z)
    y = ref.act(z, a)
    rel = 1.5e-6 + 5e-7 * exponent(z, a)
    ref.check(Y, y, y.abs() * (rel * (1 + ref.U[dtype]) + ref.U[dtype]) + ref.TINY[dtype], a)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("a", SMOOTH)
def test_slopes_keep_their_digits(a, dtype):
    """A slope is a sum of two terms, each off by its own relative error;
    1 - s of the logistic function adds 2^-24 in all where s is near 1."""
    z = every_value(dtype, REACH[a])
    got, _ = slopes(z, a, torch.ones_like(z))
    z = ref.cpu64(z).flatten()
    want = ref.act_slope(z, a)
    rel = 1.5e-6 + 5e-7 * exponent(z, a)
    if a == "gelu":
        phi = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
        terms = phi + z.abs() * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        lost = torch.zeros_like(z)
    else:
        s = torch.sigmoid(z if a == "silu" else
                          2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        du = 1.0 if a == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
        terms = s + z.abs() * s * (1 - s) * du
        lost = z.abs() * s * du * 2 * ref.EPS
    err = terms * rel + lost
    ref.check(got, want, err * (1 + ref.U[dtype]) + ref.U[dtype] * want.abs() + ref.TINY[dtype], a)
