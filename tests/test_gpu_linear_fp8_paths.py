"""The linear layer on 8-bit operands (HIP, through the public binding) on every
kernel that the plan chooses between, against its definition in fp64, value by
value and by the norm.  Bounds and their derivation: ``linear_fp8_bounds``."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
km = pytest.importorskip("means_nearest_centroid_amd")
import linear_fp8_bounds as ref  # noqa: E402
from linear_fp8_paths import PATHS  # noqa: E402

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a visible GPU")
    km.load_library()
    yield torch.device("cuda:0")
    torch.cuda.synchronize()
    km.kmeans_release_workspace()
    torch.cuda.empty_cache()


def rand(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * scale


def operands(N, D, F, kind="normal"):
    """Rows of different sizes; ``outliers``: one column in 16 is 100 times as
    large, in pairs that nearly cancel in the products; ``positive``: no signs."""
    x = rand((N, D), 1) * torch.exp(rand((N, 1), 2))
    w = rand((F, D), 3, D ** -0.5)
    if kind == "outliers":
        x[:, ::16] *= 100.0
        x[:, 1::16] = x[:, ::16][:, :x[:, 1::16].shape[1]]
        w[:, 1::16] = -w[:, ::16][:, :w[:, 1::16].shape[1]]
    if kind == "positive":
        x, w = x.abs(), w.abs()
    return *km.kmeans_quantize(x), *km.kmeans_quantize(w, rows=128)


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("N,D,F", [p[:3] for p in PATHS])
def test_every_kernel(N, D, F, dtype):
    X, sx, W, sw = operands(N, D, F)
    b, R = rand((F,), 5).to(dtype), rand((N, F), 6).to(dtype)
    for bias, residual, act in ((None, None, "none"), (b, R, "gelu_tanh")):
        want = ref.linear_fp8(X, sx, W, sw, bias, residual, act, dtype)
        got = km.kmeans_linear_fp8(X, sx, W, sw, bias, residual, act, dtype=dtype)
        ref.check(got, *want, dtype)


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("kind", ["outliers", "positive"])
@pytest.mark.parametrize("N,D,F", [(16, 700, 900), (17, 700, 900), (300, 384, 640), (700, 1300, 2000),
                                   (3000, 384, 5001)])
def test_other_values(N, D, F, kind, dtype):
    X, sx, W, sw = operands(N, D, F, kind)
    want = ref.linear_fp8(X, sx, W, sw, None, None, "none", dtype)
    ref.check(km.kmeans_linear_fp8(X, sx, W, sw, dtype=dtype), *want, dtype)


@pytest.mark.parametrize("activation", list(km.ACTIVATIONS))
@pytest.mark.parametrize("bias,residual", [(True, False), (False, True)])
def test_epilogues_of_the_wide_kernel(activation, bias, residual):
    N, D, F = 3000, 384, 5001
    X, sx, W, sw = operands(N, D, F)
    b = rand((F,), 5).to(FP) if bias else None
    R = rand((N, F), 6).to(FP) if residual else None
    want = ref.linear_fp8(X, sx, W, sw, b, R, activation, FP)
    ref.check(km.kmeans_linear_fp8(X, sx, W, sw, b, R, activation, dtype=FP), *want, FP)


def rows_in(t, extra, shift, fill):
    wide = torch.full((t.shape[0], t.shape[1] + extra + shift), fill, device="cuda").to(t.dtype)
    v = wide[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return v


@pytest.mark.parametrize("extra,shift", [(16, 0), (3, 5)])
@pytest.mark.parametrize("N,D,F", [(2050, 2050, 4100), (4096, 512, 4096)])
def test_strides_of_the_wide_kernel(N, D, F, extra, shift):
    """NaN beside all operands; nothing beside the output is written."""
    X, sx, W, sw = operands(N, D, F)
    R = rand((N, F), 6).to(BF)
    nan = float("nan")
    want = km.kmeans_linear_fp8(X, sx, W, sw, residual=R)
    out = rows_in(torch.zeros_like(want), extra, shift, 7.0)
    km.kmeans_linear_fp8(rows_in(X, extra, shift, nan), rows_in(sx, extra, shift, nan),
                         rows_in(W, extra, shift, nan), rows_in(sw, extra, shift, nan),
                         residual=rows_in(R, extra, shift, nan), out=out)
    assert torch.equal(out, want)
    wide = out._base
    assert (wide[:, :shift] == 7).all() and (wide[:, shift + F:] == 7).all()
    assert torch.equal(km.kmeans_linear_fp8(X, sx, W, sw, residual=R, out=R), want)


def test_special_values_of_the_wide_kernel():
    """A NaN reaches its own row or columns alone, from the last of each."""
    N, D, F = 2050, 2050, 4100
    X, sx, W, sw = operands(N, D, F)
    want = km.kmeans_linear_fp8(X, sx, W, sw)
    s2 = sx.clone()
    s2[N - 1, 16] = float("nan")
    got = km.kmeans_linear_fp8(X, s2, W, sw)
    assert torch.equal(got[:-1], want[:-1]) and got[-1].isnan().all()
    s2 = sw.clone()
    s2[32, 0] = float("nan")
    got = km.kmeans_linear_fp8(X, sx, W, s2)
    assert torch.equal(got[:, :4096], want[:, :4096]) and got[:, 4096:].isnan().all()
    w2 = W.float()
    w2[F - 1, D - 1] = float("nan")
    got = km.kmeans_linear_fp8(X, sx, w2.to(torch.float8_e4m3fn), sw)
    assert torch.equal(got[:, :-1], want[:, :-1]) and got[:, -1].isnan().all()
