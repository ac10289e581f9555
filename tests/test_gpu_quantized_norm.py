"""The norm with its residual and 8-bit output (HIP, through the public binding)
against its definition in fp64, with values that cancel to zero.  Bounds, block by
block: ``quantized_bounds``."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
km = pytest.importorskip("means_nearest_centroid_amd")
import prediction_reference as ref  # noqa: E402
import quantized_bounds as bounds  # noqa: E402

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a visible GPU")
    km.load_library()
    return torch.device("cuda:0")


SIZES = [(1, 1), (1, 8), (3, 7), (40, 16), (5, 128), (17, 129), (64, 256), (33, 257), (9, 512),
         (130, 1000), (7, 1024), (12, 2048), (3, 4096), (5, 4099), (2, 8192), (3, 16384),
         (2, 16385), (1, 40003)]


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("N,D", SIZES)
def test_norm_to_8_bits(N, D, dtype):
    g = torch.Generator().manual_seed(N + D)
    x, r = (torch.randn(N, D, generator=g).to(dtype) for _ in range(2))
    r = torch.where(torch.rand(N, D, generator=g) < 0.05, -x, r)
    if D > 128:
        r[N - 1, 128:256] = -x[N - 1, 128:256]           # a block of zeros
    w = torch.randn(D, generator=g).to(dtype)
    rel = bounds.norm_rel(D)
    for weight in (None, w):
        y, _, h, herr = ref.rms_norm(x, weight, r)
        Q, s, H = km.kmeans_rms_norm(x.cuda(), weight if weight is None else weight.cuda(),
                                     r.cuda(), quantize=True)
        bounds.check(Q, s, y, rel, 1, f"{N} x {D}")
        ref.check(H, h, herr, "H")
        y = ref.rms_norm(x, weight)[0]
        Q, s = km.kmeans_rms_norm(x.cuda(), weight if weight is None else weight.cuda(),
                                  quantize=True)
        bounds.check(Q, s, y, rel, 1, f"{N} x {D} alone")


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_quantize(rows, dtype):
    for N, D in ((1, 1), (3, 7), (128, 128), (127, 129), (130, 1000), (257, 260)):
        g = torch.Generator().manual_seed(N)
        x = (torch.randn(N, D, generator=g) * torch.exp(torch.randn(N, 1, generator=g))).to(dtype)
        x[torch.rand(N, D, generator=g) < 0.05] = 0
        Q, s = km.kmeans_quantize(x.cuda(), rows=rows)
        bounds.check(Q, s, x.double(), 0.0, rows, f"{N} x {D}")
