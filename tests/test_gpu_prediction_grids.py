"""Operators of label prediction (HIP, through the public binding) at sizes whose
threads a single launch cannot count: every part agrees, bit for bit, with a call
of that part alone."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
km = pytest.importorskip("means_nearest_centroid_amd")

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a visible GPU")
    km.load_library()
    yield torch.device("cuda:0")
    torch.cuda.synchronize()
    km.kmeans_release_workspace()
    torch.cuda.empty_cache()


def need(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def values(N, D, dtype=BF):
    i = torch.arange(N * D, dtype=torch.int64, device="cuda")
    return ((i * 37 % 251) - 120).to(dtype).view(N, D)


def parts(N, size):
    return [slice(i, min(N, i + size)) for i in range(0, N, size)]


def test_norm_and_its_gradient():
    need(30)
    N = (1 << 27) + 70
    X = values(N, 2)
    Y = km.kmeans_rms_norm(X)
    w = torch.tensor([1.5, -2.0], dtype=BF, device="cuda")
    dX, _ = km.kmeans_rms_norm_grad(Y, X, w, need_dw=False)
    for p in parts(N, 1 << 25):
        assert torch.equal(Y[p], km.kmeans_rms_norm(X[p])), p
        assert torch.equal(dX[p], km.kmeans_rms_norm_grad(Y[p], X[p], w, need_dw=False)[0]), p


def test_quantize():
    need(40)
    N = (1 << 30) + 77
    X = values(1 << 20, 1).repeat((N >> 20) + 1, 1)[:N]
    Q, s = km.kmeans_quantize(X)
    q, t = km.kmeans_quantize(X[:1 << 20])
    for p in parts(N, 1 << 20):
        n = p.stop - p.start
        assert torch.equal(Q[p].view(torch.uint8), q[:n].view(torch.uint8)), p
        assert torch.equal(s[p], t[:n]), p


def test_linear_fp8():
    need(40)
    N, D = (1 << 29) + 77, 16
    x, sx = km.kmeans_quantize(values(1 << 20, D))
    X = x.view(torch.uint8).repeat((N >> 20) + 1, 1)[:N].view(torch.float8_e4m3fn)
    S = sx.repeat((N >> 20) + 1, 1)[:N]
    W, sw = km.kmeans_quantize(values(1, D), rows=128)
    Y = km.kmeans_linear_fp8(X, S, W, sw)
    want = km.kmeans_linear_fp8(x, sx, W, sw)
    for p in parts(N, 1 << 20):
        if p.stop - p.start > 16:
            assert torch.equal(Y[p], want[:p.stop - p.start]), p


def test_sample():
    need(10)
    N, K = (1 << 21) + 9, 300
    z = values(N, K) / 16
    u = torch.arange(N, device="cuda") % 997 / 997
    got = km.kmeans_sample(z, u, top_p=0.9)
    for p in parts(N, 1 << 20):
        assert torch.equal(got[p], km.kmeans_sample(z[p], u[p], top_p=0.9)), p
