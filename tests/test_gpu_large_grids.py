"""Sizes whose launches have 2^32 threads or more (HIP, through the public
binding): the operators take every size that their checks accept."""

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


def test_lookup_gradient_of_a_table_past_2_to_the_30_rows():
    need(8)
    N, K = 1000, (1 << 30) + 70
    lab = torch.arange(N, dtype=torch.int64) * (K // N) + 3
    lab[-1] = K - 1
    dY = (torch.arange(N).to(BF) % 50 + 1).reshape(N, 1).cuda()
    out = torch.full((K, 1), float("nan"), dtype=BF, device="cuda")
    km.kmeans_lookup_grad(dY, lab.cuda(), K, out=out)
    assert torch.equal(out[lab.cuda()], dY)
    assert int(torch.count_nonzero(out)) == N                     # NaN would count


def test_lookup_of_2_to_the_33_pieces():
    need(150)
    N, D, K = (1 << 24) + 3, 4096, 5
    C = torch.randn(K, D, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    lab = (torch.arange(N, dtype=torch.int32, device="cuda") * 7) % (K + 1)      # K: stray
    out = km.kmeans_lookup(C, lab)
    rows = torch.cat([C, torch.zeros(1, D, dtype=BF, device="cuda")])
    for i in range(0, N, 1 << 18):
        assert torch.equal(out[i:i + (1 << 18)], rows[lab[i:i + (1 << 18)].long()]), i


def test_linear_of_2_to_the_30_unaligned_rows():
    """2^23 tiles of 512 threads each: rows that are taken as they lie."""
    need(80)
    N, D = (1 << 30) + 77, 15
    X = torch.zeros((N, D), dtype=BF, device="cuda")
    X[:, 7] = (torch.arange(N, dtype=torch.int32, device="cuda") % 251).to(BF)
    W = torch.ones((1, D), dtype=BF, device="cuda")
    W[0, 7] = 2.0
    Y = torch.full((N, 1), float("nan"), dtype=BF, device="cuda")
    km.kmeans_linear(X, W, out=Y)
    assert torch.equal(Y[:, 0], X[:, 7] * 2)


def test_norms_of_2_to_the_28_rows():
    need(20)
    K = (1 << 28) + 21
    C = torch.ones((K, 16), dtype=BF, device="cuda")
    C[-5:] = 2.0
    norms = torch.full((K,), float("nan"), device="cuda")
    km.kmeans_centroid_norms(C, norms)
    assert bool((norms[:-5] == 16.0).all()) and bool((norms[-5:] == 64.0).all())
