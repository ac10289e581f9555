"""Captured calls and the stream's workspace (HIP, through the public binding):
a graph keeps the scratch it was captured with while later calls on the stream
need more, and a capture may be a stream's first call.  Every replay is
compared with an eager call, bit for bit."""

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
    return torch.device("cuda:0")


def rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF).cuda()


def labels(N, K, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-1, K, (N,), generator=g).cuda()


def call(a):
    """The sort path, split products with operands laid out anew, and the
    clipping of a list too long for one launch: all of their scratch."""
    dC = km.kmeans_lookup_grad(a["dY"], a["lab"], 100)
    grads = km.kmeans_linear_grad(a["G"], a["dY"], a["W"])
    parts = a["dY"].view(-1).split(a["dY"].numel() // 100)
    norm, clipped = km.kmeans_clip_gradients(parts, 0.5, out=a["out"])
    return [dC, *grads, norm, clipped[0].clone(), clipped[99].clone()]


def inputs(seed, N=1500):
    return dict(dY=rand((N, 24), seed), lab=labels(N, 100, seed + 1), G=rand((N, 17), seed + 2),
                W=rand((17, 24), seed + 3, 0.1),
                out=[torch.empty(N * 24 // 100, dtype=BF, device="cuda") for _ in range(100)])


def replay_and_compare(g, args, got, s, between):
    for i in range(4):
        new = inputs(400 + 10 * i)
        for k in ("dY", "lab", "G", "W"):
            args[k].copy_(new[k])
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
            got_now = [t.clone() for t in got]
            between(i)
        s.synchronize()
        want = call(new)
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(got_now, want)):
            assert torch.equal(a, b), (i, j)


@pytest.mark.parametrize("warm", [True, False])
def test_replays_after_the_workspace_grew(warm):
    args = inputs(10)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    if warm:
        with torch.cuda.stream(s):
            call(args)
        s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = call(args)
    big = {i: inputs(700 + i, 40000 << i) for i in range(3)}
    want = {i: call(big[i])[:4] for i in big}
    torch.cuda.synchronize()

    def between(i):                       # larger eager calls on the same stream
        if i in big:
            res = call(big[i])[:4]
            s.synchronize()
            for a, b in zip(res, want[i]):
                assert torch.equal(a, b), i

    replay_and_compare(g, args, got, s, between)
    del g
    km.kmeans_release_workspace(stream=s)
    with torch.cuda.stream(s):            # the stream takes a new workspace
        again = call(args)
    s.synchronize()
    for a, b in zip(again, call(args)):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    km.kmeans_release_workspace(stream=s)
