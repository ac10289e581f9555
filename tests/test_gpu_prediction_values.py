"""Operators of label prediction (HIP, through the public binding): results that
their definitions settle to the last bit, or to a bound taken block by block."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
km = pytest.importorskip("means_nearest_centroid_amd")
import prediction_reference as ref  # noqa: E402

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a visible GPU")
    km.load_library()
    return torch.device("cuda:0")


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


# ---- quantisation: the correctly rounded quotient, rounded to e4m3 -----------

def quantized(x, rows):
    """(bits of e4m3(v / s), s) of the definition, on the CPU."""
    x = x.detach().cpu().float()
    N, D = x.shape
    n, b = -(-N // rows), -(-D // 128)
    wide = torch.nn.functional.pad(x, (0, b * 128 - D, 0, n * rows - N)).view(n, rows, b, 128)
    most = wide.abs().amax((1, 3))
    s = torch.where(most == 0, 1.0, (most / 448).clamp(min=2.0 ** -126))
    q = (wide / s[:, None, :, None]).view(n * rows, b * 128)[:N, :D]
    return q.to(FP8).view(torch.uint8), s


def check_quotients(X, rows):
    q, s = quantized(X, rows)
    Q, S = km.kmeans_quantize(X, rows=rows)
    assert torch.equal(S.cpu().nan_to_num(nan=-1.0), s.nan_to_num(nan=-1.0))
    got = Q.view(torch.uint8).cpu()
    bad = (got != q) & ~((got & 0x7f == 0x7f) & (q & 0x7f == 0x7f))      # NaN of either sign
    assert not bad.any(), (f"{int(bad.sum())} of {q.numel()} values, first at "
                           f"{torch.nonzero(bad)[0].tolist()}: {got[bad][0]:#x}, {q[bad][0]:#x}")


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_quotients_are_correctly_rounded(dtype, rows):
    """Of 16-bit values one quotient of a few hundred lies on a tie of e4m3."""
    for seed, scale in enumerate((1.0, 3e-5, 900.0)):
        check_quotients(rand((2000, 640), dtype, seed, scale), rows)
    check_quotients(rand((300, 77), dtype, 5), rows)


def ties():
    """All e4m3 values, and those halfway between two of them."""
    v = torch.arange(0x7f, dtype=torch.uint8).view(FP8).float()
    return torch.cat([v, (v[1:] + v[:-1]) / 2])


@pytest.mark.parametrize("power", [-126, -125, -110, -92, -91, -90, -89, -60, 0, 3, 100, 118])
def test_quotients_at_ties(power):
    """Scales of 16 bits, so that the products of ties with them are exact in
    fp32, and their neighbours on either side; the largest value sets the scale.
    (The neighbour of zero on its own side is a NaN here: so is its whole block.)"""
    g = torch.Generator().manual_seed(power + 200)
    N = 200
    s = (1 + torch.randint(0, 1 << 15, (N, 1), generator=g) * 2.0 ** -15).double() * 2.0 ** power
    t = ties().double()
    x = (s * t * torch.where(torch.rand(N, len(t), generator=g) < 0.5, -1.0, 1.0)).float()
    assert power < -100 or torch.equal(x.double().abs(), s * t)
    x = torch.cat([x, torch.nextafter(x, torch.tensor(0.0)),
                   torch.nextafter(x, torch.sign(x) * torch.inf)], 1)
    x = torch.where(x.abs() > (448 * s).float(), (448 * s).float() * x.sign(), x)
    # blocks of 128 with the scale's own largest value in each
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % 127)).view(N, -1, 127)
    x = torch.cat([x, (448 * s).float()[:, :, None].expand(-1, x.shape[1], 1)], 2)
    check_quotients(x.reshape(N, -1).cuda(), 1)


def test_quotients_of_zeros_and_infinities():
    x = torch.zeros(4, 130)
    x[0, ::2] = -0.0
    x[1, 3], x[1, 4], x[1, 5] = -7.0, 0.0, -0.0
    x[2, 9], x[2, 10:20] = torch.inf, -3.0
    Q, s = km.kmeans_quantize(x.cuda())
    bits = Q.view(torch.uint8).cpu()
    assert (bits[0, ::2] == 0x80).all() and (bits[0, 1::2] == 0).all()
    assert bits[1, 3:6].tolist() == [0xfe, 0, 0x80]
    assert s[2, 0].isinf() and bits[2, 9] & 0x7f == 0x7f
    assert (bits[2, 10:20] == 0x80).all() and (bits[2, 20:128] == 0).all()


@pytest.mark.parametrize("D", [128, 300, 4096])
@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_norm_quotients(D, dtype):
    """Rows of two magnitudes only, whose mean square is a power of 4: r and y are
    exact, and the 8-bit output is the definition's to the last bit."""
    N = 40
    g = torch.Generator().manual_seed(D)
    x = torch.where(torch.rand(N, D, generator=g) < 0.5, -2.0, 2.0)
    for _ in range(10):
        w = torch.randn(D, generator=g).to(dtype)
        Q, s = km.kmeans_rms_norm(x.to(dtype).cuda(), w.cuda(), eps=0.0, quantize=True)
        q, want = quantized(x / 2 * w.float(), 1)
        assert torch.equal(s.cpu(), want) and torch.equal(Q.view(torch.uint8).cpu(), q)


# ---- sampling ----------------------------------------------------------------

def rows_of(N, **kw):
    full = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    full.update({k: v.cpu().numpy() if isinstance(v, torch.Tensor) else v for k, v in kw.items()})
    return {k: np.broadcast_to(np.asarray(v), (N,)) for k, v in full.items()}


def check_draws(z, u, **kw):
    got = km.kmeans_sample(z, u, **kw)
    ref.check_sample(got, ref.sample(z, u.cpu().numpy(), **rows_of(len(z), **kw)))
    return got


def uniforms(N, seed):
    return torch.rand(N, generator=torch.Generator().manual_seed(seed)).cuda()


@pytest.mark.parametrize("K", [300, 9000, 40000, 70000])
@pytest.mark.parametrize("masked", [0, 200, 4096, 5000])
def test_settings_that_limit_nothing(K, masked):
    """NaN, and values beyond the range where nothing is cut, as array values,
    also where the row's first labels are all masked."""
    N = 16
    z = rand((N, K), F32, K, 0.5)
    z[:, :min(masked, K - 50)] = -torch.inf
    z[3, :min(masked, K - 50)] = torch.nan
    u = uniforms(N, 7)
    want = check_draws(z, u)
    for least in (torch.nan, -1.0, -0.0, 0.0):
        for p in (torch.nan, 1.0, 7.0):
            for k in (0, -3, K, K + 5):
                got = km.kmeans_sample(z, u, min_p=torch.full((N,), least).cuda(),
                                       top_p=torch.full((N,), p).cuda(),
                                       top_k=torch.full((N,), k, dtype=torch.int32).cuda())
                assert torch.equal(got, want), (least, p, k)


@pytest.mark.parametrize("K", [6000, 20000])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_at_the_ends_of_the_range(K, dtype, sign):
    """Finite logits up to the type's last, at a temperature that tells them
    apart: their distances and bins reach past the range."""
    N = 24
    g = torch.Generator().manual_seed(K)
    last = torch.finfo(dtype).max
    z = sign * last * (1 - 0.12 * torch.rand(N, K, generator=g))
    z[:, 4500] = last if sign > 0 else 0.85 * -last        # the largest, behind the first ones
    z[:, :4096] = torch.where(z[:, :4096] > 0.95 * last, 0.9 * last, z[:, :4096])
    z[4, 1::2] = -torch.inf
    z = z.to(dtype).cuda()
    u = uniforms(N, 3)
    u[0], u[1], u[2] = 0.0, 1e-3, 1e-4
    for kw in (dict(), dict(top_p=0.02), dict(top_p=0.9), dict(top_k=900), dict(top_p=0.9, min_p=0.1),
               dict(min_p=1e-6)):
        check_draws(z, u, temperature=2.0 ** 120, **kw)


def near_ties(rows, of, rest, seed):
    """Rows of `of` labels of two values, `rest` far below, and a temperature for
    each, so that half of the weight ends as closely at a whole number of labels
    as the roundings to 2^-43 of a weight see: (logits, temperatures)."""
    rng = np.random.default_rng(seed)
    wide, eight = np.longdouble, 8
    z, temps = np.full((rows, of + rest), -200.0, np.float32), np.empty(rows, np.float32)
    for r in range(0, rows, eight):
        first = int(rng.integers(of // 3, of // 2))
        t = rng.uniform(0.6, 1.9, 200000).astype(np.float32)
        n = rng.integers(first // 2 + of // 50 + 1, first, len(t))
        w = (2 * n - first).astype(wide) / wide(of - first)
        d = (-np.log(w) * t.astype(wide)).astype(np.float32)
        half = (first + (of - first) * np.exp(-d.astype(wide) / t.astype(wide))) / 2
        for i, best in enumerate(np.argsort(np.abs(half / n - 1))[:eight]):
            at = rng.permutation(of + rest)
            z[r + i, at[:first]], z[r + i, at[first:of]] = 0.0, -d[best]
            temps[r + i] = t[best]
    return torch.from_numpy(z).cuda(), torch.from_numpy(temps).cuda()


@pytest.mark.parametrize("of,rest,top_k", [(12000, 0, 0), (400, 11600, 400), (400, 69600, 400),
                                           (300, 7000, 300), (70000, 0, 0)])
def test_labels_do_not_depend_on_the_batch(of, rest, top_k):
    """Border cases one by one, and all in one call of more rows than the GPU has
    room for at once: the same labels."""
    N = 640
    z, t = near_ties(128, of, rest, of + rest)
    z, t = z.repeat(N // 128, 1), t.repeat(N // 128)
    u = torch.full((N,), 0.5).cuda()
    for kw in (dict(top_k=top_k), dict(top_k=top_k, top_p=0.5)):
        got = km.kmeans_sample(z, u, temperature=t, **kw)
        assert torch.equal(got, got[:128].repeat(N // 128))
        for n in (1, 40):
            for i in range(0, 128, n):
                few = km.kmeans_sample(z[i:i + n], u[:n], temperature=t[i:i + n], **kw)
                assert torch.equal(few, got[i:i + len(few)]), (kw, n, i)


# ---- the norm's weight gradient over many rows --------------------------------

def check_dw(dY, H, w, exact):
    """dw against `exact`, whose terms all have one sign.  At most 44 terms, then
    16 such sums, then eight of those in pairs are added in fp32, all that follows
    in fp64: 61 roundings, one to spare, one of a partial sum, one of the term's
    product, and of r: each square, the sum of D of them (8 + log2(D / 8) in a
    row), the division, eps and the root halve, then the reciprocal."""
    _, dw = km.kmeans_rms_norm_grad(dY, H, w)
    D = H.shape[1]
    bound = (63 + 1 + 1 + (9 + np.ceil(np.log2(max(1, D / 8))) + 2) / 2 + 2) * 2.0 ** -24
    got = dw.double().cpu()
    off = ((got - exact) / exact).abs().max()
    assert off <= bound + 2.0 ** -24, f"{float(off):.3g}, {float(bound):.3g}"


@pytest.mark.parametrize("N,D", [((1 << 26) + 5, 2), ((1 << 22) + 1, 60), (3_000_001, 129),
                                 (400_000, 1000), (70_003, 8200), (150_000, 16392)])
def test_dw_of_many_rows(N, D):
    """Every row the same, for several such rows: the roundings of each addition
    then tend to one side, and in fp32 alone the error grows with the rows."""
    g = torch.Generator().manual_seed(D)
    w = torch.ones(D).cuda()
    eps = float(np.float32(1e-6))
    for _ in range(3):
        h, dy = (torch.rand(D, generator=g) + 0.25 for _ in range(2))
        H, dY = torch.empty(N, D, device="cuda"), torch.empty(N, D, device="cuda")
        H.copy_(h), dY.copy_(dy)
        r = 1 / torch.sqrt(h.double().square().mean() + eps)
        check_dw(dY, H, w, N * (dy.double() * h.double() * r))
        del H, dY


@pytest.mark.parametrize("N,D", [(2_000_003, 40), (100_000, 700)])
def test_dw_of_many_rows_of_any_kind(N, D):
    """Against a sum in fp64 on the GPU; terms of one sign."""
    g = torch.Generator(device="cuda").manual_seed(N)
    H = torch.rand(N, D, generator=g, device="cuda") + 0.01
    dY = torch.rand(N, D, generator=g, device="cuda")
    r = 1 / torch.sqrt(H.double().square().mean(1, keepdim=True) + float(np.float32(1e-6)))
    exact = (dY.double() * H.double() * r).sum(0).cpu()
    check_dw(dY, H, torch.ones(D).cuda(), exact)


def test_top_k_of_any_integer():
    """More than 32 bits hold is more than all labels; below zero is refused."""
    z, u = rand((40, 900), F32, 3, 2.0), uniforms(40, 5)
    want = km.kmeans_sample(z, u)
    for k in (900, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 3, 2 ** 32 + 1, 2 ** 40 + 2):
        assert torch.equal(km.kmeans_sample(z, u, top_k=k), want), k
    for k in (-1, -2 ** 31, -2 ** 31 - 1, -2 ** 32 + 1):
        with pytest.raises(km.KmeansError, match="top_k"):
            km.kmeans_sample(z, u, top_k=k)


def test_quantize_of_any_shape():
    """Rows of [..., D], as the norm and the product beside it take them."""
    x = rand((2, 3, 5, 200), BF, 1)
    want, s = km.kmeans_quantize(x.view(-1, 200))
    Q, t = km.kmeans_quantize(x)
    assert Q.shape == x.shape and t.shape == (2, 3, 5, 2)
    assert torch.equal(Q.view(torch.uint8).view(-1, 200), want.view(torch.uint8))
    assert torch.equal(t.view(-1, 2), s)
    out, scales = torch.empty_like(Q), torch.empty_like(t)
    got = km.kmeans_quantize(x, out=out, scales=scales)
    assert got[0] is out and got[1] is scales
    assert torch.equal(out.view(torch.uint8), Q.view(torch.uint8)) and torch.equal(scales, t)
    assert km.kmeans_quantize(x[:0])[1].shape == (0, 3, 5, 2)
    W, sw = km.kmeans_quantize(rand((70, 200), BF, 2), rows=128)
    assert km.kmeans_linear_fp8(Q, t, W, sw).shape == (2, 3, 5, 70)
    with pytest.raises(ValueError, match="2-D"):
        km.kmeans_quantize(x, rows=128)
    with pytest.raises(ValueError, match="evenly spaced"):
        km.kmeans_quantize(x.transpose(1, 2))


def test_dw_of_many_rows_in_a_graph():
    """The workspace's partial sums begin anew in every replay."""
    N, D = 800_000, 40
    H, dY, w = rand((N, D), BF, 1), rand((N, D), BF, 2), rand((D,), BF, 3)
    want = km.kmeans_rms_norm_grad(dY, H, w)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = km.kmeans_rms_norm_grad(dY, H, w)
    for i in range(4):
        with torch.cuda.stream(s):
            g.replay()
            now = [t.clone() for t in got]
            km.kmeans_rms_norm_grad(dY[:N - 7 * i], H[:N - 7 * i], w)
        s.synchronize()
        for a, b in zip(now, want):
            assert torch.equal(a, b), i
    del g
    km.kmeans_release_workspace(stream=s)
