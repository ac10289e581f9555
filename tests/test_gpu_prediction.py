"""Operators of label prediction (HIP, through the public binding) against their
definitions in fp64, at the sizes where each can go wrong.  Bounds and their
derivation: ``prediction_reference``."""

import math

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


def rows_in(t, extra, shift=0, fill=7.0):
    """The same values as rows of a wider buffer, `shift` elements in."""
    wide = torch.full((t.shape[0], t.shape[1] + extra + shift), fill, device=t.device).to(t.dtype)
    v = wide[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return v


def beside(v, shift):
    """What lies beside the rows of a view made by rows_in."""
    wide = v._base
    return torch.cat([wide[:, :shift], wide[:, shift + v.shape[1]:]], 1).float()


# ---- norm ------------------------------------------------------------------

NORM_SIZES = [(1, 1), (1, 8), (3, 7), (40, 16), (5, 128), (17, 129), (64, 256), (33, 257), (9, 512),
              (130, 1000), (7, 1024), (12, 2048), (3, 4096), (5, 4099), (2, 8192), (3, 16384),
              (2, 16385), (1, 40003)]


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("N,D", NORM_SIZES)
def test_rms_norm(N, D, dtype):
    X, R, w = rand((N, D), dtype, N + D), rand((N, D), dtype, D), rand((D,), dtype, 3)
    for weight, residual in ((w, R), (None, None), (w, None)):
        y, yerr, h, herr = ref.rms_norm(X, weight, residual)
        got = km.kmeans_rms_norm(X, weight, residual)
        if residual is not None:
            got, H = got
            ref.check(H, h, herr, "H")
        ref.check(got, y, ref.rounded(y, yerr, dtype), "Y")
        got = km.kmeans_rms_norm(X, weight, residual, quantize=True)
        assert got[0].dtype == FP8 and got[1].shape == (N, -(-D // 128))
        ref.check_quantized(got[0], got[1], y, yerr, 1, "Q")
        if residual is not None:
            ref.check(got[2], h, herr, "H")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [72, 1000, 17000])
@pytest.mark.parametrize("extra,shift", [(8, 0), (1, 0), (5, 3)])
def test_rms_norm_strides(D, extra, shift, dtype):
    N = 5
    X, R, w = rand((N, D), dtype, 1), rand((N, D), dtype, 2), rand((D,), dtype, 3)
    want, H = km.kmeans_rms_norm(X, w, R)
    q, s, _ = km.kmeans_rms_norm(X, w, R, quantize=True)
    x, r = rows_in(X, extra, shift), rows_in(R, extra + 2, shift)
    out, total = (rows_in(torch.zeros_like(X), extra, shift) for _ in range(2))
    km.kmeans_rms_norm(x, w, r, out=out, sum=total)
    assert torch.equal(out, want) and torch.equal(total, H)
    out8 = rows_in(torch.zeros_like(X).to(FP8), extra, shift)
    scales = rows_in(torch.zeros_like(s), extra, shift)
    km.kmeans_rms_norm(x, w, r, quantize=True, out=out8, scales=scales, sum=total)
    assert torch.equal(out8.float(), q.float()) and torch.equal(scales, s)
    for v in (out, total, out8, scales):
        assert (beside(v, shift) == 7).all()
    # the sum in the residual's place, the output in the input's
    x, r = X.clone(), R.clone()
    y, total = km.kmeans_rms_norm(x, w, r, out=x, sum=r)
    assert y is x and total is r and torch.equal(x, want) and torch.equal(r, H)
    x = X.clone()
    km.kmeans_rms_norm(x, w, R, sum=x, quantize=True)
    assert torch.equal(x, H)


def test_rms_norm_shapes():
    X, R, w = rand((2, 3, 5, 64), BF, 1), rand((2, 3, 5, 64), BF, 2), rand((64,), BF, 3)
    Y, H = km.kmeans_rms_norm(X, w, R)
    flat, _ = km.kmeans_rms_norm(X.view(-1, 64), w, R.view(-1, 64))
    assert Y.shape == H.shape == X.shape and torch.equal(Y.view(-1, 64), flat)
    Q, s, _ = km.kmeans_rms_norm(X, w, R, quantize=True)
    assert Q.shape == X.shape and s.shape == (2, 3, 5, 1)
    Y, H = km.kmeans_rms_norm(X[:0], w, R[:0])
    assert Y.shape == (0, 3, 5, 64)
    Q, s = km.kmeans_rms_norm(X[:0], quantize=True)
    assert s.shape == (0, 3, 5, 1)


@pytest.mark.parametrize("D", [40, 300, 5000, 20000])
def test_rms_norm_of_special_values(D):
    """Values that are not finite stay in their row, and in their block."""
    X = rand((6, D), F32, 5)
    want = km.kmeans_rms_norm(X)
    q, s = km.kmeans_rms_norm(X, quantize=True)
    Z = X.clone()
    Z[1, D // 2] = math.nan
    Z[3, 0] = math.inf
    Z[4] = 0
    got = km.kmeans_rms_norm(Z)
    q2, s2 = km.kmeans_rms_norm(Z, quantize=True)
    for i in (0, 2, 5):
        assert torch.equal(got[i], want[i]) and torch.equal(s2[i], s[i])
        assert torch.equal(q2[i].float(), q[i].float())
    assert got[1].isnan().all()
    assert got[3, 0].isnan() and (got[3, 1:] == 0).all()
    assert (got[4] == 0).all() and (s2[4] == 1).all() and (q2[4].float() == 0).all()
    assert s2[1].isnan().all()
    assert s2[3, 0].isnan() and (s2[3, 1:] == 1).all()
    Z[4] = 0
    assert km.kmeans_rms_norm(Z, eps=0.0)[4].isnan().all()


def test_rms_norm_of_small_and_large_values():
    X = torch.full((3, 200), 1e-30, dtype=F32, device="cuda")
    X[1] = 1e18
    X[2] = 1e-42
    got = km.kmeans_rms_norm(X, eps=0.0)
    assert torch.allclose(got[1], torch.ones(200, device="cuda"), rtol=1e-5)
    Q, s = km.kmeans_quantize(X)
    assert (s[2] == 2.0 ** -126).all()                     # the least scale
    assert torch.allclose(Q.float()[:2] * s.repeat_interleave(128, 1)[:2, :200], X[:2], rtol=1e-6)
    v = Q.float()[2, 0] * 2.0 ** -126
    assert abs(float(v) - 1e-42) <= 2.0 ** -126 * 2.0 ** -10


def test_rms_norm_past_32_bit_offsets():
    N, D = 2_200_000, 1024
    X = torch.empty((N, D), dtype=BF, device="cuda")
    X[-64:] = rand((64, D), BF, 3)
    X[:64] = rand((64, D), BF, 4)
    w = rand((D,), BF, 5)
    Y = km.kmeans_rms_norm(X, w)
    assert torch.equal(Y[-64:], km.kmeans_rms_norm(X[-64:], w))
    assert torch.equal(Y[:64], km.kmeans_rms_norm(X[:64], w))
    Q, s = km.kmeans_quantize(X)
    q, t = km.kmeans_quantize(X[-64:])
    assert torch.equal(Q[-64:].view(torch.uint8), q.view(torch.uint8)) and torch.equal(s[-64:], t)
    dX, _ = km.kmeans_rms_norm_grad(Y, X, w)
    assert torch.equal(dX[-64:], km.kmeans_rms_norm_grad(Y[-64:], X[-64:], w)[0])


# ---- norm gradient ---------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("N,D", NORM_SIZES + [(2000, 64), (3001, 130), (1025, 520), (1100, 2100)])
def test_rms_norm_grad(N, D, dtype):
    H, dY, dH = rand((N, D), dtype, N + D), rand((N, D), dtype, D), rand((N, D), dtype, 9)
    w = rand((D,), dtype, 3)
    for weight, skip in ((w, dH), (w, None), (None, dH)):
        want = ref.rms_norm_grad(dY, H, weight, skip)
        dX, dw = km.kmeans_rms_norm_grad(dY, H, weight, dH=skip)
        ref.check(dX, *want["dX"], "dX")
        if weight is None:
            assert dw is None
        else:
            ref.check(dw, *want["dw"], "dw")
    alone, none = km.kmeans_rms_norm_grad(dY, H, w, dH=dH, need_dw=False)
    assert none is None and torch.equal(alone, km.kmeans_rms_norm_grad(dY, H, w, dH=dH)[0])


@pytest.mark.parametrize("D", [72, 1000, 17000])
def test_rms_norm_grad_strides_and_shapes(D):
    N = 37
    H, dY, dH, w = (rand(s, BF, i) for i, s in enumerate([(N, D)] * 3 + [(D,)]))
    dX, dw = km.kmeans_rms_norm_grad(dY, H, w, dH=dH)
    for extra, shift in ((8, 0), (3, 1)):
        got = km.kmeans_rms_norm_grad(rows_in(dY, extra, shift), rows_in(H, extra + 2, shift), w,
                                      dH=rows_in(dH, extra + 4, shift))
        assert torch.equal(got[0], dX) and torch.equal(got[1], dw)
    got = km.kmeans_rms_norm_grad(dY[:36].view(3, 12, D), H[:36].view(3, 12, D), w)
    assert got[0].shape == (3, 12, D)
    none, zero = km.kmeans_rms_norm_grad(dY[:0], H[:0], w)
    assert none.shape == (0, D) and (zero == 0).all()


def test_rms_norm_grad_agrees_with_differences():
    """Of the fp32 forward pass: a step of 2^-6 changes the loss by its slope, up
    to the loss's third derivative (below 60 here, a factor 1/6 2^-12) and the
    roundings of its D terms (2^-23 of their magnitudes, over the step)."""
    D = 96
    g = torch.Generator().manual_seed(8)
    X, w, dY = (torch.randn(s, generator=g).cuda() for s in ((1, D), (D,), (1, D)))
    loss = lambda x, v: float((km.kmeans_rms_norm(x, v).double() * dY.double()).sum())  # noqa: E731
    dX, dw = km.kmeans_rms_norm_grad(dY, X, w)
    h = 2.0 ** -6
    size = float((km.kmeans_rms_norm(X, w) * dY).abs().sum())
    bound = 10 * h * h + 2 * (ref.depth(D) + 8) * ref.EPS * size / h
    for j in range(0, D, 7):
        e = torch.zeros_like(X)
        e[0, j] = h
        assert abs((loss(X + e, w) - loss(X - e, w)) / (2 * h) - float(dX[0, j])) < bound
        v = (loss(X, w + e[0]) - loss(X, w - e[0])) / (2 * h)
        assert abs(v - float(dw[j])) < bound


# ---- quantisation ----------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("N,D", [(1, 1), (1, 128), (3, 7), (128, 128), (127, 129), (130, 1000),
                                 (257, 260), (1000, 77)])
def test_quantize(N, D, rows, dtype):
    X = rand((N, D), dtype, N + D) * torch.exp(rand((N, 1), F32, 4)).to(dtype)
    x = ref.cpu64(X)
    Q, s = km.kmeans_quantize(X, rows=rows)
    assert s.shape == (-(-N // rows), -(-D // 128))
    ref.check_quantized(Q, s, x, torch.zeros_like(x), rows)
    v, t = rows_in(Q, 5, 3), rows_in(s, 1)
    v.zero_(), t.zero_()
    km.kmeans_quantize(rows_in(X, 3, 1), rows=rows, out=v, scales=t)
    assert torch.equal(v.float(), Q.float()) and torch.equal(t, s)
    assert (beside(v, 3) == 7).all() and (beside(t, 0) == 7).all()


def test_quantize_of_special_values():
    X = rand((130, 300), BF, 1)
    want, s = km.kmeans_quantize(X)
    X[4, 10] = math.nan
    X[5, 290] = -math.inf
    X[6, 128:256] = 0
    got, t = km.kmeans_quantize(X)
    assert t[4, 0].isnan() and torch.equal(t[4, 1:], s[4, 1:])
    assert t[5, 2].isinf() and torch.equal(t[5, :2], s[5, :2])
    assert (got.float()[5] * t[5].repeat_interleave(128)[:300]).isnan().any()
    assert t[6, 1] == 1 and (got.float()[6, 128:256] == 0).all()
    keep = torch.ones(130, dtype=torch.bool)
    keep[[4, 5, 6]] = False
    assert torch.equal(got[keep].float(), want[keep].float())
    block, t = km.kmeans_quantize(X, rows=128)
    assert t[0, 0].isnan() and t[0, 2].isinf() and t[1].isfinite().all()


# ---- linear on 8-bit operands ----------------------------------------------

def operands(N, D, F, seed):
    X, sx = km.kmeans_quantize(rand((N, D), F32, seed) * torch.exp(rand((N, 1), F32, seed + 1)))
    W, sw = km.kmeans_quantize(rand((F, D), F32, seed + 2, D ** -0.5), rows=128)
    return X, sx, W, sw


FP8_SIZES = [(1, 1, 1), (1, 16, 5), (2, 128, 16), (16, 129, 33), (3, 4096, 100), (16, 1000, 2000),
             (17, 16, 16), (17, 128, 128), (40, 100, 200), (129, 257, 300), (200, 256, 129),
             (64, 2048, 512), (300, 384, 640), (513, 515, 1001), (600, 1040, 260), (1024, 64, 1000),
             (2600, 272, 2600)]


@pytest.mark.parametrize("N,D,F", FP8_SIZES)
@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_linear_fp8(N, D, F, dtype):
    X, sx, W, sw = operands(N, D, F, N + D + F)
    b, R = rand((F,), dtype, 5), rand((N, F), dtype, 6)
    for bias, residual, activation in ((None, None, "none"), (b, R, "gelu")):
        got = km.kmeans_linear_fp8(X, sx, W, sw, bias, residual, activation, dtype=dtype)
        assert got.dtype == dtype and got.shape == (N, F)
        ref.check(got, *ref.linear_fp8(X, sx, W, sw, bias, residual, activation, dtype))


@pytest.mark.parametrize("activation", list(km.ACTIVATIONS))
@pytest.mark.parametrize("N", [5, 70])
def test_linear_fp8_activations(N, activation):
    X, sx, W, sw = operands(N, 300, 77, 3)
    b = rand((77,), BF, 5)
    got = km.kmeans_linear_fp8(X, sx, W, sw, b, None, activation)
    ref.check(got, *ref.linear_fp8(X, sx, W, sw, b, None, activation, BF))


@pytest.mark.parametrize("N", [7, 90])
def test_linear_fp8_strides_and_shapes(N):
    D, F = 272, 130
    X, sx, W, sw = operands(N, D, F, 11)
    R = rand((N, F), BF, 1)
    want = km.kmeans_linear_fp8(X, sx, W, sw, residual=R)
    for extra, shift in ((16, 0), (48, 16), (1, 0), (7, 5)):
        out = rows_in(torch.zeros_like(want), extra, shift)
        got = km.kmeans_linear_fp8(rows_in(X, extra, shift, math.nan), rows_in(sx, extra, shift),
                                   rows_in(W, extra, shift, math.nan), rows_in(sw, extra, shift),
                                   residual=rows_in(R, extra, shift), out=out)
        assert torch.equal(got, want)
        assert (beside(out, shift) == 7).all()
    assert torch.equal(km.kmeans_linear_fp8(X, sx, W, sw, residual=R, out=R), want)  # in its place
    X3, s3 = X.view(1, N, D), sx.view(1, N, -1)
    assert km.kmeans_linear_fp8(X3, s3, W, sw).shape == (1, N, F)
    assert km.kmeans_linear_fp8(X[:0], sx[:0], W, sw).shape == (0, F)


@pytest.mark.parametrize("N", [9, 70])
def test_linear_fp8_of_special_values(N):
    """A NaN or an infinite scale reaches its own rows or columns alone, also
    from the operand's last row."""
    X, sx, W, sw = operands(N, 300, 260, 4)
    want = km.kmeans_linear_fp8(X, sx, W, sw)
    sx2 = sx.clone()
    sx2[N - 1, 2] = math.nan
    got = km.kmeans_linear_fp8(X, sx2, W, sw)
    assert torch.equal(got[:-1], want[:-1]) and got[-1].isnan().all()
    sw2 = sw.clone()
    sw2[2, 0] = math.nan
    got = km.kmeans_linear_fp8(X, sx, W, sw2)
    assert torch.equal(got[:, :256], want[:, :256]) and got[:, 256:].isnan().all()
    W2 = W.float()
    W2[259, 299] = math.nan
    got = km.kmeans_linear_fp8(X, sx, W2.to(FP8), sw)
    assert torch.equal(got[:, :259], want[:, :259]) and got[:, 259].isnan().all()


# ---- sampling --------------------------------------------------------------

def settings_of(N, **kw):
    full = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    full.update(kw)
    return {k: np.broadcast_to(np.asarray(v), (N,)) for k, v in full.items()}


def check_sample(logits, u, what="", **kw):
    got = km.kmeans_sample(logits, u, **kw)
    host = {k: v.cpu().numpy() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    N = logits.shape[0]
    ref.check_sample(got, ref.sample(logits, u.cpu().numpy(), **settings_of(N, **host)),
                     f"{what} {kw if not any(isinstance(v, torch.Tensor) for v in kw.values()) else ''}")
    return got


def uniforms(N, seed):
    return torch.rand(N, generator=torch.Generator().manual_seed(seed)).cuda()


SETTINGS = [dict(), dict(temperature=0.7), dict(top_k=5), dict(top_k=40, top_p=0.9),
            dict(top_p=0.8, temperature=1.3), dict(min_p=0.05), dict(top_p=0.95, min_p=0.1),
            dict(top_k=100, top_p=0.5, min_p=0.01, temperature=2.0), dict(temperature=0.0),
            dict(top_k=1), dict(top_p=0.0), dict(min_p=1.0)]


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 2), (50, 17), (20, 255), (16, 1000), (9, 4096), (7, 4097),
                                 (5, 20011), (3, 70001), (2, 140000)])
def test_sample(N, K, dtype):
    logits = rand((N, K), dtype, N + K, 2.5)
    u = uniforms(N, K)
    for kw in SETTINGS:
        check_sample(logits, u, **kw)


@pytest.mark.parametrize("K", [300, 9000])
def test_sample_settings_by_row(K):
    N = 64
    g = torch.Generator().manual_seed(K)
    logits = rand((N, K), F32, K, 2.0)
    r = torch.rand(4, N, generator=g)
    kw = dict(temperature=torch.where(r[0] < 0.2, 0.0, 2 * r[0]).cuda(),
              top_k=(r[1] * 60).to(torch.int32).sub(10).cuda(),
              top_p=(r[2] * 1.3).cuda(), min_p=torch.where(r[3] < 0.5, 0.0, 0.2 * r[3]).cuda())
    check_sample(logits, uniforms(N, 3), **kw)
    one = km.kmeans_sample(logits, uniforms(N, 3), **kw)
    for name in kw:                       # one as an array, the others as numbers
        rest = dict(temperature=0.9, top_k=30, top_p=0.9, min_p=0.02)
        rest[name] = kw[name]
        check_sample(logits, uniforms(N, 4), **rest)
    out = torch.full((N,), 5, dtype=torch.int64, device="cuda")
    assert km.kmeans_sample(logits, uniforms(N, 3), out=out, **kw) is out
    assert torch.equal(out, one.long())


@pytest.mark.parametrize("K", [12, 700, 6000, 33000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sample_of_equal_logits(K, dtype):
    """Ties go to the lower index, wherever a limit or the draw cuts them: all
    equal; two values; every value many times."""
    N = 24
    u = uniforms(N, K)
    u[0], u[1], u[2] = 0.0, 1.0, 0.5
    g = torch.Generator().manual_seed(K)
    for z in (torch.full((N, K), -3.0), (torch.rand(N, K, generator=g) < 0.5).float() * 2,
              torch.randint(0, 9, (N, K), generator=g).float() / 4):
        z = z.to(dtype).cuda()
        for kw in (dict(), dict(top_k=K // 3), dict(top_k=K // 2, top_p=0.7), dict(top_p=0.3),
                   dict(min_p=0.5), dict(temperature=0.0), dict(top_p=0.9, min_p=0.9)):
            check_sample(z, u, **kw)


def test_sample_of_zeros_of_either_sign():
    z = torch.tensor([[-0.0, 0.0, -1.0], [0.0, -0.0, 0.0]]).cuda()
    assert km.kmeans_sample(z, torch.zeros(2).cuda()).tolist() == [0, 0]
    assert km.kmeans_sample(z, torch.zeros(2).cuda(), temperature=0.0).tolist() == [0, 0]
    assert km.kmeans_sample(z, torch.full((2,), 0.99).cuda(), top_k=2).tolist() == [1, 1]


@pytest.mark.parametrize("K", [100, 5000, 50000])
def test_sample_of_masked_logits(K):
    N = 12
    z = rand((N, K), F32, 4, 2.0)
    z[0] = -math.inf                                   # nothing left
    z[1] = math.nan
    z[2, 1:] = -math.inf                               # one left
    z[3, : K - 1] = math.nan
    z[4] = torch.finfo(F32).min                        # all of the type's lowest value
    z[5, ::2] = torch.finfo(F32).min
    z[6, 1::3] = -math.inf
    z[7, 3::5] = math.nan
    z[8, 7] = math.inf
    z[9, [5, 50]] = math.inf
    z[9, 60] = math.nan
    z[10] = -math.inf
    z[10, 90:95] = 1.0
    z[11, 11] = math.nan
    u = uniforms(N, 1)
    for kw in SETTINGS:
        got = check_sample(z, u, **kw)
        assert got[:2].tolist() == [-1, -1] and int(got[2]) == 0 and int(got[3]) == K - 1
        assert int(got[8]) == 7 and int(got[9]) in (5, 50)
    table = rand((K, 8), BF, 2)
    rows = km.kmeans_lookup(table, km.kmeans_sample(z, u))
    assert (rows[:2] == 0).all() and torch.equal(rows[2], table[0])


@pytest.mark.parametrize("K", [64, 8000])
def test_sample_of_any_uniform(K):
    z = rand((7, K), F32, 4)
    u = torch.tensor([0.0, -1.0, math.nan, 1.0, 2.0, math.inf, 1 - 2.0 ** -24]).cuda()
    got = check_sample(z, u)
    assert got[:3].tolist() == z[:3].argmax(1).tolist()
    assert got[3:6].tolist() == z[3:6].argmin(1).tolist()
    check_sample(z, u, top_k=9, top_p=0.7)


@pytest.mark.parametrize("K", [50, 10000])
def test_sample_of_extreme_temperatures(K):
    z = rand((6, K), F32, 4, 3.0)
    u = uniforms(6, 2)
    for t in (1e-45, 1e-30, 1e-3, 1e3, 1e30, math.inf):
        for kw in (dict(), dict(top_k=7), dict(top_p=0.5)):
            check_sample(z, u, temperature=t, **kw)


def test_sample_strides_and_shapes():
    z = rand((6, 515), BF, 4, 2.0)
    u = uniforms(6, 2)
    want = km.kmeans_sample(z, u, top_p=0.9)
    for extra, shift in ((5, 0), (8, 8), (3, 1)):
        assert torch.equal(km.kmeans_sample(rows_in(z, extra, shift, 90.0), u, top_p=0.9), want)
    got = km.kmeans_sample(z.view(2, 3, 515), u.view(2, 3), top_p=0.9)
    assert got.shape == (2, 3) and got.dtype == torch.int32 and torch.equal(got.view(-1), want)
    assert int(km.kmeans_sample(z[0], u[:1], top_p=0.9)) == int(want[0])
    assert km.kmeans_sample(z[:0], u[:0]).shape == (0,)


def test_sample_follows_its_distribution():
    """Evenly spaced uniforms hit each label as often as its weight says, within
    one (each border rounds one way)."""
    z = torch.tensor([0.3, 2.0, -1.0, 2.0, 0.0, 1.1]).cuda()
    n = 4096
    u = ((torch.arange(n, dtype=torch.float64) + 0.5) / n).float().cuda()
    got = km.kmeans_sample(z.expand(n, 6).contiguous(), u, temperature=0.8)
    want = torch.softmax(z.double().cpu() / float(np.float32(0.8)), 0) * n
    assert (torch.bincount(got.cpu().long(), minlength=6).double() - want).abs().max() <= 1


@pytest.mark.parametrize("N,K", [(6, 9000), (600, 8200), (6, 17000), (300, 17000), (6, 131072),
                                 (260, 66000)])
@pytest.mark.parametrize("spread", [0.02, 0.4, 3.0])
def test_sample_bins_of_many(N, K, spread):
    """Every kernel, with hundreds to thousands of labels in one bin."""
    logits = rand((N, K), F32, N + K, spread)
    u = uniforms(N, K)
    for kw in ({}, dict(top_p=0.7), dict(top_k=K // 3), dict(min_p=0.5)):
        check_sample(logits, u, **kw)


def test_sample_past_32_bit_offsets():
    N, K = 40000, 120000
    z = torch.zeros((N, K), dtype=BF, device="cuda")
    z[:, 5] = 1.0
    z[-3:] = rand((3, K), BF, 4, 2.0)
    u = uniforms(N, 2)
    got = km.kmeans_sample(z, u, top_k=20)
    assert torch.equal(got[-3:], km.kmeans_sample(z[-3:].clone(), u[-3:].clone(), top_k=20))
    assert int(got[:-3].max()) < 20


# ---- together --------------------------------------------------------------

def generate(m, x, h, u):
    """One step of a model that generates labels: the last hidden rows and the
    residual stream in, the labels and their rows of the table out."""
    q, s, h = km.kmeans_rms_norm(x, m["gain"], h, quantize=True)
    y = km.kmeans_linear_fp8(q, s, m["W1"], m["s1"], m["b1"], activation="silu")
    q, s, h = km.kmeans_rms_norm(y, m["gain"], h, quantize=True)
    logits = km.kmeans_linear_fp8(q, s, m["head"], m["sh"], dtype=F32)
    labels = km.kmeans_sample(logits, u, temperature=0.9, top_k=30, top_p=0.95)
    return h, logits, labels, km.kmeans_lookup(m["table"], labels)


def model(D=256, K=1000):
    table = rand((K, D), BF, 1)
    W1, s1 = km.kmeans_quantize(rand((D, D), BF, 2, D ** -0.5), rows=128)
    head, sh = km.kmeans_quantize(table, rows=128)
    return dict(table=table, gain=rand((D,), BF, 3), W1=W1, s1=s1, b1=rand((D,), BF, 4), head=head,
                sh=sh)


@pytest.mark.parametrize("N", [1, 16, 100])
def test_generation(N):
    """The chain against its definition, each step from what the last one gave."""
    m = model()
    x, h, u = rand((N, 256), BF, 5), rand((N, 256), BF, 6), uniforms(N, 7)
    h2, logits, labels, rows = generate(m, x, h, u)
    y, yerr, hh, herr = ref.rms_norm(x, m["gain"], h)
    q, s, h1 = km.kmeans_rms_norm(x, m["gain"], h, quantize=True)
    ref.check_quantized(q, s, y, yerr, 1)
    ref.check(h1, hh, herr)
    y1 = km.kmeans_linear_fp8(q, s, m["W1"], m["s1"], m["b1"], activation="silu")
    ref.check(y1, *ref.linear_fp8(q, s, m["W1"], m["s1"], m["b1"], None, "silu", BF))
    q, s, h1 = km.kmeans_rms_norm(y1, m["gain"], h1, quantize=True)
    assert torch.equal(h1, h2)
    ref.check(logits, *ref.linear_fp8(q, s, m["head"], m["sh"], None, None, "none", F32))
    ref.check_sample(labels, ref.sample(logits, u.cpu().numpy(),
                                        **settings_of(N, temperature=np.float32(0.9), top_k=30,
                                                      top_p=0.95)))
    assert torch.equal(rows, m["table"][labels.long()])


def test_generation_in_a_graph():
    """Captured once, replayed on new inputs with eager calls between, also after
    larger calls on the stream."""
    m = model()
    N = 100
    x, h, u = rand((N, 256), BF, 5), rand((N, 256), BF, 6), uniforms(N, 7)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = generate(m, x, h, u)
        grads = km.kmeans_rms_norm_grad(x, h, m["gain"])
    for i in range(4):
        x.copy_(rand((N, 256), BF, 50 + i)), h.copy_(rand((N, 256), BF, 60 + i))
        u.copy_(uniforms(N, 70 + i))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
            now = [t.clone() for t in (*got, *grads)]
            big = operands(300 << i, 515, 333, i)
            km.kmeans_linear_fp8(*big)
        s.synchronize()
        want = (*generate(m, x, h, u), *km.kmeans_rms_norm_grad(x, h, m["gain"]))
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(now, want)):
            assert torch.equal(a, b), (i, j)
    del g
    km.kmeans_release_workspace(stream=s)


def test_calls_on_two_streams_at_once():
    m = model()
    args = [(rand((70, 256), BF, 5 + i), rand((70, 256), BF, 6 + i), uniforms(70, i)) for i in (0, 9)]
    big = [operands(200, 515, 400, i) for i in (1, 2)]
    want = [[*generate(m, *a), km.kmeans_linear_fp8(*b), *km.kmeans_rms_norm_grad(a[0], a[1], m["gain"])]
            for a, b in zip(args, big)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = [*generate(m, *args[i]), km.kmeans_linear_fp8(*big[i]),
                          *km.kmeans_rms_norm_grad(args[i][0], args[i][1], m["gain"])]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    for s in streams:
        km.kmeans_release_workspace(stream=s)
