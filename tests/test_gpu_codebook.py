"""Codebook-training operators (HIP, through the public binding) against the
definitions in fp64, at the sizes where each can go wrong.  Bounds and their
derivation: ``codebook_reference``."""

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
km = pytest.importorskip("means_nearest_centroid_amd")
import codebook_reference as ref  # noqa: E402

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a visible GPU")
    km.load_library()
    return torch.device("cuda:0")


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def rows_in(t, extra, shift=0):
    """The same values as rows of a wider buffer, `shift` elements in."""
    wide = torch.full((t.shape[0], t.shape[1] + extra + shift), 7.0, dtype=t.dtype,
                      device=t.device)
    v = wide[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return v


def some_labels(N, K, seed, dtype=torch.int64, kind="uniform"):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        lab = torch.full((N,), K // 2)
    elif kind == "zipf":
        lab = (torch.rand(N, generator=g).pow(6) * K).long().clamp(max=K - 1)
    else:
        lab = torch.randint(0, K, (N,), generator=g)
    r = torch.rand(N, generator=g)
    lab[r < 0.03] = -1
    lab[r > 0.98] = K
    if dtype == torch.int64:
        lab[(r > 0.03) & (r < 0.035)] = (1 << 32) + 1        # would wrap to 1 in 32 bits
    return lab.to(dtype).cuda()


# ---- lookup ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("N,K,D", [(1, 1, 1), (1, 5, 4096), (7, 3, 3), (1000, 37, 8), (513, 70, 9),
                                   (4133, 275, 64), (777, 300, 127), (300, 45, 321), (2, 9, 8191)])
def test_lookup(N, K, D, dtype):
    C = rand((K, D), dtype, N + D)
    for index, scale in ((torch.int32, 1.0), (torch.int64, -1.7)):
        lab = some_labels(N, K, N, index)
        got = km.kmeans_lookup(C, lab, scale=scale).cpu()
        lc = lab.cpu().long()
        seen = (lc >= 0) & (lc < K)
        # one fp32 product and one rounding: the same bits
        want = (C.cpu().float()[lc.clamp(0, K - 1)] * scale).to(dtype)
        want[~seen] = 0
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), (N, K, D, index)


@pytest.mark.parametrize("extra,shift", [(8, 0), (1, 0), (5, 3), (16, 8)])
def test_lookup_strides_and_shapes(extra, shift):
    C = rows_in(rand((50, 72), BF, 1), extra, shift)
    lab = torch.randint(0, 50, (6, 7, 5), dtype=torch.int32).cuda()
    out = rows_in(torch.zeros(210, 72, dtype=BF, device="cuda"), extra, shift)
    base = out._base.clone()
    km.kmeans_lookup(C, lab.reshape(-1), out=out)
    assert torch.equal(out, C[lab.reshape(-1).long()])
    assert torch.equal(out._base[:, :shift], base[:, :shift])            # nothing beside the rows
    assert torch.equal(out._base[:, shift + 72:], base[:, shift + 72:])
    assert torch.equal(km.kmeans_lookup(C, lab), C[lab.long()])
    one = km.kmeans_lookup(C, lab[0, 0, 0].clone())                       # a single token
    assert one.shape == (72,) and torch.equal(one, C[int(lab[0, 0, 0])])
    assert km.kmeans_lookup(C, lab[:0].contiguous()).shape == (0, 7, 5, 72)


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("N,D", [(1, 8), (1, 9), (3, 11), (70, 8), (600, 16), (257, 129), (40, 1003),
                                 (2, 4100)])
@pytest.mark.parametrize("shift", [0, 1, 3, 7])
def test_lookup_into_rows_that_follow_one_another(N, D, dtype, shift):
    """Rows without gaps that start anywhere: each 16 bytes of the output may
    hold the end of one row and the beginning of the next; nothing before the
    first row or after the last is touched, and a stray row beside one of
    infinities stays zero."""
    C = rand((30, D), dtype, 51)
    C[7] = float("inf")
    lab = some_labels(N, 30, 52, torch.int32)
    lab[::3] = 7
    lab[1::5] = -1
    flat = torch.full((N * D + shift + 9,), 7.0, dtype=dtype, device="cuda")
    out = flat[shift:shift + N * D].view(N, D)
    km.kmeans_lookup(C, lab, scale=0.5, out=out)
    seen = ((lab >= 0) & (lab < 30)).unsqueeze(1)
    want = (C.float()[lab.long().clamp(0, 29)] * 0.5).to(dtype)
    want = torch.where(seen, want, torch.zeros_like(want))
    assert torch.equal(out, want)
    assert (flat[:shift] == 7).all() and (flat[shift + N * D:] == 7).all()


def test_lookup_of_special_values():
    C = torch.tensor([[float("inf"), -float("inf"), float("nan"), -0.0, 3e38]] * 3,
                     dtype=F32).cuda()
    got = km.kmeans_lookup(C, torch.tensor([0, -5, 2], dtype=torch.int32).cuda(), scale=2.0).cpu()
    assert torch.isinf(got[0, [0, 1, 4]]).all() and torch.isnan(got[0, 2])
    assert math.copysign(1.0, float(got[0, 3])) == -1.0
    assert torch.equal(got[1], torch.zeros(5))                            # a stray label: zeros


def test_lookup_past_32_bit_offsets():
    """A table and an output past 2^32 bytes: the last rows are right."""
    K, D, N = 2_200_000, 1024, 2_150_000
    C = torch.empty((K, D), dtype=BF, device="cuda")
    C[-64:] = rand((64, D), BF, 3)
    C[:64] = rand((64, D), BF, 4)
    lab = torch.zeros(N, dtype=torch.int32, device="cuda")
    lab[-32:] = torch.arange(K - 32, K, device="cuda")
    out = km.kmeans_lookup(C, lab)
    assert torch.equal(out[-32:], C[-32:])
    assert torch.equal(out[-40:-32], C[:1].expand(8, D))
    dC = km.kmeans_lookup_grad(out[:, :8], lab, K)                        # rows 2^11 bytes apart
    assert torch.equal(dC[-32:], C[-32:, :8])
    assert int((dC[1:-32] != 0).sum()) == 0


# ---- lookup gradient -------------------------------------------------------

GRAD_SHAPES = [(1, 1, 1), (1, 300, 4096), (9, 4, 7), (64, 1, 64), (1000, 37, 16), (4133, 275, 64),
               (777, 300, 129), (2050, 4096, 256), (513, 70, 520), (257, 1000, 1037),
               (20000, 5, 24), (5000, 70000, 8)]


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("N,K,D", GRAD_SHAPES)
def test_lookup_grad(N, K, D, dtype):
    dY = rand((N, D), dtype, N + D)
    for kind, index in (("uniform", torch.int32), ("zipf", torch.int64)):
        lab = some_labels(N, K, N + 1, index, kind)
        out = torch.full((K, D), float("nan"), dtype=dtype, device="cuda")   # every row is written
        got = km.kmeans_lookup_grad(dY, lab, K, scale=1.5, out=out)
        again = km.kmeans_lookup_grad(dY, lab, K, scale=1.5)
        want, bound = ref.lookup_grad(dY, lab, K, 1.5, dtype)
        ref.check(got, want, bound, f"{N} {K} {D} {kind}")
        assert torch.equal(got, again)                                    # bitwise the same again


@pytest.mark.parametrize("N,D", [(3000, 8), (40000, 64), (70001, 130), (9000, 1100)])
def test_lookup_grad_of_one_label(N, D):
    """All positions on one row: a run over every chunk, summed by the joined
    workgroup path."""
    dY = rand((N, D), BF, 5)
    lab = some_labels(N, 9, 6, torch.int32, "one")
    want, bound = ref.lookup_grad(dY, lab, 9, 1.0, F32)
    got = km.kmeans_lookup_grad(dY, lab, 9, out=torch.empty(9, D, device="cuda"))
    ref.check(got, want, bound)


@pytest.mark.parametrize("N,K,D,kind", [
    (2049, 256, 8, "one"),       # one position past a workgroup's share, one run over all
    (40000, 300, 64, "one"), (70001, 5000, 130, "zipf"), (30000, 65536, 24, "zipf"),
    (262144, 257, 16, "uniform"), (100000, 256, 12, "zipf"), (9000, 4096, 1100, "one"),
    (5000, 65537, 40, "zipf"), (300000, 256, 8, "uniform")])    # the sort path again
@pytest.mark.parametrize("accumulate", [False, True])
def test_lookup_grad_of_frequent_labels(N, K, D, kind, accumulate):
    """Buckets holding more positions than one workgroup sorts, several of
    them, with absent rows beside the frequent ones; and the limits between
    the two paths."""
    dY = rand((N, D), BF, 31)
    lab = some_labels(N, K, 32, torch.int32, kind)
    into = rand((K, D), F32, 33)
    before = into.clone()
    want, bound = ref.lookup_grad(dY, lab, K, 0.75, F32, into=before if accumulate else None)
    km.kmeans_lookup_grad(dY, lab, K, scale=0.75, out=into, accumulate=accumulate)
    ref.check(into, want, bound, f"{N} {K} {D} {kind}")
    again = before.clone()
    km.kmeans_lookup_grad(dY, lab, K, scale=0.75, out=again, accumulate=accumulate)
    assert torch.equal(again, into)


@pytest.mark.parametrize("N,K,D,kind", [
    (5000, 1, 128, "one"), (129, 1, 2000, "one"), (6000, 3, 257, "uniform"),
    (40000, 16, 128, "zipf"), (20000, 255, 136, "uniform"), (7, 2, 4096, "uniform"),
    ((1 << 20) + 1, 5, 128, "uniform"), (3000, 100, 127, "zipf")])
def test_lookup_grad_of_few_wide_rows(N, K, D, kind):
    """Tables of fewer rows than the GPU has CUs, at the row width and the
    number of positions where the path changes."""
    dY = rand((N, D), BF, 41)
    lab = some_labels(N, K, 42, torch.int32, kind)
    want, bound = ref.lookup_grad(dY, lab, K, 1.5, F32)
    got = km.kmeans_lookup_grad(dY, lab, K, scale=1.5, out=torch.empty(K, D, device="cuda"))
    ref.check(got, want, bound, f"{N} {K} {D} {kind}")


@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (FP, F32), (F32, F32)])
@pytest.mark.parametrize("N,K,D", [(1000, 37, 16), (777, 300, 129), (3000, 2, 64), (50, 9, 515),
                                   (900, 270, 515), (40, 300, 5)])
def test_lookup_grad_accumulates(N, K, D, dtype, out_dtype):
    dY = rand((N, D), dtype, 11)
    lab = some_labels(N, K, 12)
    into = rows_in(rand((K, D), out_dtype, 13), 5, 1)
    before = into.clone()
    km.kmeans_lookup_grad(dY, lab, K, scale=0.5, out=into, accumulate=True)
    want, bound = ref.lookup_grad(dY, lab, K, 0.5, out_dtype, into=before)
    ref.check(into, want, bound)
    assert torch.equal(into._base[:, :1], torch.full_like(into._base[:, :1], 7.0))
    assert torch.equal(into._base[:, D + 1:], torch.full_like(into._base[:, D + 1:], 7.0))


def test_lookup_grad_without_labels():
    out = torch.full((5, 9), 3.0, device="cuda")
    empty = torch.empty(0, dtype=torch.int64, device="cuda")
    km.kmeans_lookup_grad(torch.empty(0, 9, device="cuda"), empty, 5, out=out, accumulate=True)
    assert torch.equal(out, torch.full((5, 9), 3.0, device="cuda"))
    km.kmeans_lookup_grad(torch.empty(0, 9, device="cuda"), empty, 5, out=out)
    assert int((out != 0).sum()) == 0
    stray = torch.full((300,), -1, dtype=torch.int32, device="cuda")      # labels, but none counts
    nan = torch.full((300, 9), float("nan"), device="cuda")
    assert int((km.kmeans_lookup_grad(nan, stray, 5) != 0).sum()) == 0


def test_lookup_grad_against_differences():
    """The lookup is linear in the table, so a difference of the loss
    sum(dY * lookup(C)) along any direction is its gradient's product."""
    N, K, D = 700, 90, 33
    dY, lab = rand((N, D), F32, 21), some_labels(N, K, 22)
    C, V = rand((K, D), F32, 23), rand((K, D), F32, 24)
    dC = km.kmeans_lookup_grad(dY, lab, K, scale=1.25)
    loss = [float((ref.cpu64(dY) * ref.cpu64(km.kmeans_lookup(C + s * V, lab, scale=1.25))).sum())
            for s in (2.0, -2.0)]
    slope = (loss[0] - loss[1]) / 4.0
    _, bound = ref.lookup_grad(dY, lab, K, 1.25, F32)
    tol = float((bound * ref.cpu64(V).abs()).sum())
    # each looked-up value: two roundings of 2^-24 relative (C + s V, the product)
    size = sum(float((ref.cpu64(dY).abs() * ref.cpu64(km.kmeans_lookup((C + s * V).abs(), lab,
                                                                       scale=1.25))).sum())
               for s in (2.0, -2.0))
    tol += size * 2 * ref.EPS / 4.0
    assert abs(slope - float((ref.cpu64(dC) * ref.cpu64(V)).sum())) <= tol


# ---- linear ----------------------------------------------------------------

LINEAR_SHAPES = [  # (N, D, F): single rows, odd everything, tile edges, many splits of D
    (1, 1, 1), (1, 64, 16), (1, 4096, 300), (3, 33, 5), (16, 256, 129), (17, 128, 128),
    (64, 1000, 64), (100, 515, 77), (128, 64, 128), (129, 72, 136), (257, 200, 1000),
    (130, 8, 24), (33, 3000, 40), (1000, 96, 8), (300, 320, 520), (5, 8192, 16)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("N,D,F", LINEAR_SHAPES)
def test_linear(N, D, F, dtype):
    X, W = rand((N, D), dtype, N), rand((F, D), dtype, F, D ** -0.5)
    b, R = rand((F,), dtype, 3), rand((N, F), dtype, 4)
    acts = list(km.ACTIVATIONS)
    a = acts[(N + D + F) % 5]
    y, z, yb, zb = ref.linear(X, W, b, R, a)
    Y, Z = km.kmeans_linear(X, W, bias=b, residual=R, activation=a, save_pre=True)
    ref.check(Y, y, yb, f"Y {a}")
    ref.check(Z, z, zb, "Z")
    y, _, yb, _ = ref.linear(X, W)
    P = km.kmeans_linear(X, W)
    ref.check(P, y, yb, "plain")
    assert torch.equal(P, km.kmeans_linear(X, W))


@pytest.mark.parametrize("a", list(km.ACTIVATIONS))
def test_linear_activations(a):
    """Values far into both tails of every activation, and its bias, residual
    and pre-activation output each alone."""
    X, W = rand((70, 40), BF, 1, 4.0), rand((90, 40), BF, 2)
    b, R = rand((90,), BF, 3), rand((70, 90), BF, 4)
    for kw in (dict(), dict(bias=b), dict(residual=R), dict(bias=b, residual=R)):
        y, _, yb, _ = ref.linear(X, W, kw.get("bias"), kw.get("residual"), a)
        ref.check(km.kmeans_linear(X, W, activation=a, **kw), y, yb, f"{a} {list(kw)}")
    Y, Z = km.kmeans_linear(X, W, activation=a, save_pre=True)
    _, z, _, zb = ref.linear(X, W, activation=a)
    ref.check(Z, z, zb)
    # special pre-activations through a one-feature layer
    s = torch.tensor([[float("nan")], [300.0], [-300.0], [0.0], [-0.0]], dtype=BF).cuda()
    one = torch.ones(1, 1, dtype=BF).cuda()
    got = km.kmeans_linear(s, one, activation=a).float().cpu().flatten()
    assert torch.isnan(got[0])
    assert float(got[1]) == 300.0 and float(got[2]) == (-300.0 if a == "none" else 0.0)
    assert float(got[3]) == 0.0 and float(got[4]) == 0.0


def test_linear_infinities_stay_in_their_rows_and_columns():
    X, W = rand((200, 136), BF, 1), rand((150, 136), BF, 2)
    X[7, 3] = float("inf")
    W[40, 100] = float("nan")
    Y = km.kmeans_linear(X, W).cpu()
    bad = ~torch.isfinite(Y)
    want = torch.zeros(200, 150, dtype=torch.bool)
    want[7, :] = True
    want[:, 40] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("extra,shift", [(8, 0), (3, 0), (8, 8), (7, 1)])
def test_linear_strides(extra, shift):
    """Padded, shifted and misaligned rows; nothing is read or written beside
    the rows (what lies there is NaN for the inputs)."""
    N, D, F = 150, 104, 200
    def nan_rows(t):
        v = rows_in(t, extra, shift)
        keep = v.clone()
        v._base.fill_(float("nan"))
        v.copy_(keep)
        return v
    X, W = nan_rows(rand((N, D), BF, 1)), nan_rows(rand((F, D), BF, 2, 0.1))
    R = nan_rows(rand((N, F), BF, 3))
    out = rows_in(torch.zeros(N, F, dtype=BF, device="cuda"), extra, shift)
    pre = rows_in(torch.zeros(N, F, dtype=BF, device="cuda"), extra, shift)
    y, z, yb, zb = ref.linear(X, W, None, R, "silu")
    km.kmeans_linear(X, W, residual=R, activation="silu", out=out, pre=pre)
    ref.check(out, y, yb)
    ref.check(pre, z, zb)
    for t in (out, pre):
        side = torch.cat([t._base[:, :shift], t._base[:, shift + F:]], 1)
        assert torch.equal(side, torch.full_like(side, 7.0))
    dY = nan_rows(rand((N, F), BF, 5))
    Z = nan_rows(rand((N, F), BF, 6))
    want = ref.linear_grad(dY, X, W, Z, "silu")
    for name, got in zip(("dX", "dW", "db"), km.kmeans_linear_grad(dY, X, W, Z, "silu")):
        ref.check(got, *want[name], name)


def gaps(t, extra):
    """The same values in rows of an odd stride, NaN between them."""
    v = rows_in(t, extra)
    keep = v.clone()
    v._base.fill_(float("nan"))
    v.copy_(keep)
    return v


@pytest.mark.parametrize("N,D,F,odd", [(1200, 1600, 1200, "X"), (1200, 1600, 1200, "W"),
                                       (2900, 2907, 2901, "both")])
def test_linear_of_large_unaligned_operands(N, D, F, odd):
    """Products long enough that operands whose rows are not 16-byte aligned
    are laid out anew first, one of them or both."""
    X, W = rand((N, D), BF, 1), rand((F, D), BF, 2, D ** -0.5)
    b, R = rand((F,), BF, 3), rand((N, F), BF, 4)
    y, z, yb, zb = ref.linear(X, W, b, R, "silu")
    Y, Z = km.kmeans_linear(gaps(X, 5) if odd != "W" else X, gaps(W, 3) if odd != "X" else W,
                            bias=b, residual=R, activation="silu", save_pre=True)
    ref.check(Y, y, yb, "Y")
    ref.check(Z, z, zb, "Z")


@pytest.mark.parametrize("N,D,F", [(1024, 1001, 1024), (900, 1201, 1100), (1300, 1003, 1101)])
def test_linear_grad_of_large_unaligned_operands(N, D, F):
    X, W = gaps(rand((N, D), BF, 1), 7), gaps(rand((F, D), BF, 2, D ** -0.5), 2)
    dY, Z = gaps(rand((N, F), BF, 3, 0.25), 1), gaps(rand((N, F), BF, 4, 2.0), 3)
    want = ref.linear_grad(dY, X, W, Z, "gelu")
    for name, got in zip(("dX", "dW", "db"), km.kmeans_linear_grad(dY, X, W, Z, "gelu")):
        ref.check(got, *want[name], name)


def test_linear_in_place_residual_and_leading_shape():
    X, W, R = rand((3, 5, 64), BF, 1), rand((48, 64), BF, 2, 0.1), rand((3, 5, 48), BF, 3)
    want = km.kmeans_linear(X, W, residual=R, activation="gelu")
    assert want.shape == (3, 5, 48)
    km.kmeans_linear(X, W, residual=R, activation="gelu", out=R)
    assert torch.equal(R, want)
    assert km.kmeans_linear(X[:0], W).shape == (0, 5, 48)


# ---- linear gradients ------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("N,D,F", LINEAR_SHAPES)
def test_linear_grad(N, D, F, dtype):
    X, W = rand((N, D), dtype, N), rand((F, D), dtype, F, D ** -0.5)
    dY, Z = rand((N, F), dtype, 5, 0.25), rand((N, F), dtype, 6, 2.0)
    acts = list(km.ACTIVATIONS)
    for a in (acts[(N + F) % 5], "none"):
        want = ref.linear_grad(dY, X, W, Z, a)
        got = km.kmeans_linear_grad(dY, X, W, None if a == "none" else Z, a)
        for name, g in zip(("dX", "dW", "db"), got):
            ref.check(g, *want[name], f"{name} {a}")
        again = km.kmeans_linear_grad(dY, X, W, None if a == "none" else Z, a)
        assert all(torch.equal(g, h) for g, h in zip(got, again))


@pytest.mark.parametrize("a", list(km.ACTIVATIONS))
def test_linear_grad_parts(a):
    """Each gradient alone gives the same bits as all together."""
    N, D, F = 210, 72, 50
    X, W = rand((N, D), BF, 1), rand((F, D), BF, 2, 0.1)
    dY, Z = rand((N, F), BF, 3), rand((N, F), BF, 4, 3.0)
    dX, dW, db = km.kmeans_linear_grad(dY, X, W, Z, a)
    assert torch.equal(km.kmeans_linear_grad(dY, X, W, Z, a, bias=False, need_dw=False)[0], dX)
    assert torch.equal(km.kmeans_linear_grad(dY, X, W, Z, a, bias=False, need_dx=False)[1], dW)
    assert torch.equal(km.kmeans_linear_grad(dY, X, W, Z, a, need_dx=False, need_dw=False)[2], db)


def test_linear_grad_long_batch():
    """Many rows, few outputs: the weight gradient's sum is split over N."""
    N, D, F = 20011, 48, 24
    X, W, dY = rand((N, D), BF, 1), rand((F, D), BF, 2), rand((N, F), BF, 3)
    want = ref.linear_grad(dY, X, W)
    for name, g in zip(("dX", "dW", "db"), km.kmeans_linear_grad(dY, X, W)):
        ref.check(g, *want[name], name)


def test_linear_grad_of_no_rows():
    X, W = torch.empty(0, 40, dtype=BF, device="cuda"), rand((9, 40), BF, 1)
    dX, dW, db = km.kmeans_linear_grad(torch.empty(0, 9, dtype=BF, device="cuda"), X, W)
    assert dX.shape == (0, 40) and int((dW != 0).sum()) == 0 and int((db != 0).sum()) == 0


@pytest.mark.parametrize("a", list(km.ACTIVATIONS))
def test_linear_grad_against_differences(a):
    """Directional differences of sum(dY * act(X W^T + b)) in fp64 (h = 1e-4:
    h^2 / 6 times the third derivative along the direction, which the loss's
    curvature bounds far below the rounding of the gradients themselves)."""
    N, D, F = 40, 24, 30
    X, W, b = rand((N, D), FP, 1), rand((F, D), FP, 2, 0.2), rand((F,), FP, 3)
    dY = rand((N, F), FP, 4)
    _, Z = km.kmeans_linear(X, W, bias=b, activation=a, save_pre=True)
    if a == "relu":                      # differences hold away from the kink
        dY[Z.abs() < 0.05] = 0
    dX, dW, db = km.kmeans_linear_grad(dY, X, W, Z, a)
    x, w, c, g = (ref.cpu64(t) for t in (X, W, b, dY))
    want = ref.linear_grad(dY, X, W, Z, a)
    # Z was rounded to fp16: the slope it gives is off by |act''| (< 1.2) of that
    _, z, _, zb = ref.linear(X, W, b)
    slope_err = 1.2 * zb * g.abs()
    for name, base, grad in (("dX", x, dX), ("dW", w, dW), ("db", c, db)):
        v = ref.cpu64(rand(tuple(base.shape), F32, 9))
        h = 1e-4
        def loss(s):
            p = {"dX": x, "dW": w, "db": c}
            p[name] = base + s * v
            return float((g * ref.act(p["dX"] @ p["dW"].t() + p["db"], a)).sum())
        diff = (loss(h) - loss(-h)) / (2 * h)
        tol = float((want[name][1] * v.abs()).sum())
        lever = {"dX": lambda: v.abs() @ w.abs().t(), "dW": lambda: x.abs() @ v.abs().t(),
                 "db": lambda: v.abs().expand(N, F)}[name]()
        tol += float((slope_err * lever).sum()) + 1e-6
        assert abs(diff - float((ref.cpu64(grad) * v).sum())) <= tol, (a, name)


# ---- gradient norm and clipping --------------------------------------------

def clip_reference(grads, norm, max_norm):
    """Clipped values from the norm the kernel gave: fp32, one rounding, the
    same bits."""
    n = np.float32(float(norm))
    with np.errstate(all="ignore"):
        ratio = np.float32(max_norm) / np.float32(n + np.float32(1e-6))
    factor = torch.tensor(1.0 if ratio > 1 else ratio, dtype=F32)
    return [(g.cpu().float() * factor).to(g.dtype) for g in grads]


def exact_norm(grads):
    return math.sqrt(sum(float(g.detach().cpu().double().square().sum()) for g in grads))


@pytest.mark.parametrize("sizes", [[1], [0, 3], [5, 8, 16384, 16385, 1], [100003] * 3,
                                   [7] * 95, [33] * 96, [9] * 97, [1000 + i for i in range(300)]])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
def test_clip(sizes, max_norm):
    kinds = (BF, F32, FP)
    grads = [rand((n,), kinds[i % 3], i, 10.0 ** (i % 3 - 1)) for i, n in enumerate(sizes)]
    before = [g.clone() for g in grads]
    n0 = km.kmeans_gradient_norm(grads)
    outs = [torch.full_like(g, 5.0) for g in grads]
    norm, clipped = km.kmeans_clip_gradients(grads, max_norm, out=outs)
    want = exact_norm(before)
    assert float(n0) == float(norm)
    # fp64 sums of at most 2^20 squares, one rounding to fp32
    assert abs(float(norm) - want) <= want * 2.0 ** -23
    for got, w, g, b in zip(clipped, clip_reference(before, norm, max_norm), grads, before):
        assert torch.equal(got.cpu(), w)
        assert torch.equal(g, b)                                          # the inputs are kept
    inplace, same = km.kmeans_clip_gradients(grads, max_norm)
    assert float(inplace) == float(norm) and all(a is b for a, b in zip(same, grads))
    for got, w in zip(grads, outs):
        assert torch.equal(got, w)


def test_clip_of_extreme_values():
    big = [torch.full((1000,), 1e30, device="cuda"), torch.full((9,), 3e38, dtype=BF, device="cuda")]
    # a norm past the largest fp32 (9.01e38 here) is infinite as fp32
    assert exact_norm(big) > torch.finfo(F32).max
    assert math.isinf(float(km.kmeans_gradient_norm(big)))
    big[1] *= 0.1                                                         # 9.01e37: it is not
    norm, out = km.kmeans_clip_gradients(big, 2.0, out=[torch.empty_like(g) for g in big])
    assert abs(float(norm) / exact_norm(big) - 1) < 2.0 ** -23            # no overflow in fp32
    assert abs(exact_norm(out) - 2.0) < 2.0 * 2 ** -8
    tiny = [torch.full((1000,), 1e-30, device="cuda")]
    assert abs(float(km.kmeans_gradient_norm(tiny)) / exact_norm(tiny) - 1) < 2.0 ** -23
    zero = [torch.zeros(5000, dtype=FP, device="cuda")]
    norm, out = km.kmeans_clip_gradients(zero, 1.0)
    assert float(norm) == 0.0 and int((out[0] != 0).sum()) == 0
    none, _ = km.kmeans_clip_gradients([], 1.0)
    assert float(none) == 0.0 and float(km.kmeans_gradient_norm([])) == 0.0
    bad = [torch.ones(4, device="cuda"), torch.tensor([1.0, float("inf")], device="cuda")]
    norm, out = km.kmeans_clip_gradients(bad, 1.0, out=[torch.empty_like(g) for g in bad])
    assert math.isinf(float(norm)) and torch.equal(out[0], torch.zeros(4, device="cuda"))
    assert float(out[1][0]) == 0.0 and torch.isnan(out[1][1])
    bad[1][1] = float("nan")
    norm, out = km.kmeans_clip_gradients(bad, 1.0)
    assert math.isnan(float(norm)) and all(bool(torch.isnan(o).all()) for o in out)


def test_clip_misaligned_tensors_and_an_infinite_bound():
    flat = rand((70000,), BF, 1)
    grads = [flat[1:30000], flat[30001:30009], flat[40003:70000]]
    keep = flat.clone()
    norm, _ = km.kmeans_clip_gradients(grads, 0.25)
    w = clip_reference([keep[1:30000], keep[30001:30009], keep[40003:70000]], norm, 0.25)
    assert all(torch.equal(g.cpu(), x) for g, x in zip(grads, w))
    for i in (0, 30000, 30009, 40002):
        assert torch.equal(flat[i], keep[i])                              # neighbours are kept
    one = rand((100,), F32, 2)
    same = one.clone()
    km.kmeans_clip_gradients([one], float("inf"))
    assert torch.equal(one, same)


# ---- streams and graphs ----------------------------------------------------

def everything(C, lab, dY, X, W, b, R, G, outs):
    """One pass through every operator on the current stream."""
    Y, Z = km.kmeans_linear(X, W, bias=b, residual=R, activation="silu", save_pre=True)
    grads = km.kmeans_linear_grad(G, X, W, Z, "silu")
    rows = km.kmeans_lookup(C, lab, scale=2.0)
    dC = km.kmeans_lookup_grad(dY, lab, C.shape[0])
    norm, clipped = km.kmeans_clip_gradients([*grads, dC], 0.5, out=outs)
    return [Y, Z, *grads, rows, dC, norm, *clipped]


def inputs(seed):
    K, D, N, F = 70, 72, 300, 40
    return dict(C=rand((K, D), BF, seed), lab=some_labels(N, K, seed), dY=rand((N, D), BF, seed + 1),
                X=rand((N, D), BF, seed + 2), W=rand((F, D), BF, seed + 3, 0.1),
                b=rand((F,), BF, seed + 4), R=rand((N, F), BF, seed + 5),
                G=rand((N, F), BF, seed + 6))


def out_buffers():
    return [torch.empty(s, dtype=BF, device="cuda") for s in ((300, 72), (40, 72), (40,), (70, 72))]


def test_another_stream_gives_the_same_bits():
    args = inputs(50)
    want = everything(**args, outs=out_buffers())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = everything(**args, outs=out_buffers())
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    km.kmeans_release_workspace(stream=s)


def test_graph_replays_match_eager_calls():
    """Every operator captured once the stream's workspace has its size, and
    replayed with new inputs, bitwise equal to eager calls each time."""
    args = inputs(60)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        everything(**args, outs=out_buffers())
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    outs = out_buffers()
    with torch.cuda.graph(g, stream=s):
        got = everything(**args, outs=outs)
    for i in range(5):
        new = inputs(70 + 10 * i)
        for k, v in args.items():
            v.copy_(new[k])
        g.replay()
        torch.cuda.synchronize()
        want = everything(**new, outs=out_buffers())
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (i, j)
    km.kmeans_release_workspace(stream=s)
