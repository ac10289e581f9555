"""Operators of label prediction, without a GPU: the C ABI refuses bad arguments
on the host before any HIP call, empty calls are no-ops, the binding refuses
tensors that the library cannot take, and the reference agrees with differences
and with plain sampling."""

import ctypes

import numpy as np
import pytest
import torch

import means_nearest_centroid_amd as km
import prediction_reference as ref

FAKE = ctypes.c_void_p(0x10000)        # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)
TWO = ctypes.c_void_p(0x10002)
NUL = ctypes.c_void_p(0)
INV, UNS, ALI = km.KMEANS_ERR_INVALID_ARG, km.KMEANS_ERR_UNSUPPORTED, km.KMEANS_ERR_ALIGNMENT
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    return km.load_library()


def norm(lib, X=FAKE, xs=200, R=NUL, rs=200, w=NUL, N=10, D=200, dt=0, eps=1e-6, H=NUL, hs=200,
         Y=FAKE, ys=200, Q=NUL, qs=200, S=NUL, ss=2):
    return lib.kmeans_rms_norm(X, xs, R, rs, w, N, D, dt, eps, H, hs, Y, ys, Q, qs, S, ss, NUL)


def norm_grad(lib, dY=FAKE, ys=200, H=FAKE, hs=200, w=NUL, dH=NUL, dhs=200, N=10, D=200, dt=0,
              eps=1e-6, dX=FAKE, xs=200, dw=NUL):
    return lib.kmeans_rms_norm_grad(dY, ys, H, hs, w, dH, dhs, N, D, dt, eps, dX, xs, dw, NUL)


def quantize(lib, X=FAKE, xs=200, N=10, D=200, dt=0, rows=1, Q=FAKE, qs=200, S=FAKE, ss=2):
    return lib.kmeans_quantize(X, xs, N, D, dt, rows, Q, qs, S, ss, NUL)


def linear(lib, X=FAKE, xs=200, sx=FAKE, sxs=2, W=FAKE, ws=200, sw=FAKE, sws=2, b=NUL, R=NUL, rs=32,
           N=10, D=200, F=32, dt=0, act=0, Y=FAKE, ys=32):
    return lib.kmeans_linear_fp8(X, xs, sx, sxs, W, ws, sw, sws, b, R, rs, N, D, F, dt, act, Y, ys,
                                 NUL)


def sample(lib, Z=FAKE, zs=50, N=10, K=50, dt=0, u=FAKE, t=1.0, p=1.0, m=0.0, k=0, ts=NUL, ps=NUL,
           ms=NUL, ks=NUL, labels=FAKE, kind=0, none=False):
    o = km._Sampling(t, p, m, k, ts, ps, ms, ks)
    return lib.kmeans_sample(Z, zs, N, K, dt, u, NUL if none else ctypes.addressof(o), labels, kind,
                             NUL)


BIG = (1 << 20) + 1


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(D=0), INV), (dict(N=1 << 31), UNS), (dict(D=BIG, xs=BIG, ys=BIG), UNS),
    (dict(dt=3), INV), (dict(dt=-1), INV), (dict(eps=-1e-6), INV), (dict(eps=NAN), INV),
    (dict(X=NUL), INV), (dict(Y=NUL), INV), (dict(Q=FAKE, S=FAKE), INV), (dict(xs=199), INV),
    (dict(ys=199), INV), (dict(xs=1 << 31), UNS), (dict(R=FAKE, rs=199), INV),
    (dict(H=FAKE, hs=199), INV), (dict(X=ODD), ALI), (dict(Y=ODD), ALI), (dict(w=ODD), ALI),
    (dict(R=ODD), ALI), (dict(H=ODD), ALI), (dict(dt=2, X=TWO), ALI), (dict(dt=2, w=TWO), ALI),
    (dict(Y=NUL, Q=FAKE), INV), (dict(Y=NUL, Q=FAKE, S=FAKE, ss=1), INV),
    (dict(Y=NUL, Q=FAKE, S=TWO), ALI), (dict(Y=NUL, Q=FAKE, S=FAKE, qs=199), INV),
])
def test_rms_norm_refuses(lib, kw, status):
    assert norm(lib, **kw) == status
    assert lib.kmeans_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(D=0), INV), (dict(N=1 << 31), UNS), (dict(D=BIG), UNS),
    (dict(dt=3), INV), (dict(eps=NAN), INV), (dict(dY=NUL), INV), (dict(H=NUL), INV),
    (dict(dX=NUL), INV), (dict(ys=199), INV), (dict(hs=199), INV), (dict(xs=199), INV),
    (dict(dH=FAKE, dhs=199), INV), (dict(dY=ODD), ALI), (dict(H=ODD), ALI), (dict(dH=ODD), ALI),
    (dict(dX=ODD), ALI), (dict(w=ODD), ALI), (dict(dw=ODD), ALI), (dict(N=0, dw=ODD), ALI),
])
def test_rms_norm_grad_refuses(lib, kw, status):
    assert norm_grad(lib, **kw) == status
    assert lib.kmeans_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(D=0), INV), (dict(N=1 << 31), UNS), (dict(D=BIG), UNS),
    (dict(dt=4), INV), (dict(rows=0), INV), (dict(rows=64), INV), (dict(X=NUL), INV),
    (dict(Q=NUL), INV), (dict(S=NUL), INV), (dict(xs=199), INV), (dict(qs=199), INV),
    (dict(ss=1), INV), (dict(X=ODD), ALI), (dict(S=TWO), ALI),
])
def test_quantize_refuses(lib, kw, status):
    assert quantize(lib, **kw) == status
    assert lib.kmeans_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(D=0), INV), (dict(F=0), INV), (dict(N=1 << 31), UNS),
    (dict(D=BIG), UNS), (dict(F=BIG), UNS), (dict(dt=3), INV), (dict(act=5), INV),
    (dict(act=-1), INV), (dict(X=NUL), INV), (dict(W=NUL), INV), (dict(Y=NUL), INV),
    (dict(sx=NUL), INV), (dict(sw=NUL), INV), (dict(xs=199), INV), (dict(ws=199), INV),
    (dict(sxs=1), INV), (dict(sws=1), INV), (dict(ys=31), INV), (dict(R=FAKE, rs=31), INV),
    (dict(xs=BIG), UNS), (dict(ws=BIG), UNS), (dict(sxs=BIG), UNS), (dict(sws=BIG), UNS),
    (dict(ys=BIG), UNS), (dict(R=FAKE, rs=BIG), UNS), (dict(sx=TWO), ALI), (dict(sw=TWO), ALI),
    (dict(b=ODD), ALI), (dict(R=ODD), ALI), (dict(Y=ODD), ALI), (dict(dt=2, Y=TWO), ALI),
    (dict(N=(1 << 31) - 2048, F=1 << 20, ys=1 << 20, D=16, xs=16, ws=16), UNS),
])
def test_linear_fp8_refuses(lib, kw, status):
    assert linear(lib, **kw) == status
    assert lib.kmeans_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(K=0), INV), (dict(N=1 << 31), UNS), (dict(K=BIG), UNS),
    (dict(dt=3), INV), (dict(kind=2), INV), (dict(none=True), INV), (dict(Z=NUL), INV),
    (dict(u=NUL), INV), (dict(labels=NUL), INV), (dict(zs=49), INV), (dict(Z=ODD), ALI),
    (dict(u=TWO), ALI), (dict(labels=TWO), ALI), (dict(labels=ctypes.c_void_p(0x10004), kind=1), ALI),
    (dict(t=-1.0), INV), (dict(t=NAN), INV), (dict(p=-0.1), INV), (dict(p=1.1), INV),
    (dict(p=NAN), INV), (dict(m=-0.1), INV), (dict(m=1.5), INV), (dict(m=NAN), INV),
    (dict(k=-1), INV), (dict(ts=0x10002), ALI), (dict(ps=0x10002), ALI), (dict(ms=0x10002), ALI),
    (dict(ks=0x10002), ALI),
])
def test_sample_refuses(lib, kw, status):
    assert sample(lib, **kw) == status
    assert lib.kmeans_last_error().decode()


def test_empty_calls_are_no_ops(lib):
    assert norm(lib, N=0, X=NUL, Y=NUL) == km.KMEANS_OK
    assert norm_grad(lib, N=0, dY=NUL, H=NUL, dX=NUL) == km.KMEANS_OK
    assert quantize(lib, N=0, X=NUL, Q=NUL, S=NUL) == km.KMEANS_OK
    assert linear(lib, N=0, X=NUL, W=NUL, Y=NUL, sx=NUL, sw=NUL) == km.KMEANS_OK
    assert sample(lib, N=0, Z=NUL, u=NUL, labels=NUL) == km.KMEANS_OK
    assert lib.kmeans_last_error().decode() == ""


def test_binding_refuses_what_the_library_cannot_take():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    q = torch.zeros(4, 8, dtype=torch.float8_e4m3fn)
    s = torch.zeros(4, 1)
    for call in (lambda: km.kmeans_rms_norm(x), lambda: km.kmeans_rms_norm_grad(x, x),
                 lambda: km.kmeans_quantize(x), lambda: km.kmeans_linear_fp8(q, s, q, s),
                 lambda: km.kmeans_sample(x, torch.zeros(4))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        km.kmeans_quantize([1.0])
    with pytest.raises(ValueError, match="two dimensions"):
        km.kmeans_rms_norm(x[0])


# ---- the reference itself --------------------------------------------------

def test_reference_gradients_agree_with_differences(monkeypatch):
    """Central differences of step 2^-13 in fp64: the third derivative (below 200
    here) over 6 times the square of the step, and 2^-50 of the loss over it."""
    for bounds in (ref.U, ref.TINY):
        monkeypatch.setitem(bounds, torch.float64, 0.0)
    g = torch.Generator().manual_seed(1)
    H, dY, dH = (torch.randn(3, 20, generator=g, dtype=torch.float64) for _ in range(3))
    w = torch.randn(20, generator=g, dtype=torch.float64)
    loss = lambda h, v: float((ref.rms_norm(h, v)[0] * dY).sum() + (h * dH).sum())  # noqa: E731
    want = ref.rms_norm_grad(dY, H, w, dH)
    h = 2.0 ** -13
    for i in range(3):
        for j in range(20):
            e = torch.zeros_like(H)
            e[i, j] = h
            assert abs((loss(H + e, w) - loss(H - e, w)) / (2 * h) - want["dX"][0][i, j]) < 1e-6
    for j in range(20):
        e = torch.zeros_like(w)
        e[j] = h
        assert abs((loss(H, w + e) - loss(H, w - e)) / (2 * h) - want["dw"][0][j]) < 1e-6


def test_reference_sampling():
    z = torch.tensor([[1.0, 3.0, 3.0, -float("inf"), float("nan"), 2.0]])
    one = lambda u, t=1.0, k=0, p=1.0, m=0.0: ref.sample(z, [u], [t], [k], [p], [m])[0]  # noqa: E731
    assert one(0.0) == {1} and one(1.0) == {0} and one(0.5) == {2} and one(0.99, t=0.0) == {1}
    assert one(0.99, k=2) == {2} and one(0.99, k=1) == {1} and one(0.99, p=0.0) == {1}
    assert one(0.99, m=1.0) == {2} and one(0.99, m=0.3) == {5}      # exp(-1) = 0.37
    assert one(0.99, p=0.5) == {2}                                  # 1 of 2.5 is too little
    assert ref.sample(torch.full((1, 4), -float("inf")), [0.5], [1.0], [0], [1.0], [0.0]) == [{-1}]
    n = 1000
    u = (np.arange(n) + 0.5) / n
    got = [list(a)[0] for a in ref.sample(z.expand(n, 6), u, [1.0] * n, [0] * n, [1.0] * n, [0.0] * n)]
    want = torch.softmax(z[0].double().nan_to_num(-np.inf), 0).numpy() * n
    assert np.abs(np.bincount(got, minlength=6) - want).max() <= 1


def test_reference_blocks():
    x = torch.zeros(3, 200, dtype=torch.float64)
    x[0, 3], x[1, 150], x[2, 199] = -896.0, 1e-45, 4.48
    each, s = ref.block_scales(x, 1)
    assert s.tolist() == [[2.0, 1.0], [1.0, 2.0 ** -126], [1.0, pytest.approx(0.01)]]
    assert each[0, 127] == 2 and each[0, 128] == 1
    _, s = ref.block_scales(x, 128)
    assert s.shape == (1, 2) and s[0, 0] == 2
