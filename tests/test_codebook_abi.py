"""Codebook-training operators, without a GPU: the C ABI refuses bad arguments
on the host before any HIP call, empty calls are no-ops, the binding refuses
tensors that the library cannot take, and the reference's gradients agree with
differences."""

import ctypes

import pytest
import torch

import codebook_reference as ref
import means_nearest_centroid_amd as km

FAKE = ctypes.c_void_p(0x10000)        # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)
NUL = ctypes.c_void_p(0)
INV, UNS, ALI = km.KMEANS_ERR_INVALID_ARG, km.KMEANS_ERR_UNSUPPORTED, km.KMEANS_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def lib():
    return km.load_library()


def lookup(lib, C=FAKE, cs=64, lab=FAKE, kind=0, N=10, D=64, K=5, dt=0, Y=FAKE, ys=64):
    return lib.kmeans_lookup(C, cs, lab, kind, N, D, K, dt, 1.0, Y, ys, NUL)


def lookup_grad(lib, dY=FAKE, ys=64, lab=FAKE, kind=0, N=10, D=64, K=5, dt=0, acc=0, dC=FAKE,
                odt=0, cs=64):
    return lib.kmeans_lookup_grad(dY, ys, lab, kind, N, D, K, dt, 1.0, acc, dC, odt, cs, NUL)


def linear(lib, X=FAKE, xs=64, W=FAKE, ws=64, b=NUL, R=NUL, rs=32, N=10, D=64, F=32, dt=0, act=0,
           Y=FAKE, ys=32, Z=NUL, zs=32):
    return lib.kmeans_linear(X, xs, W, ws, b, R, rs, N, D, F, dt, act, Y, ys, Z, zs, NUL)


def linear_grad(lib, dY=FAKE, ys=32, X=FAKE, xs=64, W=FAKE, ws=64, Z=NUL, zs=32, N=10, D=64, F=32,
                dt=0, act=0, dX=FAKE, dxs=64, dW=FAKE, dws=64, db=NUL):
    return lib.kmeans_linear_grad(dY, ys, X, xs, W, ws, Z, zs, N, D, F, dt, act, dX, dxs, dW, dws,
                                  db, NUL)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(D=0), INV), (dict(K=0), INV), (dict(N=1 << 31), UNS),
    (dict(D=1 << 31, cs=1 << 31, ys=1 << 31), UNS), (dict(K=1 << 31), UNS),
    (dict(dt=3), INV), (dict(dt=-1), INV), (dict(kind=2), INV),
    (dict(C=NUL), INV), (dict(lab=NUL), INV), (dict(Y=NUL), INV),
    (dict(cs=63), INV), (dict(ys=63), INV),
    (dict(C=ODD), ALI), (dict(Y=ODD), ALI), (dict(lab=ODD), ALI),
    (dict(lab=ctypes.c_void_p(0x10004), kind=1), ALI), (dict(C=ctypes.c_void_p(0x10002), dt=2), ALI),
    (dict(N=(1 << 31) - 1024, D=1 << 30, cs=1 << 30, ys=1 << 30), UNS),
])
def test_lookup_refuses(lib, kw, status):
    assert lookup(lib, **kw) == status
    assert lib.kmeans_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(D=0), INV), (dict(K=0), INV), (dict(N=1 << 31), UNS),
    (dict(K=1 << 31), UNS), (dict(dt=3), INV), (dict(kind=-1), INV),
    (dict(odt=1), INV), (dict(dt=2, odt=0), INV), (dict(dY=NUL), INV), (dict(lab=NUL), INV),
    (dict(dC=NUL), INV), (dict(N=0, dC=NUL), INV), (dict(ys=1), INV), (dict(cs=1), INV),
    (dict(dY=ODD), ALI), (dict(dC=ODD), ALI), (dict(odt=2, dC=ctypes.c_void_p(0x10002)), ALI),
])
def test_lookup_grad_refuses(lib, kw, status):
    assert lookup_grad(lib, **kw) == status
    assert lib.kmeans_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(D=0), INV), (dict(F=0), INV), (dict(N=1 << 31), UNS),
    (dict(D=(1 << 20) + 1, xs=1 << 21, ws=1 << 21), UNS), (dict(F=(1 << 20) + 1), UNS),
    (dict(xs=(1 << 20) + 1), UNS), (dict(dt=2), UNS), (dict(dt=5), INV), (dict(act=5), INV),
    (dict(act=-1), INV), (dict(X=NUL), INV), (dict(W=NUL), INV), (dict(Y=NUL), INV),
    (dict(xs=63), INV), (dict(ws=63), INV), (dict(ys=31), INV), (dict(R=FAKE, rs=31), INV),
    (dict(Z=FAKE, zs=31), INV), (dict(X=ODD), ALI), (dict(b=ODD), ALI), (dict(R=ODD), ALI),
    (dict(Z=ODD), ALI), (dict(Y=ODD), ALI),
])
def test_linear_refuses(lib, kw, status):
    assert linear(lib, **kw) == status
    assert lib.kmeans_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(D=0), INV), (dict(F=0), INV), (dict(dt=2), UNS), (dict(act=7), INV),
    (dict(dY=NUL), INV), (dict(X=NUL), INV), (dict(W=NUL), INV), (dict(act=1), INV),
    (dict(act=1, Z=FAKE, zs=31), INV), (dict(dxs=63), INV), (dict(dws=63), INV),
    (dict(ys=31), INV), (dict(dX=ODD), ALI), (dict(dW=ODD), ALI), (dict(db=ODD), ALI),
    (dict(N=0, dW=ODD), ALI),
])
def test_linear_grad_refuses(lib, kw, status):
    assert linear_grad(lib, **kw) == status
    assert lib.kmeans_last_error().decode()


class Gradient(ctypes.Structure):
    """kmeans_gradient_t."""
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def gradient(src=0x10000, dst=0x20000, numel=8, dtype=0, reserved=0):
    g = (Gradient * 1)()
    g[0].src, g[0].dst, g[0].numel, g[0].dtype, g[0].reserved = src, dst, numel, dtype, reserved
    return g


@pytest.mark.parametrize("kw,status", [
    (dict(numel=-1), INV), (dict(dtype=3), INV), (dict(dtype=-1), INV), (dict(reserved=1), INV),
    (dict(src=0), INV), (dict(dst=0), INV), (dict(src=0x10001), ALI),
    (dict(dst=0x10002, dtype=2), ALI), (dict(numel=(1 << 40) + 1), UNS),
])
def test_clip_refuses(lib, kw, status):
    assert lib.kmeans_clip_gradients(gradient(**kw), 1, 1.0, FAKE, NUL) == status
    assert lib.kmeans_last_error().decode()


def test_clip_refuses_its_other_arguments(lib):
    f = lib.kmeans_clip_gradients
    assert f(gradient(), 1, -1.0, FAKE, NUL) == INV
    assert f(gradient(), 1, float("nan"), FAKE, NUL) == INV
    assert f(gradient(), -1, 1.0, FAKE, NUL) == INV
    assert f(NUL, 1, 1.0, FAKE, NUL) == INV
    assert f(gradient(), 1, 1.0, NUL, NUL) == INV
    assert f(gradient(), 1, 1.0, ctypes.c_void_p(0x10002), NUL) == ALI
    assert lib.kmeans_gradient_norm(gradient(src=0), 1, FAKE, NUL) == INV


def test_empty_calls_are_no_ops(lib):
    assert lookup(lib, N=0, C=NUL, lab=NUL, Y=NUL) == km.KMEANS_OK
    assert lookup_grad(lib, N=0, acc=1, dY=NUL, lab=NUL) == km.KMEANS_OK
    assert linear(lib, N=0, X=NUL, W=NUL, Y=NUL) == km.KMEANS_OK
    assert linear_grad(lib, dX=NUL, dW=NUL) == km.KMEANS_OK
    assert linear_grad(lib, N=0, dW=NUL) == km.KMEANS_OK
    assert lib.kmeans_last_error().decode() == ""


def test_binding_refuses_what_the_library_cannot_take():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    lab = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        km.kmeans_lookup(x, lab)
    with pytest.raises(ValueError, match="CUDA"):
        km.kmeans_lookup_grad(x, lab, 3)
    with pytest.raises(ValueError, match="CUDA"):
        km.kmeans_linear(x, x)
    with pytest.raises(ValueError, match="one GPU"):
        km._gradient_list([x], None, torch.device("cuda:0"))
    with pytest.raises(ValueError, match="activation"):
        km._activation("tanh")
    with pytest.raises(TypeError):
        km._rows([1], "X")


@pytest.mark.parametrize("name", list(km.ACTIVATIONS))
def test_reference_slopes_agree_with_differences(name):
    z = torch.linspace(-6, 6, 601, dtype=torch.float64) + 1e-3
    h = 1e-5
    diff = (ref.act(z + h, name) - ref.act(z - h, name)) / (2 * h)
    # central differences: h^2 / 6 times the third derivative (below 3), and
    # rounding of 1e-15 |act| / h
    assert float((diff - ref.act_slope(z, name)).abs().max()) < 1e-9
