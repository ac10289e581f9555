"""MI355X (gfx950) k-means assignment and centroid update: Python binding of
``libkmeans_mi355x.so``.

The functions here only marshal torch tensors into the C ABI declared in
``include/kmeans_mi355x.h`` (device pointers, sizes, the current HIP stream);
every step of the computation runs in the library's HIP kernels.  There is no
CPU fallback: if the library is missing, the first call raises.

    norms = kmeans_centroid_norms(C)                    # fp32 [K]
    labels, min_dist = kmeans_assign(X, C, norms)       # int32 [N], fp32 [N]
    C, norms, counts, _ = kmeans_update(X, labels, C)   # next Lloyd iterate

``X`` and ``C`` are ``torch.bfloat16`` CUDA tensors of shape ``[N, D]`` and
``[K, D]``, contiguous.  Calls are asynchronous on the current stream.

A table that is trained by gradients inside a model (a codebook, an embedding)
has these operators around the two steps above (bf16 or fp16; the lookup,
its gradient and the clipping also fp32):

    Y, Z = kmeans_linear(X, W, bias, residual, activation="gelu", save_pre=True)
    rows = kmeans_lookup(C, labels, scale=1.0)
    dC = kmeans_lookup_grad(dY, labels, K, scale=1.0)
    dX, dW, db = kmeans_linear_grad(dY, X, W, Z, activation="gelu")
    norm, _ = kmeans_clip_gradients([dW, db, dC], max_norm=1.0)

A model that predicts labels has the norm with its gradient, the linear layer on
8-bit operands, and the draw of a label from each row of scores:

    Q, scales, H = kmeans_rms_norm(X, weight, residual, quantize=True)
    W8, w_scales = kmeans_quantize(W, rows=128)                 # once
    logits = kmeans_linear_fp8(Q, scales, W8, w_scales, dtype=torch.float32)
    labels = kmeans_sample(logits, uniforms, temperature=0.8, top_k=50, top_p=0.95)
    dX, dw = kmeans_rms_norm_grad(dY, H, weight, dH=dH)

Autograd does not see these calls: their results carry no gradient function,
whatever their inputs require, and the gradients are the calls above (inside a
``torch.autograd.Function``, say, whose ``backward`` makes them).
"""

from __future__ import annotations

import array
import contextlib
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# The built library; KMEANS_MI355X_LIBRARY names another build of the same
# sources instead (the host-sanitizer test loads one built with AddressSanitizer).
LIBRARY = os.environ.get("KMEANS_MI355X_LIBRARY") or os.path.join(_HERE, "libkmeans_mi355x.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "kmeans_mi355x.h")

KMEANS_OK = 0
KMEANS_ERR_INVALID_ARG = 1
KMEANS_ERR_UNSUPPORTED = 2
KMEANS_ERR_ALIGNMENT = 3
KMEANS_ERR_HIP = 4
KMEANS_ERR_NO_MEMORY = 5

PATH_AUTO = 0
PATH_DIRECT = 1
PATH_SPLIT = 2
PATH_PERSISTENT = 3
# kmeans_update_path_t
UPDATE_AUTO = 0
UPDATE_SORT = 1
UPDATE_BUCKETS = 2
# kmeans_dtype_t, kmeans_label_t
BF16, FP16, FP32 = 0, 1, 2
INT32, INT64 = 0, 1
# kmeans_activation_t, by the name the functions below take
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_STATUS_NAMES = {
    0: "KMEANS_OK", 1: "KMEANS_ERR_INVALID_ARG", 2: "KMEANS_ERR_UNSUPPORTED",
    3: "KMEANS_ERR_ALIGNMENT", 4: "KMEANS_ERR_HIP", 5: "KMEANS_ERR_NO_MEMORY",
}

_lib = None


class KmeansError(RuntimeError):
    """A non-OK status from the C ABI."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def load_library(path: str = LIBRARY):
    """Load the HIP library (after torch, so both use one HIP runtime)."""
    global _lib
    if _lib is not None and path == LIBRARY:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"HIP library {path} is not built; run `python -m "
            "means_nearest_centroid_amd.build` (or __graft_entry__.build())")
    try:
        import torch  # noqa: F401  -- maps torch's libamdhip64 first
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    i32p = ctypes.POINTER(ctypes.c_int32)
    lib.kmeans_centroid_norms.argtypes = [vp, i64, i64, vp, vp]
    lib.kmeans_centroid_norms.restype = ctypes.c_int
    lib.kmeans_assign.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp]
    lib.kmeans_assign.restype = ctypes.c_int
    lib.kmeans_assign_static.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp]
    lib.kmeans_assign_static.restype = ctypes.c_int
    lib.kmeans_assign_path.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, i32, i32, vp]
    lib.kmeans_assign_path.restype = ctypes.c_int
    lib.kmeans_plan.argtypes = [i64, i64, i64, i32, i32p, i32p, i32p, i32p, i32p, i32p]
    lib.kmeans_plan.restype = ctypes.c_int
    lib.kmeans_update.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp, vp, vp]
    lib.kmeans_update.restype = ctypes.c_int
    lib.kmeans_update_path.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp, vp, i32, vp]
    lib.kmeans_update_path.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.kmeans_lookup.argtypes = [vp, i64, vp, i32, i64, i64, i64, i32, f32, vp, i64, vp]
    lib.kmeans_lookup.restype = ctypes.c_int
    lib.kmeans_lookup_grad.argtypes = [vp, i64, vp, i32, i64, i64, i64, i32, f32, i32, vp, i32,
                                       i64, vp]
    lib.kmeans_lookup_grad.restype = ctypes.c_int
    lib.kmeans_linear.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, i32, i32, vp, i64,
                                  vp, i64, vp]
    lib.kmeans_linear.restype = ctypes.c_int
    lib.kmeans_linear_grad.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, i32,
                                       i32, vp, i64, vp, i64, vp, vp]
    lib.kmeans_linear_grad.restype = ctypes.c_int
    lib.kmeans_gradient_norm.argtypes = [vp, i64, vp, vp]
    lib.kmeans_gradient_norm.restype = ctypes.c_int
    lib.kmeans_clip_gradients.argtypes = [vp, i64, f32, vp, vp]
    lib.kmeans_clip_gradients.restype = ctypes.c_int
    lib.kmeans_rms_norm.argtypes = [vp, i64, vp, i64, vp, i64, i64, i32, f32, vp, i64, vp, i64, vp,
                                    i64, vp, i64, vp]
    lib.kmeans_rms_norm.restype = ctypes.c_int
    lib.kmeans_rms_norm_grad.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i32, f32, vp,
                                         i64, vp, vp]
    lib.kmeans_rms_norm_grad.restype = ctypes.c_int
    lib.kmeans_quantize.argtypes = [vp, i64, i64, i64, i32, i32, vp, i64, vp, i64, vp]
    lib.kmeans_quantize.restype = ctypes.c_int
    lib.kmeans_linear_fp8.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, i64, i64, i64,
                                      i64, i32, i32, vp, i64, vp]
    lib.kmeans_linear_fp8.restype = ctypes.c_int
    lib.kmeans_sample.argtypes = [vp, i64, i64, i64, i32, vp, vp, vp, i32, vp]
    lib.kmeans_sample.restype = ctypes.c_int
    lib.kmeans_release_workspace.argtypes = [vp]
    lib.kmeans_release_workspace.restype = ctypes.c_int
    lib.kmeans_last_error.argtypes = []
    lib.kmeans_last_error.restype = ctypes.c_char_p
    lib.kmeans_abi_version.argtypes = []
    lib.kmeans_abi_version.restype = ctypes.c_int
    if path == LIBRARY:
        _lib = lib
    return lib


def _check(lib, status: int):
    if status != KMEANS_OK:
        raise KmeansError(status, lib.kmeans_last_error().decode(errors="replace"))


def _stream_handle(stream, device=None):
    """The HIP stream to launch on, as an integer handle: ``stream``, or the
    current stream of ``device`` (of the current device when None).  Calls
    are often a few microseconds of GPU time, so this avoids building a
    torch Stream object per call where torch exposes the raw handle."""
    import torch
    if stream is None:
        index = device.index if device is not None else torch.cuda.current_device()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(index)
        return torch.cuda.current_stream(index).cuda_stream
    if device is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device} but the tensors on {device}")
    return stream.cuda_stream


def _on(device):
    """The library launches on the current HIP device: make it the tensors'
    (a no-op context when it already is)."""
    import torch
    if device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _matrix(t, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16 or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D torch.bfloat16 CUDA tensor "
                         f"(got {t.dtype}, {tuple(t.shape)}, {t.device})")
    return t


def _vector(t, name, dtype, n, device):
    """Check a caller-supplied 1-D output (or input) tensor: the C ABI sees
    only a pointer, so a wrong dtype, a short tensor or a strided view would
    be written out of bounds without an error."""
    import torch
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda
            or t.device != device or t.numel() != n or not t.is_contiguous()):
        got = (f"{t.dtype}, {tuple(t.shape)}, {t.device}, contiguous={t.is_contiguous()}"
               if isinstance(t, torch.Tensor) else type(t).__name__)
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements "
                         f"on {device} (got {got})")
    return t


def abi_version() -> int:
    return load_library().kmeans_abi_version()


def kmeans_plan(N: int, D: int, K: int, compute_units: int = 0) -> dict:
    """Launch plan the library would use for a shape on a GPU with
    ``compute_units`` CUs (0: 256, an MI355X); no GPU needed."""
    lib = load_library()
    vals = [ctypes.c_int32(0) for _ in range(6)]
    _check(lib, lib.kmeans_plan(N, D, K, compute_units, *[ctypes.byref(v) for v in vals]))
    keys = ("path", "splits", "workgroups", "points_per_wg", "k_block", "padded_d")
    return {k: v.value for k, v in zip(keys, vals)}


def kmeans_centroid_norms(C, norms=None, stream=None):
    """``norms[k] = sum_j C[k, j]**2`` (fp32), asynchronously on ``stream``."""
    import torch
    C = _matrix(C, "C")
    K, D = C.shape
    if norms is None:
        norms = torch.empty(K, dtype=torch.float32, device=C.device)
    _vector(norms, "norms", torch.float32, K, C.device)
    lib = load_library()
    with _on(C.device):
        _check(lib, lib.kmeans_centroid_norms(_ptr(C), K, D, _ptr(norms),
                                              _stream_handle(stream, C.device)))
    return norms


def _assign_args(X, C, norms, labels, min_dist):
    import torch
    X = _matrix(X, "X")
    C = _matrix(C, "C")
    N, D = X.shape
    K = C.shape[0]
    if C.shape[1] != D:
        raise ValueError(f"X has D={D} but C has D={C.shape[1]}")
    if C.device != X.device:
        raise ValueError(f"X is on {X.device} but C on {C.device}")
    _vector(norms, "norms", torch.float32, K, X.device)
    if labels is None:
        labels = torch.empty(N, dtype=torch.int32, device=X.device)
    if min_dist is None:
        min_dist = torch.empty(N, dtype=torch.float32, device=X.device)
    _vector(labels, "labels", torch.int32, N, X.device)
    _vector(min_dist, "min_dist", torch.float32, N, X.device)
    return X, C, norms, N, D, K, labels, min_dist


def kmeans_assign(X, C, norms, labels=None, min_dist=None, stream=None):
    """Nearest centroid per point: ``(labels int32 [N], min_dist fp32 [N])``."""
    X, C, norms, N, D, K, labels, min_dist = _assign_args(X, C, norms, labels, min_dist)
    lib = load_library()
    with _on(X.device):
        _check(lib, lib.kmeans_assign(_ptr(X), _ptr(C), _ptr(norms), N, D, K, _ptr(labels),
                                      _ptr(min_dist), _stream_handle(stream, X.device)))
    return labels, min_dist


def kmeans_assign_static(X, C, norms, labels=None, min_dist=None, stream=None):
    """``kmeans_assign`` whose K-split scratch is the library's fixed device
    buffer (no allocation inside the call; give ``labels`` and ``min_dist``
    to allocate nothing at all).  Calls that overlap on one GPU race."""
    X, C, norms, N, D, K, labels, min_dist = _assign_args(X, C, norms, labels, min_dist)
    lib = load_library()
    with _on(X.device):
        _check(lib, lib.kmeans_assign_static(_ptr(X), _ptr(C), _ptr(norms), N, D, K,
                                             _ptr(labels), _ptr(min_dist),
                                             _stream_handle(stream, X.device)))
    return labels, min_dist


def kmeans_assign_path(X, C, norms, path: int = PATH_AUTO, count: int = 0,
                       labels=None, min_dist=None, stream=None):
    """``kmeans_assign`` with a forced path (``PATH_DIRECT``, ``PATH_SPLIT`` or
    ``PATH_PERSISTENT``).  ``count``: for the split path the number of
    K-ranges (0: automatic); for the direct path 1 selects narrow point tiles
    (32 points per wave), any other value wide ones; for the persistent path
    the number of workgroups (0: one per CU)."""
    X, C, norms, N, D, K, labels, min_dist = _assign_args(X, C, norms, labels, min_dist)
    lib = load_library()
    with _on(X.device):
        _check(lib, lib.kmeans_assign_path(_ptr(X), _ptr(C), _ptr(norms), N, D, K,
                                           _ptr(labels), _ptr(min_dist), path, count,
                                           _stream_handle(stream, X.device)))
    return labels, min_dist


def kmeans_update(X, labels, C_old, C_new=None, norms=None, counts=None, means=None,
                  with_means: bool = False, stream=None, path: int = UPDATE_AUTO):
    """Centroid update from ``labels``: ``(C_new bf16 [K, D], norms fp32 [K],
    counts int32 [K], means fp32 [K, D] or None)``.  An empty cluster keeps
    its row of ``C_old``; labels outside ``[0, K)`` count for no cluster.
    ``C_new`` may be ``C_old`` itself (in-place update).  ``path``:
    ``UPDATE_AUTO``, ``UPDATE_SORT`` or ``UPDATE_BUCKETS`` (kmeans_update_path)."""
    import torch
    X = _matrix(X, "X")
    C_old = _matrix(C_old, "C_old")
    N, D = X.shape
    K = C_old.shape[0]
    if C_old.shape[1] != D:
        raise ValueError(f"X has D={D} but C_old has D={C_old.shape[1]}")
    if C_old.device != X.device:
        raise ValueError(f"X is on {X.device} but C_old on {C_old.device}")
    dev = C_old.device
    _vector(labels, "labels", torch.int32, N, dev)
    if C_new is None:
        C_new = torch.empty_like(C_old)
    else:
        C_new = _matrix(C_new, "C_new")
        if C_new.shape != C_old.shape:
            raise ValueError("C_new must have the shape of C_old")
    if norms is None:
        norms = torch.empty(K, dtype=torch.float32, device=dev)
    if counts is None:
        counts = torch.empty(K, dtype=torch.int32, device=dev)
    if means is None and with_means:
        means = torch.empty((K, D), dtype=torch.float32, device=dev)
    if C_new.device != dev:
        raise ValueError(f"C_new must be on {dev}")
    for t, name, dt, n in ((norms, "norms", torch.float32, K), (counts, "counts", torch.int32, K),
                           (means, "means", torch.float32, K * D)):
        if t is not None:
            _vector(t, name, dt, n, dev)
    lib = load_library()
    with _on(dev):
        _check(lib, lib.kmeans_update_path(_ptr(X), _ptr(labels), _ptr(C_old), N, D, K,
                                           _ptr(C_new), _ptr(norms), _ptr(counts), _ptr(means),
                                           int(path), _stream_handle(stream, dev)))
    return C_new, norms, counts, means


# ---- training a codebook by gradients ----

_DTYPES = None
_CURRENT_DEVICE = None


def _dtype(t, name):
    """kmeans_dtype_t of a tensor."""
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32 (got {t.dtype})")
    return code


def _launch(call, device, stream, *args):
    """``call(*args, stream handle)`` under ``device``, a non-OK status
    raised.  These calls are often a few microseconds of GPU time, so the
    common case (the tensors' device is the current one) does no more than
    look."""
    global _CURRENT_DEVICE
    if _CURRENT_DEVICE is None:
        import torch
        _CURRENT_DEVICE = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    handle = _stream_handle(stream, device)
    if device.index == _CURRENT_DEVICE():
        status = call(*args, handle)
    else:
        import torch
        with torch.cuda.device(device):
            status = call(*args, handle)
    if status != KMEANS_OK:
        _check(_lib, status)


def _rows(t, name, like=None, shape=None):
    """Check a 2-D CUDA tensor with unit column stride; its row stride.  A
    tensor of one row or less, or one column, may report any stride."""
    try:
        rows, cols = t.shape
        row_stride, col_stride = t.stride()
        on_gpu = t.is_cuda
    except (AttributeError, ValueError):
        import torch
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor") from None
        on_gpu = False
    if not on_gpu:
        raise ValueError(f"{name} must be a 2-D CUDA tensor (got {tuple(t.shape)}, {t.device})")
    if cols > 1 and col_stride != 1:
        raise ValueError(f"{name} must have unit column stride (strides {t.stride()})")
    if like is not None and (t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must be {like.dtype} on {like.device} "
                         f"(got {t.dtype} on {t.device})")
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name} must have shape {shape} (got {(rows, cols)})")
    if rows <= 1:
        return cols or 1
    if row_stride < cols:
        raise ValueError(f"{name}: rows overlap (strides {t.stride()})")
    return row_stride


def _flat(t, name):
    """A tensor of rows [..., D] as 2-D (a view: no copy is made)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() == 2:
        return t
    if t.dim() < 2:
        raise ValueError(f"{name} must have at least two dimensions (got {tuple(t.shape)})")
    try:
        return t.view(-1, t.shape[-1]) if t.numel() else t.reshape(-1, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}: rows of shape {tuple(t.shape)}, strides {t.stride()} are not "
                         "evenly spaced; make it contiguous") from None


def _labels(labels, index):
    """kmeans_label_t of a labels tensor on GPU ``index``."""
    import torch
    if isinstance(labels, torch.Tensor) and labels.get_device() == index and labels.is_contiguous():
        if labels.dtype is torch.int64:
            return INT64
        if labels.dtype is torch.int32:
            return INT32
    got = (f"{labels.dtype}, {labels.device}, contiguous={labels.is_contiguous()}"
           if isinstance(labels, torch.Tensor) else type(labels).__name__)
    raise ValueError(f"labels must be a contiguous int32 or int64 tensor on cuda:{index} "
                     f"(got {got})")


def kmeans_lookup(C, labels, scale: float = 1.0, out=None, stream=None):
    """``out[i] = scale * C[labels[i]]``, a row of zeros for a label outside
    ``[0, K)``.  ``C``: ``[K, D]`` bf16, fp16 or fp32, any row stride;
    ``labels``: int32 or int64 of any shape; ``out``: ``[*labels.shape, D]``."""
    c_stride = _rows(C, "C")
    code = _dtype(C, "C")
    K, D = C.shape
    kind = _labels(labels, C.get_device())
    if out is None:
        out = C.new_empty((*labels.shape, D))
        y_stride = D
    else:
        if tuple(out.shape) != (*labels.shape, D):
            raise ValueError(f"out must have shape {(*labels.shape, D)} (got {tuple(out.shape)})")
        y_stride = _rows(_flat(out, "out") if out.dim() != 1 else out.view(1, D), "out", like=C)
    lib = load_library()
    _launch(lib.kmeans_lookup, C.device, stream, C.data_ptr(), c_stride, labels.data_ptr(), kind,
            labels.numel(), D, K, code, scale, out.data_ptr(), y_stride)
    return out


def kmeans_lookup_grad(dY, labels, K: int, scale: float = 1.0, out=None,
                       accumulate: bool = False, stream=None):
    """Gradient of ``kmeans_lookup`` with respect to the table:
    ``out[k] = scale * sum of dY[i] over labels[i] == k``.  ``dY``:
    ``[*labels.shape, D]``; ``out``: ``[K, D]`` of ``dY``'s type (made when
    not given) or fp32; ``accumulate`` adds to ``out`` instead."""
    import torch
    if labels.dim() == 0:
        dY = dY.view(1, -1)
    dY = _flat(dY, "dY")
    y_stride = _rows(dY, "dY")
    code = _dtype(dY, "dY")
    N, D = dY.shape
    kind = _labels(labels, dY.get_device())
    if labels.numel() != N:
        raise ValueError(f"dY has {N} rows but there are {labels.numel()} labels")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = dY.new_empty((K, D))
    c_stride = _rows(out, "out", shape=(K, D))
    if out.get_device() != dY.get_device() or out.dtype not in (dY.dtype, torch.float32):
        raise ValueError(f"out must be {dY.dtype} or float32 on {dY.device} "
                         f"(got {out.dtype} on {out.device})")
    lib = load_library()
    _launch(lib.kmeans_lookup_grad, dY.device, stream, dY.data_ptr(), y_stride, labels.data_ptr(),
            kind, N, D, K, code, scale, int(accumulate), out.data_ptr(), _dtype(out, "out"),
            c_stride)
    return out


def _activation(name) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)} (got {name!r})")
    return code


def _bias(t, F, like):
    import torch
    if (not isinstance(t, torch.Tensor) or t.dtype is not like.dtype
            or t.get_device() != like.get_device() or t.numel() != F or not t.is_contiguous()):
        raise ValueError(f"bias must be a contiguous {like.dtype} tensor of {F} elements on "
                         f"{like.device}")
    return t


def kmeans_linear(X, W, bias=None, residual=None, activation: str = "none",
                  save_pre: bool = False, out=None, pre=None, stream=None):
    """``Z = X W^T + bias``, ``Y = act(Z) + residual``, one pass.  ``X``:
    ``[..., D]``, ``W``: ``[F, D]``, bf16 or fp16; ``activation``: a key of
    ``ACTIVATIONS``.  Returns ``Y``, or ``(Y, Z)`` with ``save_pre`` (or
    ``pre`` given), which ``kmeans_linear_grad`` needs."""
    lead = X.shape[:-1]
    X = _flat(X, "X")
    x_stride = _rows(X, "X")
    code = _dtype(X, "X")
    N, D = X.shape
    w_stride = _rows(W, "W", like=X)
    F, d = W.shape
    if d != D:
        raise ValueError(f"X has D={D} but W has D={d}")
    act = _activation(activation)
    if bias is not None:
        bias = _bias(bias, F, X).data_ptr()
    r_stride = 0
    if residual is not None:
        residual = _flat(residual, "residual")
        r_stride = _rows(residual, "residual", like=X, shape=(N, F))
        residual = residual.data_ptr()
    if out is None:
        out = X.new_empty((*lead, F))
        y_stride = F
    else:
        y_stride = _rows(_flat(out, "out"), "out", like=X, shape=(N, F))
    z_stride, z = 0, None
    if pre is not None:
        z_stride = _rows(_flat(pre, "pre"), "pre", like=X, shape=(N, F))
    elif save_pre:
        pre = X.new_empty((*lead, F))
        z_stride = F
    if pre is not None:
        z = pre.data_ptr()
    lib = load_library()
    _launch(lib.kmeans_linear, X.device, stream, X.data_ptr(), x_stride, W.data_ptr(), w_stride,
            bias, residual, r_stride, N, D, F, code, act, out.data_ptr(), y_stride, z, z_stride)
    return out if pre is None else (out, pre)


def kmeans_linear_grad(dY, X, W, Z=None, activation: str = "none", bias: bool = True,
                       need_dx: bool = True, need_dw: bool = True, stream=None):
    """Gradients of ``kmeans_linear`` for the output gradient ``dY``:
    ``(dX, dW, dbias)``, ``None`` for one not asked for.  ``Z``: the
    pre-activations that ``kmeans_linear`` kept (not needed for ``"none"``).
    The residual's gradient is ``dY`` itself.  With an activation, ``dY *
    act'(Z)`` is rounded to the inputs' 16-bit type before the products (the
    bias's sum takes it unrounded)."""
    import torch
    x_shape = X.shape
    X = _flat(X, "X")
    dY = _flat(dY, "dY")
    x_stride = _rows(X, "X")
    code = _dtype(X, "X")
    N, D = X.shape
    w_stride = _rows(W, "W", like=X)
    F = W.shape[0]
    if W.shape[1] != D:
        raise ValueError(f"X has D={D} but W has D={W.shape[1]}")
    y_stride = _rows(dY, "dY", like=X, shape=(N, F))
    act = _activation(activation)
    z_stride = 0
    if act == 0:
        Z = None
    elif Z is None:
        raise ValueError(f"activation {activation!r} needs Z")
    else:
        Z = _flat(Z, "Z")
        z_stride = _rows(Z, "Z", like=X, shape=(N, F))
    dX = X.new_empty(x_shape) if need_dx else None
    dW = X.new_empty((F, D)) if need_dw else None
    db = X.new_empty(F) if bias else None
    lib = load_library()
    _launch(lib.kmeans_linear_grad, X.device, stream, dY.data_ptr(), y_stride, X.data_ptr(),
            x_stride, W.data_ptr(), w_stride, _ptr(Z), z_stride, N, D, F, code, act, _ptr(dX), D,
            _ptr(dW), D, _ptr(db))
    return dX, dW, db


def _gradient_list(grads, out, device):
    """The list as kmeans_gradient_t entries: four 64-bit words each, the
    last one the type (and the reserved half, zero)."""
    index = device.index
    words = []
    for g, o in zip(grads, grads if out is None else out):
        if g.get_device() != index or not g.is_contiguous():
            raise ValueError(f"gradients must be contiguous tensors on one GPU "
                             f"(got {g.device}, strides {g.stride()})")
        n = g.numel()
        if o is not g and (o.dtype is not g.dtype or o.get_device() != index or o.numel() != n
                           or not o.is_contiguous()):
            raise ValueError(f"out must match the gradients: {g.dtype}, {n} elements, "
                             f"contiguous, on {device}")
        words += (g.data_ptr(), o.data_ptr(), n, _dtype(g, "gradients"))
    return array.array("q", words)


def _norm_of(grads, norm):
    import torch
    device = grads[0].device if len(grads) else torch.device("cuda", torch.cuda.current_device())
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=device)
    return _vector(norm, "norm", torch.float32, 1, device), device


def kmeans_gradient_norm(grads, norm=None, stream=None):
    """Global 2-norm of a list of contiguous gradients (bf16, fp16 and fp32
    mixed as they come): fp32 tensor of one element."""
    norm, device = _norm_of(grads, norm)
    items = _gradient_list(grads, None, device)
    lib = load_library()
    _launch(lib.kmeans_gradient_norm, device, stream, items.buffer_info()[0], len(grads),
            norm.data_ptr())
    return norm


def kmeans_clip_gradients(grads, max_norm: float, out=None, norm=None, stream=None):
    """Clip a list of contiguous gradients by their global 2-norm:
    ``g * min(1, max_norm / (norm + 1e-6))``, in place or into the list
    ``out``.  Returns ``(norm, clipped)``."""
    if out is not None and len(out) != len(grads):
        raise ValueError(f"out has {len(out)} tensors for {len(grads)} gradients")
    norm, device = _norm_of(grads, norm)
    items = _gradient_list(grads, out, device)
    lib = load_library()
    _launch(lib.kmeans_clip_gradients, device, stream, items.buffer_info()[0], len(grads),
            max_norm, norm.data_ptr())
    return norm, list(grads if out is None else out)


# ---- predicting labels ----

FP8_BLOCK = 128
_FP8 = _F32 = None


def _types():
    """float8_e4m3fn and float32, looked up once."""
    global _FP8, _F32
    import torch
    _FP8, _F32 = torch.float8_e4m3fn, torch.float32


def _typed_rows(t, name, dtype, index, shape=None):
    """Check rows of `dtype` on GPU `index`; their stride."""
    stride = _rows(t, name, shape=shape)
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be {dtype} on cuda:{index} (got {t.dtype} on {t.device})")
    return stride


def _as_rows(t, name):
    """Like _flat, quick for a matrix."""
    return t if getattr(t, "ndim", 0) == 2 else _flat(t, name)


def _blocks(D: int) -> int:
    return (D + FP8_BLOCK - 1) // FP8_BLOCK


def _gain(t, D, like):
    import torch
    if (not isinstance(t, torch.Tensor) or t.dtype is not like.dtype
            or t.get_device() != like.get_device() or t.numel() != D or not t.is_contiguous()):
        raise ValueError(f"weight must be a contiguous {like.dtype} tensor of {D} elements on "
                         f"{like.device}")
    return t.data_ptr()


def kmeans_rms_norm(X, weight=None, residual=None, eps: float = 1e-6, quantize: bool = False,
                    out=None, scales=None, sum=None, stream=None):
    """``H = X + residual``, ``Y = H / sqrt(mean(H^2) + eps) * weight`` along the
    last dimension, one pass.  ``X``: ``[..., D]`` bf16, fp16 or fp32.  With
    ``quantize`` the output is ``float8_e4m3fn`` with one fp32 scale for each
    128 columns (``scales``: ``[..., ceil(D / 128)]``).  Returns ``Y`` or ``(Y,
    scales)``, and ``H`` after it where there is a residual (``sum``: its
    tensor, which may be ``residual`` itself)."""
    x = _as_rows(X, "X")
    x_stride = _rows(x, "X")
    code = _dtype(x, "X")
    N, D = x.shape
    lead = X.shape[:-1] if x is not X else (N,)
    if weight is not None:
        weight = _gain(weight, D, x)
    r, r_stride, h, h_stride = None, 0, None, 0
    if residual is not None:
        r = _as_rows(residual, "residual")
        r_stride = _rows(r, "residual", like=x, shape=(N, D))
        r = r.data_ptr()
        if sum is None:
            sum = x.new_empty((*lead, D))
            h_stride = D
        else:
            h_stride = _rows(_as_rows(sum, "sum"), "sum", like=x, shape=(N, D))
        h = sum.data_ptr()
    elif sum is not None:
        raise ValueError("sum needs residual")
    y, y_stride, q, q_stride, s, s_stride = None, 0, None, 0, None, 0
    if quantize:
        if _FP8 is None:
            _types()
        blocks = (D + FP8_BLOCK - 1) // FP8_BLOCK
        if out is None:
            out = x.new_empty((*lead, D), dtype=_FP8)
            q_stride = D
        else:
            q_stride = _typed_rows(_as_rows(out, "out"), "out", _FP8, x.get_device(), (N, D))
        q = out.data_ptr()
        if scales is None:
            scales = x.new_empty((*lead, blocks), dtype=_F32)
            s_stride = blocks
        else:
            s_stride = _typed_rows(_as_rows(scales, "scales"), "scales", _F32, x.get_device(),
                                   (N, blocks))
        s = scales.data_ptr()
    else:
        if scales is not None:
            raise ValueError("scales need quantize=True")
        if out is None:
            out = x.new_empty((*lead, D))
            y_stride = D
        else:
            y_stride = _rows(_as_rows(out, "out"), "out", like=x, shape=(N, D))
        y = out.data_ptr()
    lib = load_library()
    _launch(lib.kmeans_rms_norm, x.device, stream, x.data_ptr(), x_stride, r, r_stride, weight, N,
            D, code, eps, h, h_stride, y, y_stride, q, q_stride, s, s_stride)
    if residual is not None:
        return (out, scales, sum) if quantize else (out, sum)
    return (out, scales) if quantize else out


def kmeans_rms_norm_grad(dY, H, weight=None, eps: float = 1e-6, dH=None, need_dw: bool = True,
                         stream=None):
    """Gradients of ``kmeans_rms_norm`` for the gradient ``dY`` of its output in
    ``X``'s type: ``(dX, dweight)``.  ``H``: the sum that it wrote (``X`` where
    there was no residual); ``dH``: the gradient that reaches the sum along the
    residual path, added to ``dX``, which is the residual's gradient too.
    ``dweight`` is ``None`` without a weight or with ``need_dw`` false."""
    h = _as_rows(H, "H")
    h_stride = _rows(h, "H")
    code = _dtype(h, "H")
    N, D = h.shape
    dY = _as_rows(dY, "dY")
    y_stride = _rows(dY, "dY", like=h, shape=(N, D))
    d, d_stride = None, 0
    if dH is not None:
        d = _as_rows(dH, "dH")
        d_stride = _rows(d, "dH", like=h, shape=(N, D))
        d = d.data_ptr()
    dw = None
    if weight is not None:
        if need_dw:
            dw = h.new_empty(D)
        weight = _gain(weight, D, h)
    dX = h.new_empty(H.shape)
    lib = load_library()
    _launch(lib.kmeans_rms_norm_grad, h.device, stream, dY.data_ptr(), y_stride, h.data_ptr(),
            h_stride, weight, d, d_stride, N, D, code, eps, dX.data_ptr(), D, _ptr(dw))
    return dX, dw


def kmeans_quantize(X, rows: int = 1, out=None, scales=None, stream=None):
    """``X`` (bf16, fp16 or fp32; ``[..., D]``, or ``[N, D]`` for blocks of 128 rows)
    as ``float8_e4m3fn`` values with an fp32 scale for each block of ``rows`` (1 or
    128) x 128: ``(Q, scales)``, ``scales`` ``[..., ceil(D / 128)]`` or
    ``[ceil(N / 128), ceil(D / 128)]``."""
    x = _as_rows(X, "X") if rows == 1 else X
    x_stride = _rows(x, "X")
    code = _dtype(x, "X")
    N, D = x.shape
    if rows not in (1, FP8_BLOCK):
        raise ValueError(f"rows must be 1 or {FP8_BLOCK} (got {rows})")
    if _FP8 is None:
        _types()
    shape = (-(-N // rows), _blocks(D))
    if out is None:
        out = x.new_empty(X.shape, dtype=_FP8)
        q_stride = D
    else:
        q_stride = _typed_rows(_as_rows(out, "out"), "out", _FP8, x.get_device(), (N, D))
    if scales is None:
        scales = x.new_empty(shape if x is X else (*X.shape[:-1], shape[1]), dtype=_F32)
        s_stride = shape[1]
    else:
        s_stride = _typed_rows(_as_rows(scales, "scales"), "scales", _F32, x.get_device(), shape)
    lib = load_library()
    _launch(lib.kmeans_quantize, x.device, stream, x.data_ptr(), x_stride, N, D, code, rows,
            out.data_ptr(), q_stride, scales.data_ptr(), s_stride)
    return out, scales


def kmeans_linear_fp8(X, x_scales, W, w_scales, bias=None, residual=None,
                      activation: str = "none", dtype=None, out=None, stream=None):
    """``Y = act(X W^T + bias) + residual`` of ``float8_e4m3fn`` operands with
    scales: ``X`` ``[..., D]`` with ``x_scales`` ``[..., ceil(D / 128)]`` (as
    ``kmeans_rms_norm`` or ``kmeans_quantize`` with ``rows=1`` give them), ``W``
    ``[F, D]`` with ``w_scales`` ``[ceil(F / 128), ceil(D / 128)]`` (``rows=128``).
    ``dtype``: of ``Y``, bias and residual (bfloat16 when not given, or
    ``out``'s).  Sums are fp32 for float32 outputs and up to 16 rows; for 16-bit
    outputs of more rows the 8-bit matrix instruction cuts each product to 2^-13
    of the largest among eight neighbouring columns."""
    if _FP8 is None:
        _types()
    x = _as_rows(X, "X")
    index = x.get_device()
    x_stride = _typed_rows(x, "X", _FP8, index)
    N, D = x.shape
    w_stride = _typed_rows(W, "W", _FP8, index)
    F, d = W.shape
    if d != D:
        raise ValueError(f"X has D={D} but W has D={d}")
    sx = _as_rows(x_scales, "x_scales")
    blocks = (D + FP8_BLOCK - 1) // FP8_BLOCK
    xs_stride = _typed_rows(sx, "x_scales", _F32, index, (N, blocks))
    ws_stride = _typed_rows(w_scales, "w_scales", _F32, index, (_blocks(F), blocks))
    act = _activation(activation)
    if out is None:
        if dtype is None:
            import torch
            dtype = torch.bfloat16
        out = x.new_empty((N, F) if x is X else (*X.shape[:-1], F), dtype=dtype)
        y_stride = F
    else:
        if dtype is not None and out.dtype is not dtype:
            raise ValueError(f"out must be {dtype} (got {out.dtype})")
        y_stride = _typed_rows(_as_rows(out, "out"), "out", out.dtype, index, (N, F))
    code = _dtype(out, "out")
    if bias is not None:
        bias = _bias(bias, F, out).data_ptr()
    r, r_stride = None, 0
    if residual is not None:
        r = _as_rows(residual, "residual")
        r_stride = _rows(r, "residual", like=out, shape=(N, F))
        r = r.data_ptr()
    lib = load_library()
    _launch(lib.kmeans_linear_fp8, x.device, stream, x.data_ptr(), x_stride, sx.data_ptr(),
            xs_stride, W.data_ptr(), w_stride, w_scales.data_ptr(), ws_stride, bias, r, r_stride, N,
            D, F, code, act, out.data_ptr(), y_stride)
    return out


class _Sampling(ctypes.Structure):
    """kmeans_sampling_t."""
    _fields_ = [("temperature", ctypes.c_float), ("top_p", ctypes.c_float),
                ("min_p", ctypes.c_float), ("top_k", ctypes.c_int32),
                ("temperatures", ctypes.c_void_p), ("top_ps", ctypes.c_void_p),
                ("min_ps", ctypes.c_void_p), ("top_ks", ctypes.c_void_p)]


def _setting(value, name, dtype, N, device, other):
    """(value for all rows, address of one for each) of a setting."""
    import torch
    if isinstance(value, torch.Tensor):
        return other, _vector(value, name, dtype, N, device).data_ptr()
    return value, None


def kmeans_sample(logits, uniforms, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None,
                  stream=None):
    """A label for each row of ``logits`` (``[..., K]`` bf16, fp16 or fp32) from
    the random numbers ``uniforms`` (fp32 in ``[0, 1)``, one for each row): labels
    in descending order of their logits, limited to the first ``top_k`` (0: all),
    to the first with ``top_p`` of their weight and to those with ``min_p`` of the
    largest weight, and the one at which their running weight exceeds ``uniform``
    of the whole.  Each setting is a number or a tensor of one for each row (fp32,
    ``top_k`` int32); a temperature of 0 takes the largest logit.  ``out``: int32
    (made when not given) or int64.  A row of -infinities and NaN gets -1."""
    import torch
    lead = logits.shape[:-1]
    z = _flat(logits, "logits") if logits.dim() != 1 else logits.view(1, -1)
    stride = _rows(z, "logits")
    code = _dtype(z, "logits")
    N, K = z.shape
    device = z.device
    _vector(uniforms, "uniforms", torch.float32, N, device)
    if out is None:
        out = torch.empty(lead, dtype=torch.int32, device=device)
    elif out.numel() != N:
        raise ValueError(f"out must have {N} elements (got {tuple(out.shape)})")
    kind = _labels(out, device.index)
    t, ts = _setting(temperature, "temperature", torch.float32, N, device, 1.0)
    k, ks = _setting(top_k, "top_k", torch.int32, N, device, 0)
    k = max(-1 << 31, min(k, (1 << 31) - 1))          # 32 bits of it would be taken else
    p, ps = _setting(top_p, "top_p", torch.float32, N, device, 1.0)
    m, ms = _setting(min_p, "min_p", torch.float32, N, device, 0.0)
    settings = _Sampling(t, p, m, k, ts, ps, ms, ks)
    lib = load_library()
    _launch(lib.kmeans_sample, device, stream, z.data_ptr(), stride, N, K, code,
            uniforms.data_ptr(), ctypes.addressof(settings), out.data_ptr(), kind)
    return out


def kmeans_release_workspace(stream=None):
    """Return the stream's workspace (scratch of the K-split path, the update,
    the lookup's gradient, the linear layers, the norm's gradient and the
    clipping, kept between calls) and its tile queue (the persistent path's) to the device's memory
    pool, in stream order; a later call on the stream allocates them again.
    Graphs that captured calls on the stream must not be replayed afterwards."""
    lib = load_library()
    _check(lib, lib.kmeans_release_workspace(_stream_handle(stream)))


def assign(X, C, norms=None):
    """Convenience: compute the norms if not given, then assign."""
    if norms is None:
        norms = kmeans_centroid_norms(C)
    return kmeans_assign(X, C, norms)
