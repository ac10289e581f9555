"""The codebook-training operators from their definitions, in fp64 on the CPU,
and the error bounds that the GPU results are held to.

Bounds.  A sum of n products in fp32, in any order, is off by at most
n 2^-24 S (S the sum of the products' magnitudes; products of 16-bit values
are exact or add half a unit of 2^-24 each).  A rounding to bf16 adds 2^-8,
to fp16 2^-11, to fp32 2^-24 of the value, and at most half the smallest
subnormal (fp16: 2^-25).  The activations are evaluated in fp32 from
v_exp_f32 and v_rcp_f32 (1 unit each) and, for gelu, a polynomial of error
1.5e-7: 1e-6 (1 + |z|) covers each, and their slopes stay below 1.13.
"""

import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-38}
EPS = 2.0 ** -24
SLOPE = 1.13


def _erf(z):
    return torch.erf(z)


def act(z, name):
    """act(z) in fp64."""
    if name == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        return z * torch.sigmoid(2 * u)
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, name):
    """act'(z) in fp64, from the formula."""
    if name == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), torch.ones_like(z))
    if name == "gelu":
        return (0.5 * torch.special.erfc(-z * math.sqrt(0.5))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        s = torch.sigmoid(2 * u)
        return s + z * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def cpu64(t):
    return None if t is None else t.detach().cpu().double()


def linear(X, W, bias=None, residual=None, activation="none"):
    """(Y, Z, bound on |Y error|, bound on |Z error|) for 16-bit inputs."""
    dt = X.dtype
    x, w = cpu64(X), cpu64(W)
    z = x @ w.t()
    mag = x.abs() @ w.abs().t()
    if bias is not None:
        z = z + cpu64(bias)
        mag = mag + cpu64(bias).abs()
    zerr = (X.shape[1] + 2) * EPS * mag
    y = act(z, activation)
    yerr = SLOPE * zerr + (0 if activation == "none" else 1e-6 * (1 + z.abs()))
    if residual is not None:
        y = y + cpu64(residual)
        yerr = yerr + EPS * y.abs()
    return (y, z, yerr * (1 + U[dt]) + U[dt] * y.abs() + TINY[dt],
            zerr * (1 + U[dt]) + U[dt] * z.abs() + TINY[dt])


def linear_grad(dY, X, W, Z=None, activation="none"):
    """{name: (value, bound on its error)} of dX, dW, db."""
    dt = X.dtype
    u, tiny = U[dt], TINY[dt]
    dy, x, w = cpu64(dY), cpu64(X), cpu64(W)
    if activation == "none":
        dz, dzerr = dy, torch.zeros_like(dy)
    else:
        z = cpu64(Z)
        dz = dy * act_slope(z, activation)
        dzerr = dy.abs() * 2e-6 * (1 + z.abs())
    op = dzerr if activation == "none" else dzerr * (1 + u) + u * dz.abs() + tiny   # as rounded
    N, F = dy.shape
    out = {}
    for name, a, b, e, n in (("dX", dz, w, op, F), ("dW", dz.t(), x, op.t(), N)):
        v = a @ b
        err = e @ b.abs() + (n + 2) * EPS * ((a.abs() + e) @ b.abs())
        out[name] = (v, err * (1 + u) + u * v.abs() + tiny)
    v = dz.sum(0)
    err = dzerr.sum(0) + (N + 2) * EPS * dz.abs().sum(0)
    out["db"] = (v, err * (1 + u) + u * v.abs() + tiny)
    return out


def lookup_grad(dY, labels, K, scale, out_dtype, into=None):
    """(dC, bound on its error); `into`: the values accumulated to."""
    dy, lab = cpu64(dY).numpy(), labels.detach().cpu().numpy().reshape(-1).astype(np.int64)
    seen = (lab >= 0) & (lab < K)
    D = dy.shape[-1]
    dy = dy.reshape(-1, D)
    s = np.zeros((K, D))
    m = np.zeros((K, D))
    np.add.at(s, lab[seen], dy[seen])
    np.add.at(m, lab[seen], np.abs(dy[seen]))
    n = np.bincount(lab[seen], minlength=K)[:, None]
    scale = float(np.float32(scale))
    v = s * scale
    err = (n + 2) * EPS * m * abs(scale)
    if into is not None:
        v = v + cpu64(into).numpy()
        err = err + EPS * np.abs(v)
        untouched = np.broadcast_to(n == 0, v.shape)
    u = U[out_dtype]
    bound = err * (1 + u) + u * np.abs(v) + TINY[out_dtype]
    if into is not None:
        bound = np.where(untouched, 0.0, bound)
    return torch.from_numpy(v), torch.from_numpy(bound)


def check(got, want, bound, what=""):
    g = cpu64(got).reshape(want.shape)
    bad = ~((g - want).abs() <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
        f"{float(((g - want).abs() / bound).nan_to_num(nan=float('inf')).max()):.3g} bounds, "
        f"first at {torch.nonzero(bad)[0].tolist()}: got {float(g[bad][0])}, "
        f"want {float(want[bad][0])}")
