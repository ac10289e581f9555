"""The operators of label prediction from their definitions, in fp64 on the CPU,
and the error bounds that the GPU results are held to.

Bounds.  Roundings are relative: 2^-24 for an fp32 operation, U[t] for the
output's type (bf16 2^-8, fp16 2^-11, fp32 2^-24), 2^-4 for e4m3, whose
subnormals are 2^-9 apart (half of it: 2^-10 of the scale).

A row's sum of squares is formed by lanes that add at most 64 terms (rows of up
to 16384 columns; D / 256 beyond) one after another and by a tree of at most 8
additions: ``depth`` roundings at most on the way of a term.  All terms of the
sum of squares have one sign, so its relative error is at most depth 2^-24,
that of r half of it, and 4 roundings more for the division, the sum with eps,
the root and the reciprocal.  H is rounded once (twice that in its square).
"""

import math

import numpy as np
import torch

from codebook_reference import EPS, TINY, U, act, check, cpu64  # noqa: F401

FP8_U = 2.0 ** -4
FP8_TINY = 2.0 ** -10
WEIGHT_BITS = 43


def depth(D):
    return max(64, D // 256) + 8


def rms_norm(X, weight=None, residual=None, eps=1e-6):
    """(y, bound on |y error| before its rounding, H, bound on |H error|)."""
    h = cpu64(X)
    if residual is not None:
        h = h + cpu64(residual)
    r = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + float(np.float32(eps)))
    y = h * r
    if weight is not None:
        y = y * cpu64(weight)
    t = X.dtype
    herr = EPS * h.abs()
    # r, H, and the two products
    yerr = (depth(X.shape[1]) / 2 + 8) * EPS * y.abs() + TINY[torch.float32]
    return y, yerr, h, herr * (1 + U[t]) + U[t] * h.abs() + TINY[t]


def rounded(v, err, t):
    return err * (1 + U[t]) + U[t] * v.abs() + TINY[t]


def block_scales(y, rows):
    """Scale of every value, and of every block."""
    N, D = y.shape
    n, b = -(-N // rows), -(-D // 128)
    s = torch.ones(n, b, dtype=torch.float64)
    for i in range(n):
        for j in range(b):
            most = y[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128].abs().max()
            if most != 0:
                s[i, j] = max(float(most) / 448, 2.0 ** -126)
    return s.repeat_interleave(rows, 0)[:N].repeat_interleave(128, 1)[:, :D], s


def check_quantized(Q, scales, y, yerr, rows, what=""):
    """Q times its scales against y, whose own error before rounding is yerr."""
    rel = float((yerr / y.abs().clamp(min=1e-300)).max()) if y.numel() else 0.0
    rel = min(rel, 1.0)
    each, blocks = block_scales(y, rows)
    check(scales, blocks, (rel + 2 * EPS) * blocks + TINY[torch.float32], what + " scales")
    got = cpu64(scales).repeat_interleave(rows, 0)[:y.shape[0]]
    got = got.repeat_interleave(128, 1)[:, :y.shape[1]]
    v = Q.cpu().float().double() * got
    # v / s and its product with 1 / s are rounded to fp32 before e4m3
    bound = torch.maximum(FP8_U * y.abs(), FP8_TINY * got) * (1 + 2.0 ** -20)
    bound = bound + yerr + 4 * EPS * y.abs() + rel * y.abs()
    check(v, y, bound + TINY[torch.float32], what + " values")


def rms_norm_grad(dY, H, weight=None, dH=None, eps=1e-6):
    """{name: (value, bound on its error)} of dX and dw."""
    dy, h, t = cpu64(dY), cpu64(H), H.dtype
    N, D = h.shape
    w = cpu64(weight) if weight is not None else torch.ones(D, dtype=torch.float64)
    d = cpu64(dH) if dH is not None else torch.zeros_like(h)
    r = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + float(np.float32(eps)))
    g = dy * w
    gh = (g * h).mean(1, keepdim=True)
    dx = r * g - h * r ** 3 * gh + d
    n = depth(D)
    # the sum of g h has terms of either sign: n + 2 roundings of their magnitudes
    err = EPS * ((n / 2 + 8) * r * g.abs()
                 + h.abs() * r ** 3 * (n + 2 + 1.5 * n + 16) * (g * h).abs().mean(1, keepdim=True)
                 + 2 * d.abs() + 2 * dx.abs())
    out = {"dX": (dx, rounded(dx, err, t))}
    dw = (dy * h * r).sum(0)
    err = (N + 40 + n / 2 + 8) * EPS * (dy * h * r).abs().sum(0)
    out["dw"] = (dw, rounded(dw, err, t))
    return out


def linear_fp8(X, x_scales, W, w_scales, bias, residual, activation, t):
    """(Y, bound on its error).  Products of e4m3 values are exact in fp32; a
    block's 128 are added in fp32, its sum scaled (two roundings) and added.

    For 16-bit outputs of more than 16 rows the 8-bit matrix instruction adds a
    block's products in groups of eight, aligned to the group's largest, of which
    it keeps 13 bits below: each of the seven others loses less than 2^-13 of the
    largest, which is no more than the group's magnitudes together."""
    N, D = X.shape
    b = x_scales.shape[1]
    sx = cpu64(x_scales).repeat_interleave(128, 1)[:, :D]
    sw = cpu64(w_scales).repeat_interleave(128, 0)[:W.shape[0]].repeat_interleave(128, 1)[:, :D]
    x, w = X.cpu().float().double() * sx, W.cpu().float().double() * sw
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z = z + cpu64(bias)
        mag = mag + cpu64(bias).abs()
    zerr = (D + 3 * b + 4) * EPS * mag
    if t != torch.float32 and N > 16:
        zerr = zerr + 7 * 2.0 ** -13 * mag
    y = act(z, activation)
    yerr = 1.13 * zerr + (0 if activation == "none" else 1e-6 * (1 + z.abs()))
    if residual is not None:
        y = y + cpu64(residual)
        yerr = yerr + EPS * y.abs()
    return y, rounded(y, yerr, t)


def sample(logits, u, temperature, top_k, top_p, min_p):
    """For each row the ranks' order and the range of labels that roundings of
    the weights allow: (list of sets).  Each argument after ``u`` is one number
    per row.  A weight is rounded to 2^-43 and its exponential may be off by one
    unit, so a running sum of K of them by K units, and by 2^-50 of itself where
    it is compared in double precision."""
    allowed = []
    for i, row in enumerate(logits.detach().cpu().float().double().numpy()):
        z = np.where(np.isnan(row), -np.inf, row)
        K = len(z)
        top = int(np.argmax(z))
        t, k, p, m = (float(temperature[i]), int(top_k[i]), float(np.float32(top_p[i])),
                      float(np.float32(min_p[i])))
        if z[top] == -np.inf:
            allowed.append({-1})
            continue
        if not t > 0:
            allowed.append({top})
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            w = np.where(z == z[top], 1.0, np.exp((z - z[top]) / np.float64(np.float32(t))))
        w = np.nan_to_num(w)
        order = np.lexsort((np.arange(K), -z))
        order = order[w[order] >= 2.0 ** -(WEIGHT_BITS + 1)]
        if k > 0:
            order = order[:k]
        sums = np.cumsum(w[order])
        inexact = int((w[order] != 1).sum())            # weights of 1 have no rounding
        slack = inexact * 2.0 ** -WEIGHT_BITS + (sums[-1] * 2.0 ** -50 if inexact else 0.0)
        ends = {len(order)}
        if p < 1:
            target = p * sums[-1]
            ends = {int(np.searchsorted(sums, target + s)) + 1 for s in (-2 * slack, 2 * slack)}
        ends = {min(e, len(order)) for e in ends}
        if m > 0:
            mm = min(m, 1.0)
            ends = {min(e, max(1, int((w[order] >= mm * (1 + s)).sum())))
                    for e in ends for s in (-2.0 ** -42, 2.0 ** -42 if mm < 1 else 0.0)}
        labels = set()
        for e in ends:
            total = sums[e - 1]
            uu = min(max(float(np.float32(u[i])) if not np.isnan(u[i]) else 0.0, 0.0), 1.0)
            lo = int(np.searchsorted(sums[:e], uu * total - 2 * slack, side="right"))
            hi = int(np.searchsorted(sums[:e], uu * total + 2 * slack, side="right"))
            if uu == 0.0:
                hi = 0
            labels |= {int(order[min(x, e - 1)]) for x in range(lo, hi + 1)}
        allowed.append(labels)
    return allowed


def check_sample(got, allowed, what="", most_open=0.02):
    got = got.detach().cpu().reshape(-1).tolist()
    assert len(got) == len(allowed)
    bad = [(i, g, sorted(a)[:4]) for i, (g, a) in enumerate(zip(got, allowed)) if g not in a]
    assert not bad, f"{what}: {len(bad)} of {len(got)} rows, first {bad[0]}"
    open_rows = sum(len(a) > 1 for a in allowed)
    assert open_rows <= max(1, most_open * len(allowed)), f"{what}: {open_rows} rows undecided"
