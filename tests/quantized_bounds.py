"""Values in 8 bits with a scale for each block of 128 columns, against values of
which a relative error is known: bounds taken block by block.

Let every value be known to a factor 1 +- rel.  The block's largest magnitude then
is, and its scale to 1 +- (rel + 2^-24).  A value is off by rel of itself, its
quotient by 2^-24 more, and the rounding to e4m3 by half the distance of its
neighbours: 2^-4 of the power of two at or below the quotient, 2^-10 for
quotients below 2^-6.  A value of zero is zero, and so is its quotient."""

import torch

from codebook_reference import EPS, cpu64
from prediction_reference import block_scales, depth


def norm_rel(D):
    """Relative error of kmeans_rms_norm's y: r, H and two products."""
    return (depth(D) / 2 + 8) * EPS


def check(Q, scales, y, rel, rows, what=""):
    each, blocks = block_scales(y, rows)
    s = cpu64(scales)
    assert s.shape == blocks.shape, what
    off = (s / blocks - 1).abs()
    off = torch.where(blocks == 2.0 ** -126, off.clamp(max=rel), off)     # the least scale
    assert bool((off <= rel + 2 * EPS).all()), f"{what} scales: {float(off.max()):.3g}, {rel:.3g}"
    assert bool((s[(each_max(y, rows) == 0)] == 1).all()), f"{what} scales of zeros"
    s = s.repeat_interleave(rows, 0)[:y.shape[0]].repeat_interleave(128, 1)[:, :y.shape[1]]
    q = Q.detach().cpu().float().double()
    v = y.abs() / s * (1 + rel + 4 * EPS)
    half = torch.where(v < 2.0 ** -6, torch.tensor(2.0 ** -10, dtype=torch.float64),
                       torch.ldexp(torch.ones_like(v), torch.frexp(v).exponent - 5))
    bound = torch.where(y == 0, 0.0, half * s + (rel + 4 * EPS) * y.abs())
    bad = ~((q * s - y).abs() <= bound)
    assert not bool(bad.any()), (
        f"{what} values: {int(bad.sum())} of {bad.numel()} off, first at "
        f"{torch.nonzero(bad)[0].tolist()}: {float((q * s)[bad][0])}, {float(y[bad][0])}")


def each_max(y, rows):
    """Largest magnitude of every block."""
    n, b = -(-y.shape[0] // rows), -(-y.shape[1] // 128)
    wide = torch.nn.functional.pad(y, (0, b * 128 - y.shape[1], 0, n * rows - y.shape[0]))
    return wide.view(n, rows, b, 128).abs().amax((1, 3))
