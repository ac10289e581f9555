"""The bounds of 8-bit values with scales, on the CPU: they hold for a norm with its
residual formed in fp32, and reject what is a little wrong, also where values are
exactly zero."""

import pytest
import torch

import quantized_bounds as bounds
from prediction_reference import rms_norm


def quantized(y, rows):
    most = bounds.each_max(y, rows).float()
    s = torch.where(most == 0, 1.0, (most / 448).clamp(min=2.0 ** -126))
    each = s.repeat_interleave(rows, 0)[:y.shape[0]].repeat_interleave(128, 1)[:, :y.shape[1]]
    return (y.float() / each).to(torch.float8_e4m3fn), s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("N,D", [(64, 256), (17, 129), (5, 1000), (130, 77)])
@pytest.mark.parametrize("rows", [1, 128])
def test_bounds(N, D, rows, dtype):
    g = torch.Generator().manual_seed(N)
    x = torch.randn(N, D, generator=g).to(dtype)
    r = torch.where(torch.rand(N, D, generator=g) < 0.05, -x, torch.randn(N, D, generator=g).to(dtype))
    r[3, :128] = -x[3, :128]                             # a block of zeros
    y = rms_norm(x, None, r)[0]
    assert (y == 0).any()
    h = x.float() + r.float()
    Q, s = quantized(h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6), rows)
    rel = bounds.norm_rel(D)
    bounds.check(Q, s, y, rel, rows)

    def off(q, t):
        with pytest.raises(AssertionError):
            bounds.check(q, t, y, rel, rows)

    off(torch.zeros_like(Q), s)
    off(Q, torch.zeros_like(s))
    off(Q, s * 1.01)
    off(Q, s * 1.9)
    off(Q, torch.ones_like(s))
    flipped = Q.view(torch.uint8).clone()
    most = int(Q.float().abs().view(-1).argmax())
    flipped.view(-1)[most] ^= 2                          # a step or two of one value
    off(flipped.view(Q.dtype), s)
    left = Q.float()
    left.view(-1)[most] = 0
    off(left.to(Q.dtype), s)
    zero = Q.float()
    zero[y == 0] = 1
    off(zero.to(Q.dtype), s)
