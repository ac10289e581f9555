"""The bounds of the linear layer on 8-bit operands, on the CPU: they hold for the
definition with its roundings, and reject results that are a little wrong."""

import pytest
import torch

import linear_fp8_bounds as ref

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def quantized(x, rows):
    N, D = x.shape
    n, b = -(-N // rows), -(-D // 128)
    wide = torch.nn.functional.pad(x, (0, b * 128 - D, 0, n * rows - N)).view(n, rows, b, 128)
    s = wide.abs().amax((1, 3)) / 448
    q = (wide / s[:, None, :, None]).view(n * rows, b * 128)[:N, :D]
    return q.to(torch.float8_e4m3fn), s


@pytest.fixture(scope="module")
def operands():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(150, 300, generator=g) * torch.exp(torch.randn(150, 1, generator=g))
    return *quantized(x, 1), *quantized(torch.randn(200, 300, generator=g) * 0.06, 128)


def cut_product(X, sx, W, sw):
    """As the 8-bit matrix instruction forms it, in fp64: each product cut."""
    x, w = X.double(), W.double()
    z = torch.zeros(len(x), len(w), dtype=torch.float64)
    for c in range(0, x.shape[1], 8):
        p = x[:, None, c:c + 8] * w[None, :, c:c + 8]
        unit = 2.0 ** (torch.floor(torch.log2(p.abs().amax(2, keepdim=True).clamp(min=1e-9))) - 13)
        s = sx[:, c // 128].double()[:, None] * sw[torch.arange(len(w)) // 128, c // 128].double()
        z += s * (torch.trunc(p / unit) * unit).sum(2)
    return z


def off(got, want, t):
    with pytest.raises(AssertionError):
        ref.check(got, *want, t)


@pytest.mark.parametrize("t", [BF, FP, F32])
def test_bounds(operands, t):
    X, sx, W, sw = operands
    want = ref.linear_fp8(X, sx, W, sw, None, None, "none", t)
    y = want[0]
    ref.check(y.to(t), *want, t)
    if t != F32:
        ref.check(cut_product(*operands).to(t), *want, t)
    # scales of X and of W in bf16
    rounded = ref.product(X, sx.to(BF).float(), W, sw.to(BF).float(), True)[0]
    off(rounded.to(t), want, t)
    # the last column of k left out; one scale of its neighbour; rows or columns moved
    off(ref.product(X[:, :-1], sx, W[:, :-1], sw, True)[0].to(t), want, t)
    other = sx.clone()
    other[7, 1] = sx[7, 2]
    off(ref.product(X, other, W, sw, True)[0].to(t), want, t)
    off(y.roll(1, 0).to(t), want, t)
    off(y.roll(1, 1).to(t), want, t)
    wrong = y.clone()
    wrong[-1, -1] = 0
    off(wrong.to(t), want, t)


def test_bounds_of_few_rows(operands):
    X, sx, W, sw = operands
    assert (ref.product(X[:16], sx[:16], W, sw, True)[2] == 0).all()
    want = ref.linear_fp8(X[:16], sx[:16], W, sw, None, None, "none", FP)
    ref.check(want[0].to(FP), *want, FP)


def test_cut_takes_less_than_it_may(operands):
    """Less than 7 2^-13 of a group's largest product, so of all magnitudes."""
    _, mag, lost = ref.product(*operands)
    assert (lost > 0).any() and (lost < 7 * 2.0 ** -13 * mag).all()
