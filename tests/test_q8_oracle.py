"""Pins of the 8-bit matrices' oracle: rounding against exact fractions, slopes
against differences, the gradient's formulas against differences of the loss."""
import math
from fractions import Fraction

import pytest
import torch

from oracle import q8

F64 = torch.float64
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def nearest(f):
    low = math.floor(f)
    rest = f - low
    return low + (1 if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and low % 2) else 0)


@pytest.mark.parametrize("group", [0, 32])
def test_quantize_against_fractions(group):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, 70, generator=g)
    x[1] = x[1].to(torch.bfloat16).float()
    x[2] = torch.arange(70) * 0.5 - 17.0
    x[2, 0], x[2, 33], x[2, 65] = 127.0, 63.5, 127.0      # scales of 1 and 1/2: ties
    x[3] = 0.0
    q, s = q8.quantize(x, group)
    for m in range(4):
        for k0 in range(0, 70, group or 70):
            part = [Fraction(v.item()) for v in x[m, k0:k0 + (group or 70)]]
            sc = (s[m] if group == 0 else s[m, k0 // group]).item()
            top = max(abs(v) for v in part)
            if top:
                assert abs(Fraction(sc) - top / 127) <= top / 127 * Fraction(1, 2 ** 24)
            else:
                assert sc == 2.0 ** -126
            for i, v in enumerate(part):
                assert q[m, k0 + i].item() == nearest(v / Fraction(sc)), (m, k0 + i)


def test_not_finite_and_tiny():
    x = torch.randn(5, 40, generator=torch.Generator().manual_seed(2))
    x[0, 7], x[1, 35], x[2, 0] = math.nan, math.inf, -math.inf
    x[3] *= 1e-42
    q, s = q8.quantize(x, 32)
    assert torch.isnan(s[0, 0]) and not torch.isnan(s[0, 1]) and torch.isnan(s[1, 1]) and torch.isnan(s[2, 0])
    assert (q[0, :32] == 0).all() and (q[1, 32:] == 0).all() and (q[3] == 0).all() and (s[3] == 2.0 ** -126).all()
    assert (q[4].abs() <= 127).all() and q[4, :32].abs().max() == 127


@pytest.mark.parametrize("name", ACTS)
def test_slopes_against_differences(name):
    z = torch.linspace(-9, 9, 1801, dtype=F64) + 1e-3
    h = 1e-5
    d = (q8.act(name, z + h) - q8.act(name, z - h)) / (2 * h)
    # truncation h^2 / 6 of a third derivative below 4, rounding 2^-53 |z| / h
    assert (d - q8.slope(name, z)).abs().max() < 4 * h * h / 6 + 2.0 ** -53 * 12 / h
    assert q8.slope("relu", torch.zeros(1, dtype=F64)).item() == 0.0


@pytest.mark.parametrize("name", ["none", "gelu", "gelu_tanh", "silu"])
def test_backward_against_differences(name):
    """d/dt of sum(dy act(z + t (x D^T + b))) at 0 for directions D, b."""
    g = torch.Generator().manual_seed(3)
    M, N, K = 7, 5, 6
    dy = torch.randn(M, N, generator=g, dtype=F64)
    x, xs = q8.quantize(torch.randn(M, K, generator=g))
    z, zs = q8.quantize(torch.randn(M, N, generator=g) * 2, 32)
    out = q8.backward(dy, x, xs, z, zs, 32, name, torch.float32)
    D, b = torch.randn(N, K, generator=g, dtype=F64), torch.randn(N, generator=g, dtype=F64)
    v, base = q8.values(x, xs), q8.values(z, zs, 32)

    def loss(t):
        return (dy * q8.act(name, base + t * (v @ D.t() + b))).sum()

    h = 1e-4
    want = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)
    got = (out["dw"][0] * D).sum() + (out["dbias"][0] * b).sum()
    # fourth-order differences: h^4 / 30 of a fifth derivative; rounding 2^-53 |loss| / h
    assert abs(got - want) < 1e-8 * (1 + abs(want))
