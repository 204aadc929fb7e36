"""Oracle of the 8-bit matrices (test infrastructure only): the definitions in
binary64 torch, on the exact inputs that the library is given, and bounds on
how far a binary32 computation of them may be off, element by element.

    scale = binary32(max(max |x| / 127, 2^-126)),  q = x / scale to the nearest, ties to even
    y = act(x_scale w_scale (q_x . q_w) + bias)
    dz = dy act'(z),  dw = dz^T . x,  dbias = sum of dz's rows
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64
U = 2.0 ** -24                       # half a unit of binary32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}   # half the smallest subnormal
# sup |act'| (gelu' = Phi + x phi peaks at x = sqrt 2, silu' near 2.40)
LIPSCHITZ = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "gelu_tanh": 1.13, "silu": 1.10}


def quantize(x, group=0):
    """(q int8, scale binary32) of a binary64 or narrower x (M, K)."""
    x = x.to(F64)
    M, K = x.shape
    size = group or max(K, 1)
    qs, ss = [], []
    for k in range(0, K, size):
        part = x[:, k:k + size]
        top = part.abs().amax(1)
        bad = ~torch.isfinite(part).all(1)
        # (a binary64 quotient of binary32 values rounds to binary32 as the exact one does)
        s = (torch.where(bad, torch.zeros_like(top), top) / 127.0).clamp(min=2.0 ** -126).to(torch.float32)
        t = part / s.to(F64)[:, None]
        q = torch.where(bad[:, None], torch.zeros_like(t), torch.round(t))
        qs.append(q.to(torch.int8))
        ss.append(torch.where(bad, torch.full_like(s, math.nan), s))
    if not qs:
        return torch.zeros((M, 0), dtype=torch.int8, device=x.device), torch.zeros((M, 0), device=x.device)
    scale = torch.stack(ss, 1)
    return torch.cat(qs, 1), scale if group else scale[:, 0]


def values(q, scale, group=0):
    """What q and scale stand for, binary64."""
    if scale.dim() == 1:
        return q.to(F64) * scale.to(F64)[:, None]
    return q.to(F64) * scale.to(F64)[:, torch.arange(q.shape[1], device=q.device) // group]


def act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.where(torch.isnan(z), z, torch.zeros_like(z)))
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(name, z):
    """d act / dz; the rectifier's is 0 at 0."""
    if name == "relu":
        return torch.where(torch.isnan(z), z, (z > 0).to(F64))
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return p + z * p * (1.0 - p) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def linear(x, xs, w, ws, bias, name, dtype):
    """(y, tolerance) for integers x (M, K), w (N, K) and their scales.

    The sum is exact; its conversion, two products and a fused addition round
    once each: 3 U of the scaled sum and U of the pre-activation v, carried
    through the activation, whose own roundings are within 8 U (|v| + |y|)."""
    p = (x.to(F64) @ w.to(F64).t()) * ws.to(F64) * xs.to(F64)[:, None]
    v = p if bias is None else p + bias.to(F64)
    y = act(name, v)
    tol = LIPSCHITZ[name] * U * (3.0 * p.abs() + v.abs()) + 8.0 * U * (v.abs() + y.abs()) + LEAST[torch.float32] * 4
    return y, tol * (1 + 2 ** -7) + HALF[dtype] * y.abs() + LEAST[dtype]


# act' in binary32, absolute: 0.75e-7 of the distribution function (half of 1.5e-7), values of at most 1.2
# rounded a few times, and z's own rounding (|z act''| < 1)
SLOPE = 0.75e-7 + 8.0 * U


def backward(dy, x, xs, z, zs, group, name, dtype):
    """{"dz", "dw", "dbias": (value, tolerance)}.

    dz: the slope's error times |dy|, one product, one rounding to bf16.
    dbias: M additions of binary32.  dw: dz's error, its product with the scale
    and that one's rounding to bf16 (for a binary32 dw: to the sum of two bf16
    parts, the second within 2^-8 of what the first leaves) in every term, then M
    additions (of each part)."""
    dy = dy.to(F64)
    M = dy.shape[0]
    dz, e = dy, torch.zeros_like(dy)
    if name != "none":
        dz = dy * slope(name, values(z, zs, group))
        e = dy.abs() * SLOPE + 2.0 * U * dz.abs()
    half, least = HALF[torch.bfloat16], LEAST[torch.bfloat16]
    out = {"dz": (dz, e + half * dz.abs() * (1 + 2 ** -7) + least)}
    # (sums of 8 rows, then of 4 of those, then of the blocks: never more than M additions deep)
    add = (M + 2) * U
    out["dbias"] = (dz.sum(0), e.sum(0) * (1 + add) + add * dz.abs().sum(0))
    if x is not None:
        v = values(x, xs)
        operand = half if dtype is torch.bfloat16 else half * half * (1 + 2 ** -7)
        each = dz.abs() * (operand + 4.0 * U) + e * (1 + half)
        terms = dz.abs().t() @ v.abs()
        dw = dz.t() @ v
        tol = (each.t() @ v.abs()) * (1 + add) + 2.0 * add * terms + least * x.to(F64).abs().sum(0)
        out["dw"] = (dw, tol + HALF[dtype] * (dw.abs() + tol) + LEAST[dtype])
    return out
