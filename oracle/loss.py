"""Vocabulary losses in 64 bits, with the logits held: the plain definitions
that the library's kernels are checked against, and a bound on how far a
computation in binary32 with bf16 gradient entries may be from them.

Test infrastructure only; shares no code with the library.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24        # half a step of binary32, relative
UB = 2.0 ** -8        # half a step of bf16, relative (finfo.eps / 2)


def _logits(x, w, bias, scale, softcap):
    s = scale * (x @ w.t())
    if bias is not None:
        s = s + bias
    if softcap > 0:
        # (1 - tanh^2 as it stays exact where the tanh rounds to 1)
        return softcap * torch.tanh(s / softcap), 1.0 / torch.cosh(s / softcap) ** 2
    return s, torch.ones_like(s)


def _lse(z):
    top = z.max(1, keepdim=True).values
    base = torch.where(torch.isinf(top) & (top < 0), torch.zeros_like(top), top)
    return (base + torch.log(torch.exp(z - base).sum(1, keepdim=True)))[:, 0]


def xent(x, w, labels, bias=None, scale=1.0, softcap=0.0, smoothing=0.0, z_loss=0.0, dloss=None):
    """{"loss", "lse"} and, with dloss, {"dx", "dw", "dbias"}; float64 in and out."""
    V = w.shape[0]
    live = ((labels >= 0) & (labels < V)).nonzero()[:, 0]
    y = labels[live]
    z, slope = _logits(x[live], w, bias, scale, softcap)
    lse = _lse(z)
    zy = z.gather(1, y[:, None])[:, 0]
    part = lse - (1.0 - smoothing) * zy + z_loss * lse ** 2
    if smoothing > 0:
        part = part - smoothing * z.mean(1)
    loss, out_lse = x.new_zeros(x.shape[0]), x.new_zeros(x.shape[0])
    loss[live], out_lse[live] = part, lse
    out = {"loss": loss, "lse": out_lse}
    if dloss is not None:
        q = torch.exp(z - torch.where(torch.isinf(lse), torch.full_like(lse, math.inf), lse)[:, None])
        q = q * (1.0 + 2.0 * z_loss * lse[:, None]) if z_loss else q
        d = q - smoothing / V
        d[torch.arange(len(live), device=x.device), y] -= 1.0 - smoothing
        f = dloss[live][:, None] * slope
        _finish(out, x, w, live, d * f, q * f, scale)
    return out


def distill(x, w, ids, teacher, bias=None, temperature=1.0, scale=1.0, softcap=0.0, teacher_lse=None, dloss=None):
    V, T = w.shape[0], temperature
    there = (ids >= 0) & (ids < V) & (teacher != -math.inf)
    live = there.any(1).nonzero()[:, 0]
    there, at = there[live], ids[live].clamp(0, V - 1)
    z, slope = _logits(x[live], w, bias, scale, softcap)
    lse = _lse(z / T)
    t = torch.where(there, teacher[live] / T, torch.full_like(teacher[live], -math.inf))
    norm = teacher_lse[live] if teacher_lse is not None else torch.logsumexp(t, 1)
    p = torch.where(there, torch.exp(t - norm[:, None]), torch.zeros_like(t))
    logq = z.gather(1, at) / T - lse[:, None]
    terms = torch.where(p > 0, p * (t - norm[:, None] - logq), torch.zeros_like(p))
    loss, out_lse = x.new_zeros(x.shape[0]), x.new_zeros(x.shape[0])
    loss[live], out_lse[live] = T * T * terms.sum(1), lse
    out = {"loss": loss, "lse": out_lse, "weight": float(p.sum(1).max()) if len(live) else 0.0,
           "terms": float(terms.abs().sum(1).max()) if len(live) else 0.0}
    if dloss is not None:
        q = torch.exp(z / T - torch.where(torch.isinf(lse), torch.full_like(lse, math.inf), lse)[:, None])
        q = q * p.sum(1, keepdim=True)
        d = q.clone()
        d.scatter_add_(1, at, -p)
        f = T * dloss[live][:, None] * slope
        _finish(out, x, w, live, d * f, q * f, scale)
    return out


def _finish(out, x, w, live, d, q, scale):
    dx = x.new_zeros(x.shape)
    dx[live] = scale * (d @ w)
    out.update(dx=dx, dw=scale * (d.t() @ x[live]), dbias=d.sum(0), d=d, q=q, live=live)


def bounds(out, x, w, bias=None, scale=1.0, softcap=0.0, T=1.0, weight=1.0, terms=0.0):
    """Largest error of each result of a computation in binary32 (gradient
    entries d rounded to bf16), element by element, from first principles.

    Logits: K products of bf16 values, exact in binary32, summed in binary32:
    |ds| <= (K + 4) U (|scale| |x||w| + |bias|) (the summation bound and the
    scale's and bias's roundings).  tanh is good to 2^-21 of itself and has
    slope at most 1.
    Log-partition: moves by at most the largest |dz| / T; its exponentials are
    off by 2^-22 and by the rounding of their argument (U |z / T| each way),
    the sums of V positive terms by (64 + V / 16) U (at most 64 in a lane, then
    tiles), the logarithm and the products by 8 U of the result.
    Loss: T^2 weight times the errors of z and lse, where weight bounds the
    sum of the |weights| they enter with; terms: the sum of the |summands|,
    each good to 2^-20 (exponentials and roundings of the teacher's side).
    Gradient entries d: their probability part (out["q"]) is as exact as the
    probability, the target's part to 16 U; then bf16 (UB of the entry).
    Products: those errors through |w| and |x|, sums in binary32, and (keys
    without 32) the output's own rounding to bf16.
    """
    K, V = x.shape[1], w.shape[0]
    keep = ~torch.isnan(x).any(1)
    xf = torch.where(keep[:, None], x, torch.zeros_like(x))
    ds = (K + 4) * U * (abs(scale) * (xf.abs() @ w.abs().t()) + (bias.abs() if bias is not None else 0.0))
    z, _ = _logits(xf, w, bias, scale, softcap)
    dz = ds + 2.0 ** -21 * z.abs() if softcap > 0 else ds
    fin = torch.isfinite(z) & (z > -1e30)   # (lower ones are masked out: probability 0 either way)
    z, dz = torch.where(fin, z, torch.zeros_like(z)), torch.where(fin, dz, torch.zeros_like(dz))
    zmax, dzm = z.abs().max(1).values, dz.max(1).values
    lse = torch.where(torch.isfinite(out["lse"]), out["lse"].abs(), torch.zeros_like(out["lse"]))
    dlse = dzm / T + U * (8.0 * zmax / T + 64.0 + V / 16.0 + 8.0 + 8.0 * lse)
    tol = {"lse": dlse, "loss": T * T * (weight * (dzm / T + dlse + 16.0 * U * (zmax / T + lse)) + terms * 2.0 ** -20)}
    if "d" not in out:
        return tol
    live, d, q = out["live"], out["d"].abs(), out["q"].abs()
    dz, n, s = dz[live], max(len(out["live"]), 1), abs(scale)
    err = q * (dz / T + dlse[live][:, None] + 2.0 ** -20) + (d + q) * 16.0 * U
    if softcap > 0:   # the slope 1 - (z / cap)^2
        err = err + (q + d) * (2.0 * dz / softcap + 2.0 ** -20)
    errb = err + UB * (d + err)
    xa, wa = x[live].abs(), w.abs()
    tdx = x.new_zeros(x.shape)
    tdx[live] = s * (errb @ wa) + (V + 8) * U * s * ((d + errb) @ wa)
    tdw = s * (errb.t() @ xa) + (n + 8) * U * s * ((d + errb).t() @ xa)
    tiny = 1e-37
    tol.update(dx32=tdx + tiny, dw32=tdw + tiny, dx=tdx + UB * (out["dx"].abs() + tdx) + tiny,
               dw=tdw + UB * (out["dw"].abs() + tdw) + tiny,
               dbias=err.sum(0) + (n + 8) * U * (d + err).sum(0) + tiny)
    return tol
