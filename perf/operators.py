"""The vocabulary losses of this library, as cases to measure.

A language model's last linear layer is its widest product: M tokens of K
features against a vocabulary of V rows.  The loss that follows needs one
number per token of the M x V logits, and its gradient needs them once more,
so the operators here take the layer's input and weight and never hold the
logits:

  linear_xent      softmax cross entropy of each token's label (ignored rows,
                   label smoothing, the squared log-partition penalty, logit
                   scale, tanh cap, bias), and its gradient
  linear_distill   Kullback-Leibler divergence from a teacher known by its k
                   top logits per token, at a temperature, and its gradient

`own` False computes them in plain torch in 32 bits, `own` True calls the
library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def _case(name, op, train, M, V, K, **more):
    c = {"name": name, "op": op, "train": train, "M": M, "V": V, "K": K, "keep": 1.0, "bias": False, "scale": 1.0,
         "cap": 0.0, "smooth": 0.0, "zloss": 0.0, "k": 0, "temp": 1.0, "tlse": False, "weights": False, "pad": 0}
    c.update(more)
    return c


def listed():
    return [
        # the log-probability of one chosen token (a decode step that reports
        # its score): the weight streams past a single row
        _case("score_1_token", "xent", False, 1, 32000, 4096),
        # scores of a decode batch over a wide vocabulary
        _case("score_24_tokens_wide", "xent", False, 24, 128256, 4096),
        # evaluation of a short text on a small layer with an odd vocabulary
        _case("score_509_tokens_odd", "xent", False, 509, 50257, 768),
        # evaluation (perplexity) of a long text
        _case("score_4096_tokens", "xent", False, 4096, 32000, 4096),
        # a short fine-tuning batch: bias and label smoothing
        _case("train_333_tokens_smooth", "xent", True, 333, 30522, 768, bias=True, smooth=0.1),
        # masked-token training: 15 % of the positions carry a label
        _case("train_masked_15_percent", "xent", True, 8192, 30522, 768, bias=True, keep=0.15),
        # next-token training, with the log-partition penalty
        _case("train_4096_tokens_zloss", "xent", True, 4096, 32000, 4096, zloss=1e-4),
        # the largest: a wide vocabulary, capped logits, prompts left out
        _case("train_8192_tokens_wide_cap", "xent", True, 8192, 128256, 4096, keep=0.9, cap=30.0),
        # a student checked against its teacher on a few tokens
        _case("distill_score_7_tokens", "distill", False, 7, 32000, 4096, k=20, temp=2.0),
        # distillation of a small student, tokens weighted
        _case("distill_train_1000_tokens", "distill", True, 1000, 50257, 768, k=16, temp=2.0, weights=True, keep=0.95),
        # distillation with many teacher logits and the teacher's own log-partition
        _case("distill_train_2048_top64", "distill", True, 2048, 32000, 4096, k=64, tlse=True),
        # distillation over a wide vocabulary
        _case("distill_train_4096_wide", "distill", True, 4096, 128256, 2048, k=32, temp=1.5, bias=True),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["xent", "distill"])
    train = rng.random() < 0.6
    V = _between(rng, 1000, 131072)
    K = _between(rng, 256, 5120)
    how = rng.random()
    K = max(64, K // 64 * 64) if how < 0.7 else K // 8 * 8 if how < 0.9 else K
    M = _between(rng, 48 if train else 1, 8192)
    # no more work than the largest listed case
    M = max(1, min(M, 8192 * 128256 * 4096 // (V * K)))
    c = {"op": op, "train": train, "M": M, "V": V, "K": K, "keep": rng.choice([1.0, 1.0, 0.9, 0.5, 0.15]),
         "bias": rng.random() < 0.4, "scale": rng.choice([1.0, 1.0, 0.125]), "cap": rng.choice([0.0, 0.0, 0.0, 30.0]),
         "smooth": 0.0, "zloss": 0.0, "k": 0, "temp": 1.0, "tlse": False, "weights": rng.random() < 0.3,
         "pad": rng.choice([0, 0, 0, 64, 5])}
    if op == "xent":
        c["smooth"] = rng.choice([0.0, 0.0, 0.1])
        c["zloss"] = rng.choice([0.0, 0.0, 1e-4])
    else:
        c["k"] = _between(rng, 1, 128)
        c["temp"] = rng.choice([1.0, 2.0, 4.0])
        c["tlse"] = rng.random() < 0.3
    return c


def _rows(case):
    """How many rows carry a target."""
    return max(1, int(round(case["keep"] * case["M"])))


def prepare(case, seed):
    M, V, K, k = case["M"], case["V"], case["K"], case["k"]
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    w = (torch.randn((V, K), generator=g, device=DEV) * 0.02).to(torch.bfloat16)
    x = torch.randn((M, K), generator=g, device=DEV)
    n = _rows(case)
    live = torch.zeros(M, dtype=torch.bool, device=DEV)
    live[torch.randperm(M, generator=g, device=DEV)[:n]] = True
    s = {"case": case}
    if case["op"] == "xent":
        top = torch.randint(0, V, (M,), generator=g, device=DEV)
        s["labels"] = torch.where(live, top, torch.full_like(top, -100))
    else:
        # k different ids a row, strongest teacher logit first; some rows name
        # fewer, their places filled up with -1
        at = (torch.arange(k, device=DEV) + 0.999 * uniform(M, k)) * (V / k)
        ids = at.to(torch.int64).clamp_(max=V - 1)
        ids = ids.gather(1, uniform(M, k).argsort(1))
        top = ids[:, 0].clone()
        t = 12.0 - torch.cumsum(-torch.log(uniform(M, k).clamp_(min=1e-6)), 1)
        few = uniform(M, 1) < 0.1
        gone = (few & (torch.arange(k, device=DEV) >= (k + 1) // 2)) | ~live[:, None]
        s["ids"] = torch.where(gone, torch.full_like(ids, -1), ids)
        s["teacher"] = t.contiguous()
        if case["tlse"]:
            lse = torch.where(gone, torch.full_like(t, -1e30), t / case["temp"]).logsumexp(1)
            s["teacher_lse"] = lse + 0.2 * uniform(M)
    # a model that has learnt something: the target's logit stands out by a
    # random amount
    wt = w[top].float()
    x += (14.0 / max(case["scale"], 0.3) * uniform(M, 1)) * wt / wt.square().sum(1, keepdim=True)
    if case["pad"]:
        wide = torch.zeros((M, K + case["pad"]), dtype=torch.bfloat16, device=DEV)
        wide[:, :K] = x.to(torch.bfloat16)
        s["x"] = wide[:, :K]
    else:
        s["x"] = x.to(torch.bfloat16)
    s["w"] = w
    s["bias"] = 0.5 * torch.randn(V, generator=g, device=DEV) if case["bias"] else None
    # the mean over the rows with a target, or weighted tokens
    s["dloss"] = (0.25 + uniform(M) if case["weights"] else torch.ones(M, device=DEV)) / n
    return s


def _logits(s, c):
    z = s["x"].float() @ s["w"].float().t()
    if c["scale"] != 1.0:
        z = z * c["scale"]
    if s["bias"] is not None:
        z = z + s["bias"]
    if c["cap"] > 0:
        z = c["cap"] * torch.tanh(z / c["cap"])
    return z


def _log_partition(z):
    top = z.amax(1, keepdim=True)
    return (top + torch.log(torch.exp(z - top).sum(1, keepdim=True)))[:, 0]


def _gradients(s, c, z, dz):
    """From the gradient by the (capped) logits to those by x, w and the bias."""
    if c["cap"] > 0:
        dz = dz * (1.0 - (z / c["cap"]).square())
    dx = dz @ s["w"].float()
    dw = dz.t() @ s["x"].float()
    if c["scale"] != 1.0:
        dx, dw = dx * c["scale"], dw * c["scale"]
    out = {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}
    if s["bias"] is not None:
        out["dbias"] = dz.sum(0)
    return out


def _xent(s, c):
    z = _logits(s, c)
    V = z.shape[1]
    live = s["labels"] >= 0
    y = s["labels"].clamp(min=0)[:, None]
    lse = _log_partition(z)
    loss = lse - (1.0 - c["smooth"]) * z.gather(1, y)[:, 0] + c["zloss"] * lse.square()
    if c["smooth"] > 0:
        loss = loss - c["smooth"] * z.mean(1)
    zero = torch.zeros_like(lse)
    out = {"loss": torch.where(live, loss, zero), "lse": torch.where(live, lse, zero)}
    if c["train"]:
        dl = torch.where(live, s["dloss"], zero)[:, None]
        dz = torch.exp(z - lse[:, None]) * (1.0 + 2.0 * c["zloss"] * lse[:, None])
        if c["smooth"] > 0:
            dz -= c["smooth"] / V
        dz.scatter_add_(1, y, torch.full_like(dl, c["smooth"] - 1.0))
        dz *= dl
        out.update(_gradients(s, c, z, dz))
    return out


def _distill(s, c):
    z = _logits(s, c)
    T = c["temp"]
    there = s["ids"] >= 0
    at = s["ids"].clamp(min=0)
    live = there.any(1)
    zero = torch.zeros(z.shape[0], device=z.device)
    t = torch.where(there, s["teacher"] / T, torch.full_like(s["teacher"], -math.inf))
    tlse = s["teacher_lse"] if c["tlse"] else torch.where(live, _log_partition(t), zero)
    logp = t - tlse[:, None]
    p = torch.exp(logp)
    lse = _log_partition(z / T)
    logq = z.gather(1, at) / T - lse[:, None]
    kl = torch.where(there, p * (logp - logq), torch.zeros_like(p)).sum(1)
    out = {"loss": torch.where(live, T * T * kl, zero), "lse": torch.where(live, lse, zero)}
    if c["train"]:
        dl = torch.where(live, T * s["dloss"], zero)[:, None]
        dz = torch.exp(z / T - lse[:, None]) * p.sum(1, keepdim=True)
        dz.scatter_add_(1, at, -p)
        dz *= dl
        out.update(_gradients(s, c, z, dz))
    return out


def _with_library(s, c):
    import dynamic_shape_gemm_amd as mkp

    more = {"bias": s["bias"], "scale": c["scale"], "softcap": c["cap"]}
    if c["op"] == "xent":
        args = (s["x"], s["w"], s["labels"])
        more.update(smoothing=c["smooth"], z_loss=c["zloss"])
        forward, backward = mkp.linear_xent, mkp.linear_xent_backward
    else:
        args = (s["x"], s["w"], s["ids"], s["teacher"])
        more.update(temperature=c["temp"], teacher_lse=s.get("teacher_lse"))
        forward, backward = mkp.linear_distill, mkp.linear_distill_backward
    loss, lse = forward(*args, **more)
    out = {"loss": loss, "lse": lse}
    if c["train"]:
        dx, dw, dbias = backward(*args, lse, s["dloss"], **more)
        out.update(dx=dx, dw=dw)
        if dbias is not None:
            out["dbias"] = dbias
    return out


def run(state):
    c = state["case"]
    if own:
        return _with_library(state, c)
    return _xent(state, c) if c["op"] == "xent" else _distill(state, c)


def work(case):
    M, V, K, n = case["M"], case["V"], case["K"], _rows(case)
    products = 3 if case["train"] else 1   # the logits; and the two gradients
    size = 2.0 * n * K + 2.0 * V * K + 8.0 * M   # x (rows with a target), w; loss and log-partition
    size += 8.0 * M if case["op"] == "xent" else 12.0 * M * case["k"]
    size += 4.0 * V if case["bias"] else 0.0
    if case["train"]:
        size += 2.0 * M * K + 2.0 * V * K + 4.0 * M + (4.0 * V if case["bias"] else 0.0)
    return {"bytes": size, "flops": 2.0 * products * n * V * K}


def exact(case, seed):
    """The definition in 64 bits, a block of rows with targets at a time."""
    s = prepare(case, seed)
    M, V, K = case["M"], case["V"], case["K"]
    T, f64 = case["temp"], torch.float64
    w = s["w"].double()
    bias = np.zeros(V) if s["bias"] is None else s["bias"].double().cpu().numpy()
    bias = torch.from_numpy(bias).to(DEV)
    targets = s["labels"][:, None] if case["op"] == "xent" else s["ids"]
    rows = (targets >= 0).any(1).nonzero()[:, 0]
    loss, lse = torch.zeros(M, dtype=f64, device=DEV), torch.zeros(M, dtype=f64, device=DEV)
    dx, dw = torch.zeros((M, K), dtype=f64, device=DEV), torch.zeros((V, K), dtype=f64, device=DEV)
    dbias = torch.zeros(V, dtype=f64, device=DEV)
    for r in torch.split(rows, max(1, (1 << 27) // V)):
        x = s["x"][r].double()
        a = case["scale"] * (x @ w.T) + bias
        z, slope = a, None
        if case["cap"] > 0:
            th = torch.tanh(a / case["cap"])
            z, slope = case["cap"] * th, 1 - th * th
        logq = torch.log_softmax(z / T, 1)
        lse[r] = torch.logsumexp(z / T, 1)
        # the target distribution, dense
        p = torch.zeros_like(z)
        if case["op"] == "xent":
            p += case["smooth"] / V
            p[torch.arange(len(r), device=DEV), targets[r, 0]] += 1 - case["smooth"]
            loss[r] = -(p * logq).sum(1) + case["zloss"] * lse[r] ** 2
            grad = logq.exp() * (1 + 2 * case["zloss"] * lse[r][:, None]) - p
        else:
            t = (s["teacher"][r].double() / T).masked_fill(targets[r] < 0, -math.inf)
            norm = s["teacher_lse"][r].double() if case["tlse"] else torch.logsumexp(t, 1)
            pj = torch.exp(t - norm[:, None])
            p.scatter_add_(1, targets[r].clamp(min=0), pj)
            loss[r] = T * T * (torch.special.xlogy(pj, pj).sum(1) - (p * logq).sum(1))
            grad = T * (logq.exp() * pj.sum(1, keepdim=True) - p)
        if case["train"]:
            grad *= s["dloss"][r].double()[:, None]
            if slope is not None:
                grad *= slope
            dx[r] = case["scale"] * (grad @ w)
            dw += case["scale"] * (grad.T @ x)
            dbias += grad.sum(0)
    out = {"loss": loss, "lse": lse}
    if case["train"]:
        out.update(dx=dx, dw=dw)
        if case["bias"]:
            out["dbias"] = dbias
    return out
