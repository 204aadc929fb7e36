"""The 64-bit vocabulary-loss oracle against torch's own definitions, its
gradients against central differences, and what a left-out row means."""
import math

import pytest
import torch

from oracle import loss as oracle

F64 = torch.float64


def make(seed, M, V, K):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g, dtype=F64)
    w = torch.randn(V, K, generator=g, dtype=F64) * 0.5
    b = torch.randn(V, generator=g, dtype=F64)
    return g, x, w, b


def test_cross_entropy_is_torchs():
    g, x, w, b = make(1, 13, 40, 9)
    y = torch.randint(0, 40, (13,), generator=g)
    y[3] = -100
    out = oracle.xent(x, w, y, b, scale=0.7, smoothing=0.1)
    ref = torch.nn.functional.cross_entropy(0.7 * x @ w.t() + b, y, reduction="none", label_smoothing=0.1)
    assert torch.allclose(out["loss"], ref, atol=1e-12)
    assert out["loss"][3] == 0 and out["lse"][3] == 0


def test_distillation_over_the_whole_vocabulary_is_kl():
    g, x, w, b = make(2, 7, 12, 5)
    t = torch.randn(7, 12, generator=g, dtype=F64) * 3
    ids = torch.stack([torch.randperm(12, generator=g) for _ in range(7)])
    T = 2.0
    out = oracle.distill(x, w, ids, t.gather(1, ids), b, temperature=T)
    lp, lq = torch.log_softmax(t / T, 1), torch.log_softmax((x @ w.t() + b) / T, 1)
    assert torch.allclose(out["loss"], T * T * (lp.exp() * (lp - lq)).sum(1), atol=1e-12)


def test_a_target_named_twice_counts_twice():
    _, x, w, b = make(3, 1, 6, 4)
    ids = torch.tensor([[2, 2, 5]])
    t = torch.tensor([[1.0, 0.5, -1.0]], dtype=F64)
    p = torch.softmax(t, 1)
    out = oracle.distill(x, w, ids, t, b)
    lq = torch.log_softmax(x @ w.t() + b, 1)[0, ids[0]]
    assert torch.allclose(out["loss"], (p * (torch.log(p) - lq)).sum(1), atol=1e-12)


def test_rows_left_out():
    _, x, w, b = make(4, 4, 6, 4)
    x[1] = math.nan
    y = torch.tensor([0, -100, 6, 5])
    out = oracle.xent(x, w, y, b, dloss=torch.ones(4, dtype=F64))
    assert out["loss"][1] == 0 and out["loss"][2] == 0
    assert all(torch.isfinite(out[k]).all() for k in ("loss", "lse", "dx", "dw", "dbias"))
    assert (out["dx"][1:3] == 0).all()


@pytest.mark.parametrize("kind", ["xent", "xent_all", "distill", "distill_lse"])
def test_gradients_against_differences(kind):
    g, x, w, b = make(5, 6, 11, 4)
    dl = torch.rand(6, generator=g, dtype=F64) + 0.5
    if kind.startswith("xent"):
        y = torch.randint(0, 11, (6,), generator=g)
        y[2] = -1
        more = dict(scale=0.8, softcap=3.0, smoothing=0.2, z_loss=0.05) if kind == "xent_all" else {}
        f = lambda x, w, b, **k: oracle.xent(x, w, y, b, **more, **k)  # noqa: E731
    else:
        ids = torch.randint(-2, 12, (6, 3), generator=g)
        t = torch.randn(6, 3, generator=g, dtype=F64)
        tl = torch.logsumexp(t / 1.5, 1) + 0.3 if kind == "distill_lse" else None
        f = lambda x, w, b, **k: oracle.distill(x, w, ids, t, b, temperature=1.5, softcap=4.0,  # noqa: E731
                                                teacher_lse=tl, **k)
    out = f(x, w, b, dloss=dl)
    h = 1e-5
    for name, v in (("dx", x), ("dw", w), ("dbias", b)):
        num = torch.zeros_like(v)
        for i in range(v.numel()):
            keep = v.view(-1)[i].item()
            v.view(-1)[i] = keep + h
            up = (f(x, w, b)["loss"] * dl).sum()
            v.view(-1)[i] = keep - h
            dn = (f(x, w, b)["loss"] * dl).sum()
            v.view(-1)[i] = keep
            num.view(-1)[i] = (up - dn) / (2 * h)
        # second-order differences: h^2 of third derivatives of order one, and
        # 1e-16 / h of rounding
        assert torch.allclose(out[name], num, atol=1e-8), name
