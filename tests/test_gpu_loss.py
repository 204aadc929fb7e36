"""GPU parity of the vocabulary losses (linear_xent, linear_distill and their
gradients) with the 64-bit oracle on the same bf16 inputs.  Tolerances are
oracle.loss.bounds: errors followed through the formulas, element by element.
"""
import math

import pytest
import torch

from oracle import loss as oracle

pytestmark = pytest.mark.gpu

BF, F64 = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def mkp(gpu):
    import dynamic_shape_gemm_amd as m
    return m


def inputs(seed, M, V, K, *, pad_x=0, pad_w=0, shift=0, std=0.2, sharp=4.0, bias=False, k=0, keep=1.0):
    """bf16 x and w in rows of K + pad elements starting `shift` elements into
    their buffers, and targets; some rows without any."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rows(n, pad, s):
        buf = torch.full((n * (K + pad) + shift + 8,), float("nan"), device="cuda", dtype=BF)
        v = buf[shift:shift + n * (K + pad)].view(n, K + pad)[:, :K]
        v.copy_(torch.randn(n, K, generator=g, device="cuda") * s)
        return v

    t = {"x": rows(M, pad_x, 1.0), "w": rows(V, pad_w, std)}
    on = torch.rand(M, generator=g, device="cuda") < keep
    if keep < 1.0 and M > 1:
        on[0], on[M - 1] = False, True
    top = torch.randint(0, V, (M,), generator=g, device="cuda")
    t["x"].add_((sharp * torch.rand(M, 1, generator=g, device="cuda") * torch.nn.functional.normalize(
        t["w"][top].float(), dim=1)).to(BF))
    if k:
        ids = torch.randint(0, V, (M, k), generator=g, device="cuda")
        ids[torch.rand(M, k, generator=g, device="cuda") < 0.1] = -1
        ids[~on] = -1
        t["ids"], t["teacher"] = ids, 2.0 * torch.randn(M, k, generator=g, device="cuda")
    else:
        t["labels"] = torch.where(on, top, torch.full_like(top, -100))
    t["bias"] = torch.randn(V, generator=g, device="cuda") if bias else None
    t["dloss"] = torch.rand(M, generator=g, device="cuda") * 2 - 0.5
    return t


def within(name, got, ref, tol, what):
    got = got.to(F64)
    assert got.shape == ref.shape, (what, name)
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    err = torch.where(same, torch.zeros_like(ref), (got - ref).abs())
    bad = ~(err <= tol)
    if bad.any():
        i = int(torch.nan_to_num(err / tol, nan=math.inf).argmax())
        raise AssertionError(f"{what} {name}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: "
                             f"{got.reshape(-1)[i].item()} for {ref.reshape(-1)[i].item()}, "
                             f"{err.reshape(-1)[i].item():.3e} > {torch.broadcast_to(tol, ref.shape).reshape(-1)[i].item():.3e}")


def check(mkp, t, what, *, grad=True, f32=False, **opt):
    """Forward and backward of one set of inputs against the oracle."""
    print(f"[case] {what} x={tuple(t['x'].shape)} w={tuple(t['w'].shape)} {opt}", flush=True)
    d = {n: (v.to(F64) if v is not None and v.is_floating_point() else v) for n, v in t.items()}
    tl = opt.pop("teacher_lse", None)
    dt = torch.float32 if f32 else BF
    if "labels" in t:
        loss, lse = mkp.linear_xent(t["x"], t["w"], t["labels"], t["bias"], **opt)
        if grad:
            dx, dw, db = mkp.linear_xent_backward(t["x"], t["w"], t["labels"], lse, t["dloss"], t["bias"],
                                                  need_dbias=True, grad_dtype=dt, **opt)
        ref = oracle.xent(d["x"], d["w"], d["labels"], d["bias"], dloss=d["dloss"] if grad else None, **opt)
        fin = ref["lse"][torch.isfinite(ref["lse"])]
        most = float(fin.abs().max()) if fin.numel() else 0.0
        more = {"weight": 1.0 + 2.0 * abs(opt.get("z_loss", 0.0)) * most,
                "terms": abs(opt.get("z_loss", 0.0)) * most * most + 16.0 * most}
        T = 1.0
    else:
        loss, lse = mkp.linear_distill(t["x"], t["w"], t["ids"], t["teacher"], t["bias"], teacher_lse=tl, **opt)
        if grad:
            dx, dw, db = mkp.linear_distill_backward(t["x"], t["w"], t["ids"], t["teacher"], lse, t["dloss"], t["bias"],
                                                     teacher_lse=tl, need_dbias=True, grad_dtype=dt, **opt)
        ref = oracle.distill(d["x"], d["w"], d["ids"], d["teacher"], d["bias"], dloss=d["dloss"] if grad else None,
                             teacher_lse=None if tl is None else tl.to(F64), **opt)
        more = {"weight": ref["weight"], "terms": ref["terms"] + ref["weight"] * 16.0}
        T = opt.get("temperature", 1.0)
    torch.cuda.synchronize()
    tol = oracle.bounds(ref, d["x"], d["w"], d["bias"], opt.get("scale", 1.0), opt.get("softcap", 0.0), T, **more)
    within("lse", lse, ref["lse"], tol["lse"], what)
    within("loss", loss, ref["loss"], tol["loss"], what)
    if grad:
        s = "32" if f32 else ""
        within("dbias", db, ref["dbias"], tol["dbias"], what)
        within("dx", dx, ref["dx"], tol["dx" + s], what)
        within("dw", dw, ref["dw"], tol["dw" + s], what)
        return loss, lse, dx, dw, db
    return loss, lse


SIZES = [(1, 1, 1), (1, 2, 8), (2, 63, 64), (3, 65, 72), (17, 256, 65), (64, 257, 128), (65, 300, 192), (129, 1000, 200),
         (256, 513, 64), (300, 129, 320), (513, 700, 264)]


@pytest.mark.parametrize("M,V,K", SIZES)
def test_xent(mkp, M, V, K):
    check(mkp, inputs(M + V, M, V, K, keep=0.8), "xent")


@pytest.mark.parametrize("M,V,K", SIZES)
def test_distill(mkp, M, V, K):
    check(mkp, inputs(M + V, M, V, K, keep=0.8, k=min(V, 5)), "distill", temperature=2.0)


@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 64, 65])
@pytest.mark.parametrize("V,K", [(3, 64), (255, 256), (1000, 320), (20000, 192), (33000, 512)])
def test_few_rows(mkp, M, V, K):
    """The forms for few rows: blocks of the vocabulary that end inside a
    workgroup's run, K steps that end inside a stage, workgroups without any."""
    check(mkp, inputs(M + V, M, V, K, keep=0.8), "few", grad=False)
    check(mkp, inputs(M + V, M, V, K, bias=True), "few", grad=False, smoothing=0.1, softcap=4.0, scale=0.8)
    for k in (2, 70):
        check(mkp, inputs(M + V, M, V, K, keep=0.8, k=k), "few", grad=False, temperature=2.0)


@pytest.mark.parametrize("M", [127, 128, 129, 200, 255, 256, 257, 384, 385, 513, 640, 641])
@pytest.mark.parametrize("V,K", [(700, 192), (20000, 128), (300, 776)])
def test_where_the_tiles_change(mkp, M, V, K):
    """Either side of the rows where the tile and the forward's gather change."""
    check(mkp, inputs(M + V, M, V, K, keep=0.8, bias=True), "tiles", smoothing=0.1)
    check(mkp, inputs(M + V, M, V, K, keep=0.8, k=9), "tiles", temperature=1.5)


@pytest.mark.parametrize("opt", [dict(scale=0.5), dict(scale=-1.5), dict(softcap=5.0), dict(smoothing=0.1),
                                 dict(smoothing=1.0), dict(z_loss=1e-2), dict(scale=1.3, softcap=2.0, smoothing=0.3,
                                                                             z_loss=1e-3)], ids=str)
@pytest.mark.parametrize("M", [50, 290])
def test_xent_options(mkp, opt, M):
    check(mkp, inputs(9, M, 333, 136, keep=0.7, bias=True), "xent options", **opt)


@pytest.mark.parametrize("k", [1, 4, 33, 200, 1024])
@pytest.mark.parametrize("own_lse", [False, True])
def test_distill_targets(mkp, k, own_lse):
    """From one target to the most, ids drawn with repetition (so named twice
    or more), at a temperature, with a bias and a cap."""
    for M in (40, 270):
        t = inputs(k, M, 600, 72, keep=0.8, bias=True, k=k)
        tl = None
        if own_lse:
            there = t["ids"] >= 0
            tl = torch.where(there, t["teacher"] / 1.5, torch.full_like(t["teacher"], -1e30)).logsumexp(1) + 0.25
        check(mkp, t, f"distill k={k}", temperature=1.5, softcap=6.0, scale=0.9, teacher_lse=tl)


@pytest.mark.parametrize("pad_x,pad_w,shift", [(0, 8, 0), (5, 0, 0), (0, 3, 0), (8, 8, 1), (1, 1, 3)])
@pytest.mark.parametrize("M", [1, 33, 280])
def test_strides_and_alignment(mkp, pad_x, pad_w, shift, M):
    check(mkp, inputs(3, M, 321, 120, pad_x=pad_x, pad_w=pad_w, shift=shift, keep=0.9), "strides")


@pytest.mark.parametrize("M", [30, 300])
def test_float32_gradients(mkp, M):
    check(mkp, inputs(5, M, 260, 96, keep=0.9), "fp32 gradients", f32=True)
    check(mkp, inputs(6, M, 260, 97, keep=0.9, k=3), "fp32 gradients", f32=True)


def test_teacher_strides(mkp):
    """ids and teacher as columns of wider arrays."""
    t = inputs(8, 40, 200, 64, k=6)
    wide = torch.full((40, 11), -7, device="cuda", dtype=torch.int64)
    wide[:, 2:8] = t["ids"]
    tw = torch.full((40, 9), float("nan"), device="cuda")
    tw[:, 1:7] = t["teacher"]
    a = check(mkp, t, "narrow")
    t["ids"], t["teacher"] = wide[:, 2:8], tw[:, 1:7]
    b = check(mkp, t, "wide")
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("M", [40, 300])
def test_no_row_has_a_target(mkp, M):
    t = inputs(11, M, 90, 64, bias=True)
    t["labels"][:] = -100
    t["labels"][0], t["labels"][1] = 90, 1 << 40   # beyond the vocabulary
    t["x"][:] = float("nan")
    loss, lse, dx, dw, db = check(mkp, t, "no labels")
    for v in (loss, lse, dx, dw, db):
        assert (v == 0).all()


@pytest.mark.parametrize("M", [24, 301])
def test_left_out_rows_may_hold_anything(mkp, M):
    """NaN and infinity in rows without a target, in their dloss, lse and
    teacher logits, reach nothing."""
    t = inputs(12, M, 150, 80, keep=0.6)
    dead = t["labels"] < 0
    clean = check(mkp, t, "clean")
    t["x"][dead] = float("nan")
    t["x"][0] = float("inf")
    t["dloss"][dead] = float("nan")
    dirty = check(mkp, t, "dirty")
    assert all(torch.equal(p, q) for p, q in zip(clean, dirty))
    t = inputs(13, M, 150, 80, keep=0.6, k=4)
    dead = (t["ids"] < 0).all(1)
    t["teacher"] = torch.where(t["ids"] < 0, torch.full_like(t["teacher"], -math.inf), t["teacher"])
    clean = check(mkp, t, "clean")
    t["x"][dead] = float("nan")
    t["dloss"][dead] = float("inf")
    t["teacher"] = torch.where(t["ids"] < 0, torch.full_like(t["teacher"], float("nan")), t["teacher"])
    dirty = check(mkp, t, "dirty")
    assert all(torch.equal(p, q) for p, q in zip(clean, dirty))


@pytest.mark.parametrize("M", [24, 301])
def test_masked_vocabulary(mkp, M):
    """A bias of -inf, and of the type's lowest value, takes entries out; a
    label that is taken out has an infinite loss, and so has every label where
    all entries are, with no NaN in any gradient."""
    for low in (-math.inf, torch.finfo(torch.float32).min):
        t = inputs(14, M, 400, 64, bias=True)
        t["bias"][50:390] = low
        t["labels"] = torch.where(t["labels"] % 2 == 0, t["labels"] % 50, 390 + t["labels"] % 10)
        check(mkp, t, "masked")
        check(mkp, t, "masked", z_loss=1e-3, scale=0.7)
        t["labels"][3] = 100
        loss, _ = mkp.linear_xent(t["x"], t["w"], t["labels"], t["bias"])
        assert torch.isposinf(loss[3]) and torch.isfinite(loss[:3]).all() and torch.isfinite(loss[4:]).all()
        t["bias"][:] = low
        loss, lse = mkp.linear_xent(t["x"], t["w"], t["labels"], t["bias"])
        assert torch.isposinf(loss).all() and torch.isneginf(lse).all()
        dx, dw, db = mkp.linear_xent_backward(t["x"], t["w"], t["labels"], lse, t["dloss"], t["bias"])
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()
        _, lse = mkp.linear_xent(t["x"], t["w"], t["labels"], t["bias"], z_loss=1e-3)
        again = mkp.linear_xent_backward(t["x"], t["w"], t["labels"], lse, t["dloss"], t["bias"], z_loss=1e-3)
        assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


@pytest.mark.parametrize("M", [24, 301])
def test_teacher_of_lowest_values(mkp, M):
    """Teacher logits of the type's lowest value among others have no weight;
    rows of nothing else (finite over T) are uniform."""
    t = inputs(17, M, 120, 64, k=4)
    t["ids"] = torch.arange(4, device="cuda").expand(M, 4) + 7 * (torch.arange(M, device="cuda")[:, None] % 5)
    low = torch.finfo(torch.float32).min
    t["teacher"][:, 2] = low
    t["teacher"][5] = low
    check(mkp, t, "lowest", temperature=2.0)
    t["teacher"][5] = 0.0
    check(mkp, t, "lowest over T is -inf", temperature=0.5)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_largest_scale_over_a_temperature(mkp, M):
    """scale / T past the largest binary32: logits of 0 stay 0."""
    t = inputs(14, M, 100, 64, k=2)
    x = torch.zeros_like(t["x"])
    loss, lse = mkp.linear_distill(x, t["w"], t["ids"], t["teacher"], scale=3e38, temperature=0.5)
    # a sum of 100 exponentials of 0, its logarithm to 1 ulp of log2(100) = 6.6 and of ln 2 times that;
    # a row whose ids are both -1 is left out, its lse 0
    want = torch.where((t["ids"] >= 0).any(1), math.log(100), 0.0)
    assert (lse - want).abs().max() <= 4 * 2.0 ** -21
    assert torch.isfinite(loss).all()


def test_a_nan_row_stays_its_own(mkp):
    """A row with a target and NaN features: its loss, its dx row and dw are
    NaN, no other row's."""
    for M in (40, 300):
        t = inputs(15, M, 100, 64)
        t["x"][7] = float("nan")
        loss, lse = mkp.linear_xent(t["x"], t["w"], t["labels"])
        dx, _, _ = mkp.linear_xent_backward(t["x"], t["w"], t["labels"], lse, t["dloss"])
        nan = torch.isnan(loss)
        assert nan[7] and nan.sum() == 1
        rows = torch.isnan(dx).any(1)
        assert rows[7] and rows.sum() == 1


@pytest.mark.parametrize("M", [0, 1, 40])
def test_only_the_gradients_asked_for(mkp, M):
    t = inputs(16, max(M, 1), 130, 72, bias=True)
    t = {n: (v[:M] if n in ("x", "labels", "dloss") else v) for n, v in t.items()}
    loss, lse = mkp.linear_xent(t["x"], t["w"], t["labels"], t["bias"])
    assert loss.shape == (M,) and lse.shape == (M,)
    args = (t["x"], t["w"], t["labels"], lse, t["dloss"], t["bias"])
    full = mkp.linear_xent_backward(*args)
    if M == 0:
        assert (full[1] == 0).all() and (full[2] == 0).all() and full[0].shape == (0, 72)
    for need in range(8):
        part = mkp.linear_xent_backward(*args, need_dx=bool(need & 1), need_dw=bool(need & 2),
                                        need_dbias=bool(need & 4))
        for i in range(3):
            if need >> i & 1:
                assert torch.equal(part[i], full[i])
            else:
                assert part[i] is None


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_several_pieces_of_the_vocabulary(mkp, op):
    """Enough rows and a wide enough vocabulary that the gradient takes more
    than one piece and dX more than one tile of rows."""
    t = inputs(21, 4200, 70000, 64, bias=True, k=6 if op == "distill" else 0, keep=0.9)
    ws1 = mkp.mkp_linear_loss_workspace(4200, 70000, 64, 0, t["w"], 64, True)
    assert ws1 < 2 * 4200 * 70000   # less than the whole gradient by the logits
    check(mkp, t, op + " pieces", **({"temperature": 2.0} if op == "distill" else {"smoothing": 0.05}))


@pytest.mark.parametrize("f32", [False, True])
def test_gradients_written_at_once(mkp, f32):
    """Enough rows and features that dX is one split, written by the product
    itself: rows left out between live ones, features that end inside a tile."""
    t = inputs(23, 3000, 300, 4424, keep=0.7, std=0.02)
    check(mkp, t, "dX at once", f32=f32)
    t = inputs(24, 2900, 270, 4101, keep=0.7, std=0.02, k=3)
    check(mkp, t, "dX at once", f32=f32)


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_many_rows(mkp, op):
    """More rows than the gather counts by itself."""
    check(mkp, inputs(22, 16600, 130, 64, bias=True, k=3 if op == "distill" else 0, keep=0.4), op + " many rows")


def past_32_bits(mkp, what, t, rows, cols):
    """A call on the whole of t against the oracle on those of its rows and
    vocabulary entries that count (the others have dloss 0, bias -inf)."""
    print(f"[case] {what} x={tuple(t['x'].shape)} w={tuple(t['w'].shape)}", flush=True)
    loss, lse = mkp.linear_xent(t["x"], t["w"], t["labels"], t["bias"])
    dx, dw, db = mkp.linear_xent_backward(t["x"], t["w"], t["labels"], lse, t["dloss"], t["bias"])
    x, w, bias, dloss = (v.to(F64) for v in (t["x"][rows], t["w"][cols], t["bias"][cols], t["dloss"][rows]))
    place = torch.full((len(t["bias"]),), -1, device="cuda")
    place[cols] = torch.arange(len(cols), device="cuda")
    ref = oracle.xent(x, w, place[t["labels"][rows]], bias, dloss=dloss)
    tol = oracle.bounds(ref, x, w, bias, terms=16.0 * float(ref["lse"].abs().max()))
    for name, got in (("lse", lse[rows]), ("loss", loss[rows]), ("dx", dx[rows]), ("dw", dw[cols]), ("dbias", db[cols])):
        within(name, got, ref[name], tol[name], what)
    # the rest is 0: as many entries that are not as among those
    assert torch.count_nonzero(dx) == torch.count_nonzero(dx[rows])
    assert torch.count_nonzero(dw) == torch.count_nonzero(dw[cols])
    assert torch.count_nonzero(db) == torch.count_nonzero(db[cols])


@pytest.mark.parametrize("M", [20, 300])
def test_a_weight_of_more_than_4_gib(mkp, M):
    V, K, n = (1 << 20) + 5, 2112, 300
    t = inputs(26, M, n, K, bias=True)
    few = t["w"]
    t["w"] = torch.randn(V, K, device="cuda", dtype=BF)
    cols = torch.cat([torch.arange(100, device="cuda"), torch.arange(V - n + 100, V, device="cuda")])
    t["w"][cols] = few
    bias = torch.full((V,), -math.inf, device="cuda")
    bias[cols] = t["bias"]
    t["bias"], t["labels"] = bias, cols[t["labels"]]
    past_32_bits(mkp, "long weight", t, torch.arange(M, device="cuda"), cols)


def test_rows_of_more_than_4_gib(mkp):
    M, V, K, n = (1 << 20) + 5, 300, 2112, 200
    t = inputs(27, n, V, K, bias=True)
    few = {name: t[name] for name in ("x", "labels", "dloss")}
    rows = torch.cat([torch.arange(70, device="cuda"), torch.arange(M - n + 70, M, device="cuda")])
    t["x"] = torch.randn(M, K, device="cuda", dtype=BF)
    t["labels"] = torch.randint(0, V, (M,), device="cuda")
    t["dloss"] = torch.zeros(M, device="cuda")
    for name, v in few.items():
        t[name][rows] = v
    past_32_bits(mkp, "many long rows", t, rows, torch.arange(V, device="cuda"))


@pytest.mark.parametrize("grad_dtype", [BF, torch.float32])
def test_writes_stay_inside(mkp, grad_dtype):
    """Raw entry points with outputs inside larger buffers: what lies between
    and behind the rows is left as it was."""
    M, V, K = 70, 130, 72
    t = inputs(31, M, V, K, keep=0.8, bias=True)
    x, w = t["x"].contiguous(), t["w"].contiguous()
    for lddx, lddw, off in ((K, K, 0), (K + 5, K + 3, 1), (K + 8, K + 16, 0)):
        dxb = torch.full((M * lddx + off + 64,), float("nan"), device="cuda", dtype=grad_dtype)
        dwb = torch.full((V * lddw + off + 64,), float("nan"), device="cuda", dtype=grad_dtype)
        dbb = torch.full((V + 64,), float("nan"), device="cuda")
        out = torch.full((2, M + 64), float("nan"), device="cuda")
        nf, nb = (mkp.mkp_linear_loss_workspace(M, V, K, 0, w, K, b) for b in (0, 1))
        ws = torch.full((max(nf, nb) + 256,), 255, device="cuda", dtype=torch.uint8)
        es = dxb.element_size()
        mkp.mkp_linear_xent(M, V, K, x, K, w, K, t["bias"], t["labels"], 1.0, 0.0, 0.0, 0.0, out[0], out[1], ws, nf)
        mkp.mkp_linear_xent_backward(M, V, K, x, K, w, K, t["bias"], t["labels"], 1.0, 0.0, 0.0, 0.0, out[1], t["dloss"],
                                     dxb.data_ptr() + es * off, lddx, dwb.data_ptr() + es * off, lddw, dbb,
                                     mkp.MKP_F32 if grad_dtype == torch.float32 else mkp.MKP_BF16, ws, nb)
        torch.cuda.synchronize()
        ref = mkp.linear_xent_backward(x, w, t["labels"], out[1, :M].clone(), t["dloss"], t["bias"],
                                       grad_dtype=grad_dtype)
        for buf, ld, rows, want in ((dxb, lddx, M, ref[0]), (dwb, lddw, V, ref[1])):
            body = buf[off:off + rows * ld].view(rows, ld)
            assert torch.equal(body[:, :K], want)
            assert torch.isnan(body[:, K:]).all() and torch.isnan(buf[:off]).all() and torch.isnan(buf[off + rows * ld:]).all()
        assert torch.equal(dbb[:V], ref[2]) and torch.isnan(dbb[V:]).all()
        assert torch.isfinite(out[:, :M]).all() and torch.isnan(out[:, M:]).all()
        assert (ws[max(nf, nb):] == 255).all()


@pytest.mark.parametrize("M", [3, 600])
def test_same_call_same_bits(mkp, M):
    t = inputs(41, M, 1500, 136, keep=0.8, bias=True)
    run = lambda: (lambda f: f + mkp.linear_xent_backward(t["x"], t["w"], t["labels"], f[1], t["dloss"], t["bias"]))(  # noqa: E731
        mkp.linear_xent(t["x"], t["w"], t["labels"], t["bias"]))
    a, b = run(), run()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_streams(mkp):
    """Two streams with calls of different sizes in flight, from torch's
    current stream and from the stream argument."""
    ts = [inputs(50 + i, 40 + 260 * i, 900, 128, keep=0.8) for i in range(2)]
    ref = [mkp.linear_xent(t["x"], t["w"], t["labels"]) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(3):
        got = []
        for t, s in zip(ts, streams):
            s.wait_stream(torch.cuda.current_stream())
            if rep == 0:
                with torch.cuda.stream(s):
                    f = mkp.linear_xent(t["x"], t["w"], t["labels"])
                    got.append(f + mkp.linear_xent_backward(t["x"], t["w"], t["labels"], f[1], t["dloss"]))
            else:
                arg = s if rep == 1 else s.cuda_stream
                f = mkp.linear_xent(t["x"], t["w"], t["labels"], stream=arg)
                got.append(f + mkp.linear_xent_backward(t["x"], t["w"], t["labels"], f[1], t["dloss"], stream=arg))
        torch.cuda.synchronize()
        for g, r, t in zip(got, ref, ts):
            assert torch.equal(g[0], r[0]) and torch.equal(g[1], r[1])
            again = mkp.linear_xent_backward(t["x"], t["w"], t["labels"], r[1], t["dloss"])
            assert torch.equal(g[2], again[0]) and torch.equal(g[3], again[1])


def test_inputs_freed_while_their_stream_runs(mkp):
    """With the stream argument the inputs may be dropped as soon as the call
    returns: their memory is not handed out again before the call is done."""
    side = torch.cuda.Stream()
    t = inputs(55, 700, 20000, 256, keep=0.9)
    ref = mkp.linear_xent(t["x"], t["w"], t["labels"])[0].clone()
    torch.cuda.synchronize()
    for _ in range(5):
        x, w, y = t["x"].clone(), t["w"].clone(), t["labels"].clone()
        side.wait_stream(torch.cuda.current_stream())
        loss, _ = mkp.linear_xent(x, w, y, stream=side)
        shapes = (x.shape, w.shape)
        del x, w, y
        junk = [torch.full(s, float("nan"), device="cuda", dtype=BF) for s in shapes for _ in range(2)]
        torch.cuda.synchronize()
        assert torch.equal(loss, ref)
        del junk


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_captured_into_graphs(mkp, op):
    """Two graphs of forward and backward, replayed by turns with new inputs
    and with the program's own calls between, equal the eager results."""
    k = 5 if op == "distill" else 0
    sizes = [(30, 700, 136), (310, 700, 136)]
    ts = [inputs(60 + i, M, V, K, keep=0.8, k=k, bias=True) for i, (M, V, K) in enumerate(sizes)]
    tgt = (lambda t: (t["ids"], t["teacher"])) if k else (lambda t: (t["labels"],))
    fwd = mkp.linear_distill if k else mkp.linear_xent
    bwd = mkp.linear_distill_backward if k else mkp.linear_xent_backward

    def step(t):
        f = fwd(t["x"], t["w"], *tgt(t), t["bias"])
        return f + bwd(t["x"], t["w"], *tgt(t), f[1], t["dloss"], t["bias"])

    graphs, outs = [], []
    for t in ts:
        step(t)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(t))
        graphs.append(g)
    for rep in range(4):
        for t in ts:
            new = inputs(70 + rep, *t["x"].shape[:1], t["w"].shape[0], t["x"].shape[1], keep=0.3 + 0.2 * rep, k=k, bias=True)
            for n in t:
                t[n].copy_(new[n])
        for g in graphs:
            g.replay()
        want = [step(t) for t in ts]
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(o, w))


def test_a_training_step_with_both_losses(mkp):
    """Labels and a teacher together, as a student is trained: the two losses'
    gradients add up to the gradient of the weighted sum."""
    t = inputs(80, 200, 500, 128, k=8)
    y = inputs(80, 200, 500, 128, keep=0.9)["labels"]
    a, b = 0.3, 0.7
    l1, s1 = mkp.linear_xent(t["x"], t["w"], y)
    l2, s2 = mkp.linear_distill(t["x"], t["w"], t["ids"], t["teacher"], temperature=2.0)
    n = int((y >= 0).sum())
    g1 = torch.full((200,), a / n, device="cuda")
    g2 = torch.full((200,), b / 200, device="cuda")
    f32 = torch.float32
    dx1, dw1, _ = mkp.linear_xent_backward(t["x"], t["w"], y, s1, g1, grad_dtype=f32)
    dx2, dw2, _ = mkp.linear_distill_backward(t["x"], t["w"], t["ids"], t["teacher"], s2, g2, temperature=2.0,
                                              grad_dtype=f32)
    d = {k: v.to(F64) if v is not None and v.is_floating_point() else v for k, v in t.items()}
    r1 = oracle.xent(d["x"], d["w"], y, dloss=g1.to(F64))
    r2 = oracle.distill(d["x"], d["w"], d["ids"], d["teacher"], temperature=2.0, dloss=g2.to(F64))
    t1 = oracle.bounds(r1, d["x"], d["w"])
    t2 = oracle.bounds(r2, d["x"], d["w"], T=2.0)
    u = 2 * oracle.U
    within("dx", dx1 + dx2, r1["dx"] + r2["dx"], t1["dx32"] + t2["dx32"] + u * (r1["dx"].abs() + r2["dx"].abs()), "both")
    within("dw", dw1 + dw2, r1["dw"] + r2["dw"], t1["dw32"] + t2["dw32"] + u * (r1["dw"].abs() + r2["dw"].abs()), "both")
    total = (g1 * l1).sum() + (g2 * l2).sum()
    ref = (g1.to(F64) * r1["loss"]).sum() + (g2.to(F64) * r2["loss"]).sum()
    assert abs(total.item() - ref.item()) <= 1e-5 * abs(ref.item()) + 1e-6


def test_gradients_against_differences(mkp):
    """The forward pass's own loss, moved along a direction of w by steps that
    bf16 holds exactly."""
    M, V, K = 60, 200, 64
    t = inputs(90, M, V, K, keep=0.9)
    w0 = (t["w"].float() * 64).round() / 64          # multiples of 1/64, below 4: bf16 keeps them and +- 1/64
    w0 = w0.clamp(-1.5, 1.5)
    g = torch.Generator(device="cuda").manual_seed(1)
    dire = torch.randint(-1, 2, (V, K), generator=g, device="cuda").float() / 64
    f = lambda w: (t["dloss"].to(F64) * mkp.linear_xent(t["x"], w.to(BF), t["labels"])[0].to(F64)).sum().item()  # noqa: E731
    up, dn = f(w0 + dire), f(w0 - dire)
    _, lse = mkp.linear_xent(t["x"], w0.to(BF), t["labels"])
    _, dw, _ = mkp.linear_xent_backward(t["x"], w0.to(BF), t["labels"], lse, t["dloss"], grad_dtype=torch.float32)
    slope = (dw.to(F64) * dire.to(F64)).sum().item()
    # the oracle's own central difference differs from its slope by the third
    # order; the library's may differ by that and the forward's and bf16's errors
    d = {k: v.to(F64) if v is not None and v.is_floating_point() else v for k, v in t.items()}
    fo = lambda w: (d["dloss"] * oracle.xent(d["x"], w, d["labels"])["loss"]).sum().item()  # noqa: E731
    ro = oracle.xent(d["x"], w0.to(F64), d["labels"], dloss=d["dloss"])
    third = abs((fo((w0 + dire).to(F64)) - fo((w0 - dire).to(F64))) / 2 - (ro["dw"] * dire.to(F64)).sum().item())
    tol = oracle.bounds(ro, d["x"], w0.to(F64))
    slack = third + (tol["dw32"] * dire.abs().to(F64)).sum().item() + (tol["loss"] * d["dloss"].abs()).sum().item()
    assert abs((up - dn) / 2 - slope) <= slack


def test_trace_names_the_launches(mkp):
    t = inputs(95, 40, 300, 64, k=3, bias=True)
    try:
        mkp.mkp_set_option("trace", 1)
        _, lse = mkp.linear_distill(t["x"], t["w"], t["ids"], t["teacher"], t["bias"])
        mkp.linear_distill_backward(t["x"], t["w"], t["ids"], t["teacher"], lse, t["dloss"], t["bias"])
        names = [r["kernel"] for r in mkp.mkp_trace_dump()]
    finally:
        mkp.mkp_set_option("trace", 0)
    assert names == ["loss_forward", "loss_finish", "loss_flags", "loss_gather", "loss_grad", "loss_products",
                     "loss_outputs"]


@pytest.mark.parametrize("M", [32, 200, 4096])
def test_capped_logits_keep_their_digits(mkp, M):
    """With one vocabulary entry lse is the logit itself, cap tanh(s / cap).
    s and s / 4 are exact (x0 + x1 / 256 of bf16 values, cap 4).  In units of
    U = 2^-24: lse = fl(ln2 fl(log2e z)) adds 1 + 1 and the constants' 0.3.
    Below |s / 4| = 1/2 tanh is a polynomial: its own 0.25, the last addition's
    0.6, what is rounded before it times s^2 / 48 < 0.1 (0.3), the product's 1.
    From 1/2 on it is 1 - 2 / (1 + e), e = e^(2 |s / 4|) good to 2.5 |s / 4| + 2:
    with the sum's and the reciprocal's 3 at most 6.5."""
    U = 2.0 ** -24
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.zeros(M, 64, device="cuda", dtype=BF)
    x[:, 0] = (torch.randint(1, 129, (M,), generator=g, device="cuda") / 16).to(BF)     # 1/16 .. 8
    x[:, 1] = (torch.randint(0, 256, (M,), generator=g, device="cuda") / 16).to(BF)     # over 256: below 1/16
    x *= torch.where(torch.rand(M, 1, generator=g, device="cuda") < 0.5, -1.0, 1.0).to(BF)
    w = torch.zeros(1, 64, device="cuda", dtype=BF)
    w[0, 0], w[0, 1] = 1.0, 2.0 ** -8
    y = torch.zeros(M, dtype=torch.int64, device="cuda")
    _, lse = mkp.linear_xent(x, w, y, softcap=4.0)
    s = x[:, 0].to(F64) + x[:, 1].to(F64) / 256
    ref = 4.0 * torch.tanh(s / 4)
    within("lse", lse, ref, torch.where(s.abs() < 2.0, 4.5, 9.0) * U * ref.abs(), "capped")


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("op", ["xent", "distill"])
def test_slope_of_saturated_logits(mkp, op, M):
    """dbias of one row is its D.  With x = 0 the logits are cap tanh(b / cap)
    of known b, up to 15 caps: their slope (1 - tanh^2, down to 4e-13) keeps
    its digits.  Relative errors: the slope's exponential (6 |b / cap| + 16) U;
    a probability's (|z|, lse < 10, cap tanh good to 2^-21) 2^-18."""
    cap, V = 2.0, 97
    t = inputs(33, M, V, 64, k=3 if op == "distill" else 0)
    t["x"][:] = 0
    t["bias"] = torch.linspace(-15.0 * cap, 15.0 * cap, V, device="cuda")
    t["dloss"][:] = 0
    t["dloss"][0] = 0.75
    if op == "xent":
        t["labels"][0] = V - 3
        _, lse = mkp.linear_xent(t["x"], t["w"], t["labels"], t["bias"], softcap=cap)
        _, _, db = mkp.linear_xent_backward(t["x"], t["w"], t["labels"], lse, t["dloss"], t["bias"], softcap=cap)
    else:
        t["ids"][0] = torch.tensor([1, V // 2, V - 3])
        _, lse = mkp.linear_distill(t["x"], t["w"], t["ids"], t["teacher"], t["bias"], softcap=cap)
        _, _, db = mkp.linear_distill_backward(t["x"], t["w"], t["ids"], t["teacher"], lse, t["dloss"], t["bias"],
                                               softcap=cap)
    b = t["bias"].to(F64)
    slope = 1.0 / torch.cosh(b / cap) ** 2
    q = torch.softmax(cap * torch.tanh(b / cap), 0)
    p = torch.zeros(V, device="cuda", dtype=F64)
    if op == "xent":
        p[V - 3] = 1.0
    else:
        p[t["ids"][0]] = torch.softmax(t["teacher"][0].to(F64), 0)
    f = 0.75 * slope
    tol = f * ((q + p) * 2.0 ** -18 + (q - p).abs() * (6.0 * b.abs() / cap + 16.0) * 2.0 ** -24)
    within("dbias", db, (q - p) * f, tol, "saturated")


@pytest.mark.parametrize("M", [20, 300])
@pytest.mark.parametrize("K", [8, 72, 200, 76])
def test_weight_rows_of_minus_infinity(mkp, M, K):
    """Rows of W that hold -inf under features above 0: their logits are -inf,
    so they are out of the sum, also where the last K step is not full."""
    t = inputs(34, M, 150, K)
    t["x"].abs_().clamp_(min=0.01)
    t["w"][::7] = -math.inf
    t["labels"] = t["labels"] // 7 * 7 + 1
    loss, lse = check(mkp, t, "-inf in w", grad=False)
    assert torch.isfinite(loss).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("V", [500, 70000])
@pytest.mark.parametrize("M", [20, 200, 1000])
def test_small_losses_at_a_large_log_partition(mkp, M, V, bias):
    """Labels ahead of the rest by margins that leave losses from ln V down to
    1e-5, every logit near 960 and exact (small multiples of 1/8).  In units of
    U = 2^-24: the label's exponential, 1, takes part in about 30 additions,
    with its own error, the logarithm's and the last products' at most 40; the
    other terms' sum is good to 80 of itself (their exponents' rounding, 30
    additions), the result to 4.  Rounding lse before the label's logit is
    taken off would cost 700."""
    U = 2.0 ** -24
    g = torch.Generator(device="cuda").manual_seed(M + V)
    y = 7
    w = torch.zeros(V, 64, device="cuda", dtype=BF)
    n = torch.randint(-24, 25, (V,), generator=g, device="cuda") / 8
    n[y] = 0
    w[:, 1] = n.to(BF)
    w[y, 2] = 1.0
    x = torch.zeros(M, 64, device="cuda", dtype=BF)
    x[:, 1] = 1.0
    margin = torch.linspace(0, math.log(V) + 14, M, device="cuda").mul(4).round().div(4)
    x[:, 2] = margin.to(BF)
    b = None
    if bias:
        b = torch.full((V,), 960.0, device="cuda")
    else:
        x[:, 0], w[:, 0] = 30.0, 32.0
    labels = torch.full((M,), y, device="cuda")
    loss, lse = mkp.linear_xent(x, w, labels, b)
    rest = torch.cat([n[:y], n[y + 1:]]).to(F64)
    ref = torch.log1p(torch.exp(torch.logsumexp(rest, 0) - x[:, 2].to(F64)))
    within("loss", loss, ref, U * (40 + 80 * -torch.expm1(-ref) + 4 * ref), "small losses")
    want = 960 + x[:, 2].to(F64) + ref
    within("lse", lse, want, U * (120 + 8 * want), "small losses")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("M,V,K", [(1, 9000, 64), (40, 20000, 128), (300, 20000, 128), (1000, 50257, 64), (700, 33000, 264)])
def test_dx_alone(mkp, M, V, K, op, f32):
    """dX without dW is cut into more splits of the vocabulary, up to what its
    workspace is sized for, on both tiles."""
    print(f"[case] dx alone {op} {M} {V} {K}", flush=True)
    t = inputs(36, M, V, K, keep=0.9, k=5 if op == "distill" else 0, std=0.1)
    d = {n: (v.to(F64) if v is not None and v.is_floating_point() else v) for n, v in t.items()}
    more = dict(need_dw=False, need_dbias=False, grad_dtype=torch.float32 if f32 else BF)
    if op == "xent":
        _, lse = mkp.linear_xent(t["x"], t["w"], t["labels"])
        dx, dw, db = mkp.linear_xent_backward(t["x"], t["w"], t["labels"], lse, t["dloss"], **more)
        ref = oracle.xent(d["x"], d["w"], d["labels"], dloss=d["dloss"])
    else:
        _, lse = mkp.linear_distill(t["x"], t["w"], t["ids"], t["teacher"])
        dx, dw, db = mkp.linear_distill_backward(t["x"], t["w"], t["ids"], t["teacher"], lse, t["dloss"], **more)
        ref = oracle.distill(d["x"], d["w"], d["ids"], d["teacher"], dloss=d["dloss"])
    assert dw is None and db is None
    within("dx", dx, ref["dx"], oracle.bounds(ref, d["x"], d["w"])["dx32" if f32 else "dx"], "dx alone")


@pytest.mark.parametrize("need", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("M,V,K,pad_w,k", [(20, 5000, 128, 0, 0), (20, 5000, 128, 0, 200), (40, 20000, 128, 0, 0),
                                           (300, 20000, 128, 0, 5), (1000, 50257, 64, 0, 0), (600, 3000, 100, 0, 3),
                                           (70, 1300, 72, 3, 7), (5000, 1300, 72, 3, 0), (4200, 70000, 64, 0, 6),
                                           (9000, 40000, 64, 0, 0)])
def test_calls_stay_inside_their_workspace(mkp, M, V, K, pad_w, k, need):
    """A workspace of exactly the bytes reported, between guards: splits of dX,
    several pieces of the vocabulary, both losses, a copied weight.  What it
    holds before (bytes of 0xA5, or of 0xFF: NaN) does not matter."""
    print(f"[case] workspace {M} {V} {K} pad {pad_w} k {k} {need}", flush=True)
    t = inputs(37, M, V, K, pad_w=pad_w, keep=0.9, k=k)
    ldw = t["w"].stride(0)
    loss, lse = torch.empty(2, M, device="cuda")
    dx, dw, db = torch.empty(M, K, device="cuda"), torch.empty(V, K, device="cuda"), torch.empty(V, device="cuda")
    out = (dx if need[0] else None, K, dw if need[1] else None, K, db, mkp.MKP_F32)
    got = []
    for fill in (0xA5, 0xFF):
        for back in (False, True):
            n = mkp.mkp_linear_loss_workspace(M, V, K, k, t["w"], ldw, back)
            buf = torch.full((n + 2048,), fill, device="cuda", dtype=torch.uint8)
            ws = buf.data_ptr() + 1024
            tgt = (t["labels"], 1.0, 0.0, 0.1, 0.0) if not k else (k, t["ids"], k, t["teacher"], k, 0, 1.0, 1.0, 0.0)
            fwd = mkp.mkp_linear_distill if k else mkp.mkp_linear_xent
            bwd = mkp.mkp_linear_distill_backward if k else mkp.mkp_linear_xent_backward
            args = (M, V, K, t["x"], K, t["w"], ldw, None) + tgt
            if back:
                bwd(*args, lse, t["dloss"], *out, ws, n)
            else:
                fwd(*args, loss, lse, ws, n)
            torch.cuda.synchronize()
            assert (buf[:1024] == fill).all() and (buf[1024 + n:] == fill).all(), back
        got.append([v.clone() for v in (loss, lse, db) + (dx,) * need[0] + (dw,) * need[1]])
        assert all(torch.isfinite(v).all() for v in got[-1])
    assert all(torch.equal(p, q) for p, q in zip(*got))


LARGE = [(513, 20000, 512), (400, 16000, 1024), (400, 16000, 1000), (700, 8000, 1021)]


@pytest.mark.parametrize("opt", [dict(), dict(smoothing=0.1, z_loss=1e-3), dict(scale=0.8, softcap=4.0)], ids=str)
@pytest.mark.parametrize("M,V,K", LARGE)
def test_xent_on_large_tiles(mkp, M, V, K, opt):
    """Extents for which 256 x 256 tiles cost less, forward and backward: whole
    and halved last rounds, halves without a live row, K steps not full."""
    check(mkp, inputs(M + K, M, V, K, keep=0.8, std=0.05, bias=bool(opt)), "large", f32=not opt, **dict(opt))


@pytest.mark.parametrize("k", [1, 9, 300])
@pytest.mark.parametrize("M,V,K", LARGE)
def test_distill_on_large_tiles(mkp, M, V, K, k):
    check(mkp, inputs(M + K + k, M, V, K, keep=0.8, std=0.05, bias=k == 9, k=k), "large", temperature=1.5,
          **({"softcap": 5.0} if k == 9 else {}))


@pytest.mark.parametrize("M,V,K", [(200, 20000, 200), (256, 33000, 1024), (129, 65000, 192)])
def test_few_rows_on_large_tiles(mkp, M, V, K):
    """Rows as they come, on 256 x 256 tiles."""
    check(mkp, inputs(M, M, V, K, keep=0.8, std=0.05), "large", grad=False)
    check(mkp, inputs(M, M, V, K, keep=0.8, std=0.05, bias=True, k=9), "large", grad=False, temperature=2.0, softcap=4.0)
    x = torch.randn(M, (K + 63) // 64 * 64, device="cuda", dtype=BF)   # K a multiple of 64: nothing is gathered
    w = torch.randn(V, x.shape[1], device="cuda", dtype=BF) * 0.05
    y = torch.randint(-20, V, (M,), device="cuda")
    check(mkp, {"x": x, "w": w, "labels": y, "bias": None}, "direct", grad=False, smoothing=0.1)
    ids = torch.randint(-2000, V, (M, 7), device="cuda")
    check(mkp, {"x": x, "w": w, "ids": ids, "teacher": torch.randn(M, 7, device="cuda"), "bias": None}, "direct", grad=False)


def test_left_out_and_masked_on_large_tiles(mkp):
    M, V, K = 400, 16000, 1024
    t = inputs(44, M, V, K, keep=0.6, std=0.05, bias=True)
    dead = t["labels"] < 0
    clean = check(mkp, t, "clean")
    t["x"][dead] = float("nan")
    t["dloss"][dead] = float("nan")
    assert all(torch.equal(p, q) for p, q in zip(clean, check(mkp, t, "dirty")))
    t["bias"][50:15000] = -math.inf
    t["labels"] = torch.where(dead, t["labels"], t["labels"] % 50)
    check(mkp, t, "masked", z_loss=1e-3)
    t["bias"][:] = torch.finfo(torch.float32).min
    loss, lse = mkp.linear_xent(t["x"], t["w"], t["labels"], t["bias"])
    assert torch.isposinf(loss[~dead]).all() and torch.isneginf(lse[~dead]).all() and (loss[dead] == 0).all()
    for v in mkp.linear_xent_backward(t["x"], t["w"], t["labels"], lse, t["dloss"], t["bias"]):
        assert torch.isfinite(v).all()
    t["labels"][:] = -1
    for v in mkp.linear_xent_backward(t["x"], t["w"], t["labels"], lse, t["dloss"], t["bias"]):
        assert (v == 0).all()


@pytest.mark.parametrize("M", [5000, 8200])
def test_many_rows_on_small_tiles(mkp, M):
    """A narrow vocabulary, for which 128 x 128 tiles cost less at any M."""
    check(mkp, inputs(45, M, 700, 136, keep=0.7, bias=True), "small", smoothing=0.05)
    check(mkp, inputs(46, M, 700, 136, keep=0.7, k=20), "small", temperature=2.0, softcap=6.0)
