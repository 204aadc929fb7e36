"""GPU parity of the 8-bit matrices (quantize_rows, dequantize_rows, linear_i8,
linear_q8_backward) with the 64-bit oracle on the same inputs.  Integers, scales
and what they are read back as have to be equal; tolerances of the others are
oracle.q8's, followed through the formulas element by element."""
import math

import pytest
import torch

from oracle import q8 as oracle

pytestmark = pytest.mark.gpu

BF, F32, F64, I8 = torch.bfloat16, torch.float32, torch.float64, torch.int8
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
NAN = float("nan")


@pytest.fixture(scope="module")
def mkp(gpu):
    import dynamic_shape_gemm_amd as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def placed(v, pad=0, shift=0):
    """v in rows of v.shape[1] + pad elements that start `shift` elements into
    their buffer, with NaN (integers: 77) around them."""
    M, K = v.shape
    fill = NAN if v.is_floating_point() else 77
    buf = torch.full((M * (K + pad) + shift + 64,), fill, device="cuda", dtype=v.dtype)
    out = buf[shift:shift + M * (K + pad)].view(M, K + pad)[:, :K]
    out.copy_(v)
    return out


def features(g, M, K, t=BF):
    x = torch.randn(M, K, generator=g, device="cuda") * torch.exp(torch.randn(K, generator=g, device="cuda"))
    return x.to(t)


def same(got, want, what):
    assert got.dtype == want.dtype and got.shape == want.shape, what
    ok = (got == want) | (torch.isnan(got) & torch.isnan(want)) if got.is_floating_point() else got == want
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.numel()} differ, first at {int((~ok).reshape(-1).nonzero()[0])}"


def within(got, ref, tol, what):
    got = got.to(F64)
    assert got.shape == ref.shape, what
    equal = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    err = torch.where(equal, torch.zeros_like(ref), (got - ref).abs())
    bad = ~(equal | (err <= tol))
    if bad.any():
        i = int(torch.nan_to_num(err / tol, nan=math.inf).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: {got.reshape(-1)[i].item()} for "
                             f"{ref.reshape(-1)[i].item()}, {err.reshape(-1)[i].item():.3e} > {tol.reshape(-1)[i].item():.3e}")


# ---- quantisation ------------------------------------------------------------

def check_store(mkp, x, group, what):
    print(f"[case] {what} {tuple(x.shape)} {x.dtype} group={group}", flush=True)
    q, s = mkp.quantize_rows(x, group=group)
    wq, ws = oracle.quantize(x, group)
    same(s, ws, what + " scale")
    same(q, wq, what + " integers")
    for t in (BF, F32):
        y = mkp.dequantize_rows(q, s, group=group, dtype=t)
        # (one product in binary32, rounded once more for bf16)
        same(y, oracle.values(q, s, group).to(F32).to(t), what + " values")
    return q, s


@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 4096), (3, 31), (5, 512), (2, 513), (7, 1024), (4, 1030), (9, 2048), (3, 2100),
                                 (2, 4097), (3, 8192), (2, 8200), (2, 16384), (2, 16400), (1, 40000), (301, 257), (1000, 8),
                                 (3, 32767), (2, 32772), (2, 65536), (3, 65543), (2, 70001)])
def test_store(mkp, M, K, t, group):
    check_store(mkp, features(gen(M + K), M, K, t), group, "store")


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 5), (8, 0), (7, 8)])
def test_store_strides(mkp, pad, shift, t, group):
    for M, K in ((5, 100), (3, 2051), (2, 5000)):
        x = placed(features(gen(K), M, K, t), pad, shift)
        q, s = check_store(mkp, x, group, "strides")
        # integers and scales in places of any alignment, their surroundings left alone
        wide = torch.full((M, K + 9), 77, dtype=I8, device="cuda")
        G = 1 if group == 0 else -(-K // group)
        sw = torch.full((M, G + 2), NAN, device="cuda")
        mkp.mkp_quantize_rows(M, K, x.data_ptr(), x.stride(0), mkp.MKP_F32 if t == F32 else mkp.MKP_BF16, group,
                              wide.data_ptr() + 5, K + 9, sw.data_ptr() + 4, G + 2)
        same(wide.view(-1)[5:].unfold(0, K, K + 9)[:M].contiguous() if M == 1 else
             torch.as_strided(wide, (M, K), (K + 9, 1), 5), q, "strided integers")
        keep = torch.as_strided(wide, (M - 1, 9), (K + 9, 1), 5 + K)
        assert (keep == 77).all() and (wide.view(-1)[:5] == 77).all()
        same(torch.as_strided(sw, (M, G), (G + 2, 1), 1).reshape(s.shape), s, "strided scales")
        out = torch.full((M, K + 3), NAN, dtype=t, device="cuda")
        mkp.mkp_dequantize_rows(M, K, wide.data_ptr() + 5, K + 9, sw.data_ptr() + 4, G + 2, group, out.data_ptr(), K + 3,
                                mkp.MKP_F32 if t == F32 else mkp.MKP_BF16)
        same(out[:, :K], mkp.dequantize_rows(q, s, group=group, dtype=t), "strided values")
        assert torch.isnan(out[:, K:]).all()


@pytest.mark.parametrize("group", [0, 32])
def test_quotients_next_to_a_half(mkp, group):
    """Scales of powers of two make ties; values one unit beside a half of a
    scale that has all 24 digits, on either side, must not be taken for ties."""
    K = 1024
    x = (torch.arange(K, device="cuda", dtype=F32) * 0.5 - 255.75).clamp(-127, 127).repeat(3, 1)
    x[:, ::32] = 127.0
    x[1] *= 2.0 ** -20
    x[2] *= 2.0 ** 90
    check_store(mkp, x, group, "ties")
    check_store(mkp, x.to(BF), group, "ties")
    for k, top in enumerate((1.0, 1.7182817, 3.3333333e-5, 6.1e30)):
        s = (torch.tensor(top, dtype=F64) / 127.0).to(F32).to(F64)
        half = ((torch.arange(K, device="cuda", dtype=F64) % 126) + 0.5) * s.cuda()
        for step in (-2, -1, 0, 1, 2):
            v = (half.to(F32).view(torch.int32) + step).view(F32)
            v[::32] = top
            check_store(mkp, v[None].repeat(2, 1), group, f"beside halves {k} {step}")


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_extremes(mkp, t, group):
    big = torch.finfo(t).max
    x = features(gen(5), 12, 700, t)
    x[0, 3], x[1, 650], x[2, 699], x[3] = NAN, math.inf, -math.inf, NAN
    x[4] = 0
    x[5] = (x[5].float() * 1e-38).to(t)
    x[6] = (x[6].float() * 1e-42).to(t)
    x[7, 100], x[8, 100] = big, -big
    x[9, :] = 2.0 ** -126 * 63
    x[10, :] = -0.0
    q, s = check_store(mkp, x, group, "extremes")
    bad = torch.isnan(s if group else s[:, None])
    assert bad[:4].any(1).all() and bad[3].all() and not bad[4:].any()


def test_past_4_gib(mkp):
    """Offsets that pass 32 bits: rows far into a wide array, two of them looked at."""
    M, K = 70000, 65600
    x = torch.empty((M, K), dtype=BF, device="cuda")
    x[:] = 1.0
    x[-1] = features(gen(1), 1, K)[0]
    x[40000] = features(gen(2), 1, K)[0]
    for group in (0, 128):
        q, s = mkp.quantize_rows(x, group=group)
        y = mkp.dequantize_rows(q, s, group=group)
        for m in (0, 40000, M - 1):
            wq, ws = oracle.quantize(x[m:m + 1], group)
            same(q[m:m + 1], wq, "far integers")
            same(s[m:m + 1], ws, "far scales")
            same(y[m:m + 1], oracle.values(wq, ws, group).to(F32).to(BF), "far values")
        del q, s, y


# ---- linear layer --------------------------------------------------------------

def layer(g, M, N, K, t=BF, bias=True):
    w, ws = oracle.quantize(torch.randn(N, K, generator=g, device="cuda") / math.sqrt(max(K, 1)))
    b = 0.5 * torch.randn(N, generator=g, device="cuda") if bias else None
    return features(g, M, K, t), w, ws, b


def check_linear(mkp, x, w, ws, b, act="none", t=F32, xs=None, what="linear", out=None):
    print(f"[case] {what} x={tuple(x.shape)} {x.dtype} w={tuple(w.shape)} act={act} out={t}", flush=True)
    y = mkp.linear_i8(x, w, ws, b, act=act, x_scale=xs, dtype=t, out=out)
    q, s = (x, xs) if xs is not None else oracle.quantize(x)
    ref, tol = oracle.linear(q, s, w, ws, b, act, t)
    within(y, ref, tol, what)
    return y


SIZES = [(1, 1, 1), (1, 2, 16), (2, 5, 130), (1, 300, 4096), (3, 64, 127), (16, 200, 128), (17, 129, 272), (33, 1000, 640),
         (64, 31, 1024), (65, 257, 2048), (100, 1024, 12544), (128, 128, 512), (129, 130, 1030), (200, 700, 768),
         (257, 513, 96), (300, 2304, 768), (512, 300, 4000)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(mkp, M, N, K):
    x, w, ws, b = layer(gen(M + N), M, N, K)
    check_linear(mkp, x, w, ws, b)
    check_linear(mkp, x.float() * 1.001, w, ws, None, "gelu", BF)
    q, s = oracle.quantize(x)
    check_linear(mkp, placed(q, (-K) % 16), w, ws, b, "silu", BF, s)


@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("N,K", [(40, 256), (4096, 1024), (1000, 4112), (20000, 192)])
def test_few_tokens(mkp, M, N, K):
    """Every number of tokens where another form may be taken, on both sides."""
    x, w, ws, b = layer(gen(M), M, N, K)
    check_linear(mkp, x, w, ws, b, "relu", F32)
    q, s = oracle.quantize(x)
    check_linear(mkp, placed(q, (-K) % 16), w, ws, None, "none", BF, s)


@pytest.mark.parametrize("M,N,K", [(32, 200, 4096), (32, 200, 4097), (31, 1024, 12544), (9, 130, 20011), (4, 600, 32768),
                                   (4, 600, 32770), (2, 33, 131071), (1, 1000, 131071)])
def test_few_tokens_of_many_features(mkp, M, N, K):
    """On both sides of where tiles are taken; the same bits wherever W lies."""
    x, w, ws, b = layer(gen(M + K), M, N, K)
    q, s = oracle.quantize(x)
    aligned = placed(w, (-K) % 16)
    for xs, a in ((None, x), (s, q), (s, placed(q, (-K) % 16))):
        y = check_linear(mkp, a, aligned, ws, b, "silu", BF, xs)
        same(check_linear(mkp, a, placed(w, 1, 3), ws, b, "silu", BF, xs), y, "an unaligned weight")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 20, 150, 4100])
def test_linear_activations(mkp, act, t, M):
    x, w, ws, b = layer(gen(7), M, 520, 200)
    check_linear(mkp, x, w, ws, 4.0 * b, act, t)


@pytest.mark.parametrize("M,N,K", [(1025, 4000, 256), (4096, 4096, 384), (3000, 6000, 130)])
def test_large_tiles(mkp, M, N, K):
    x, w, ws, b = layer(gen(M), M, N, K)
    check_linear(mkp, x, w, ws, b, "gelu_tanh", BF)
    check_linear(mkp, x, w, ws, b, "none", F32)


@pytest.mark.parametrize("M", [1, 12, 40, 300])
@pytest.mark.parametrize("pad_x,pad_w,shift", [(0, 0, 1), (1, 3, 0), (16, 16, 0), (5, 0, 16), (0, 7, 3)])
def test_linear_strides(mkp, M, pad_x, pad_w, shift):
    """Operands and outputs of any alignment; the output's surroundings stay."""
    N, K = 333, 208
    x, w, ws, b = layer(gen(M), M, N, K)
    q, s = oracle.quantize(x)
    w2 = placed(w, pad_w, shift)
    for pad_y in (0, 3, 8):
        for t in (BF, F32):
            out = torch.full((M, N + pad_y + 8), NAN, dtype=t, device="cuda")
            check_linear(mkp, placed(x, pad_x, shift), w2, ws, b, "gelu", t, out=out[:, pad_y:N + pad_y])
            assert torch.isnan(out[:, :pad_y]).all() and torch.isnan(out[:, N + pad_y:]).all()
            out.fill_(NAN)
            check_linear(mkp, placed(q, pad_x, shift), w2, ws, b, "none", t, s, out=out[:, pad_y:N + pad_y])
            assert torch.isnan(out[:, :pad_y]).all() and torch.isnan(out[:, N + pad_y:]).all()


@pytest.mark.parametrize("M", [1, 8, 40, 300, 4200])
def test_largest_sums(mkp, M):
    """-128 and 127 everywhere, at the most features whose sums fit 32 bits; what
    lies behind a row's end reaches nothing."""
    for K in (131071, 131056, 1000):
        N = 20 if M < 1000 else 4000
        if M * K > 1 << 27:
            K = 4095
        x = torch.full((M, K), -128, dtype=I8, device="cuda")
        w = torch.full((N, K), -128, dtype=I8, device="cuda")
        w[1::2] = 127
        one = torch.ones(max(M, N), device="cuda")
        check_linear(mkp, placed(x, 5), placed(w, (-K) % 16), one[:N] * 2.0 ** -20, None, "none", F32, one[:M], "largest sums")


def test_empty_sums(mkp):
    b = torch.randn(9, device="cuda")
    for M in (5, 40):
        for xs in (None, torch.ones(M, device="cuda")):
            for t in (F32, BF):
                y = mkp.linear_i8(torch.empty((M, 0), dtype=BF if xs is None else I8, device="cuda"),
                                  torch.empty((9, 0), dtype=I8, device="cuda"), torch.ones(9, device="cuda"), b, act="relu",
                                  x_scale=xs, dtype=t)
                same(y, b.clamp(min=0).to(t).repeat(M, 1), "no features")
    assert mkp.linear_i8(torch.empty((0, 16), dtype=BF, device="cuda"), torch.ones((3, 16), dtype=I8, device="cuda"),
                         torch.ones(3, device="cuda")).shape == (0, 3)
    assert mkp.linear_i8(torch.ones((4, 16), dtype=BF, device="cuda"), torch.ones((0, 16), dtype=I8, device="cuda"),
                         torch.ones(0, device="cuda")).shape == (4, 0)


@pytest.mark.parametrize("M", [3, 60, 400])
def test_rows_that_are_not_finite(mkp, M):
    """NaN and infinities in a token reach its own outputs only, all of them."""
    x, w, ws, b = layer(gen(M), M, 100, 300)
    x[0, 5], x[M // 2, 299], x[M - 1, 0] = NAN, math.inf, -math.inf
    y = check_linear(mkp, x, w, ws, b, "gelu", F32)
    bad = torch.isnan(y)
    assert bad[[0, M // 2, M - 1]].all() and int(bad.sum()) == 300
    x[:] = 0
    y = mkp.linear_i8(x, w, ws, b)
    same(y, b.repeat(M, 1), "tokens of zeros")


def test_far_weights(mkp):
    """Offsets that pass 32 bits in the weight and in the output."""
    N, K = 300000, 16400
    w = torch.randint(-127, 128, (1, K), device="cuda", dtype=torch.int32).to(I8).repeat(N, 1)
    w[N - 1] = 3
    ws = torch.full((N,), 0.01, device="cuda")
    for M in (2, 40):
        x = features(gen(M), M, K)
        q, s = oracle.quantize(x)
        y = mkp.linear_i8(x, w, ws)
        for sl in (slice(0, 70), slice(N // 2, N // 2 + 70), slice(N - 70, N)):
            ref, tol = oracle.linear(q, s, w[sl], ws[sl], None, "none", F32)
            within(y[:, sl], ref, tol, "far weights")
    del w, y
    M, N, K = 70000, 20000, 64
    x, w, ws, _ = layer(gen(3), M, N, K)
    y = mkp.linear_i8(x, w, ws)
    for sl in (slice(0, 33), slice(M - 33, M)):
        q, s = oracle.quantize(x[sl])
        ref, tol = oracle.linear(q, s, w, ws, None, "none", F32)
        within(y[sl], ref, tol, "far rows")


# ---- backward --------------------------------------------------------------------

def kept(g, M, N, K, group, t=BF):
    x, xs = oracle.quantize(features(g, M, K))
    z, zs = oracle.quantize(2.0 * torch.randn(M, N, generator=g, device="cuda"), group)
    return torch.randn(M, N, generator=g, device="cuda").to(t), x, xs, z, zs


def check_backward(mkp, dy, x, xs, z, zs, group, act, t=BF, what="backward", **need):
    print(f"[case] {what} dy={tuple(dy.shape)} {dy.dtype} x={tuple(x.shape)} group={group} act={act} {t} {need}", flush=True)
    dz, dw, db = mkp.linear_q8_backward(dy, x, xs, z, zs, z_group=group, act=act, grad_dtype=t, **need)
    ref = oracle.backward(dy, x, xs, z, zs, group, act, t)
    for name, got in (("dz", dz), ("dw", dw), ("dbias", db)):
        assert (got is None) == (need.get("need_" + name) is False)
        if got is not None:
            within(got, *ref[name], what + " " + name)
    return dz, dw, db


BACK = [(1, 1, 1), (2, 8, 16), (31, 33, 40), (32, 7, 130), (33, 64, 64), (63, 256, 9), (64, 128, 128), (65, 130, 258),
        (200, 300, 500), (333, 768, 768), (1000, 100, 36), (2049, 40, 300), (130, 2304, 768)]


@pytest.mark.parametrize("M,N,K", BACK)
def test_backward(mkp, M, N, K):
    a = kept(gen(M + N), M, N, K, 64)
    check_backward(mkp, *a, 64, "gelu")
    check_backward(mkp, *a, 64, "silu", F32)
    check_backward(mkp, *a[:3], None, None, 0, "none")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_backward_activations(mkp, act, group, t):
    check_backward(mkp, *kept(gen(3), 70, 300, 48, group, t), group, act)


@pytest.mark.parametrize("M,N,K", [(100, 4096, 2048), (700, 2900, 3000)])
def test_backward_large_tiles(mkp, M, N, K):
    a = kept(gen(M), M, N, K, 128)
    check_backward(mkp, *a, 128, "silu")
    check_backward(mkp, *a, 128, "gelu_tanh", F32)


def test_backward_of_what_is_needed(mkp):
    a = kept(gen(9), 150, 200, 96, 0, F32)
    every = check_backward(mkp, *a, 0, "gelu")
    for need in (dict(need_dw=False), dict(need_dz=False), dict(need_dbias=False), dict(need_dw=False, need_dbias=False),
                 dict(need_dz=False, need_dbias=False), dict(need_dz=False, need_dw=False)):
        got = check_backward(mkp, *a, 0, "gelu", **need)
        for g, e in zip(got, every):
            assert g is None or torch.equal(g, e)
    assert mkp.linear_q8_backward(*a[:3], need_dz=False, need_dw=False, need_dbias=False) == (None, None, None)


@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 5), (16, 16)])
@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_backward_strides(mkp, pad, shift, t):
    dy, x, xs, z, zs = kept(gen(1), 77, 203, 101, 32, t)
    ref = check_backward(mkp, dy, x, xs, z, zs, 32, "silu")
    wide = torch.full((77, zs.shape[1] + 3), NAN, device="cuda")
    wide[:, 1:-2] = zs
    got = check_backward(mkp, placed(dy, pad, shift), placed(x, pad, shift), xs, placed(z, pad, shift), wide[:, 1:-2], 32, "silu")
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
    # outputs inside wider arrays
    M, N, K = 77, 203, 101
    n = mkp.mkp_linear_q8_backward_workspace(M, N, K, True, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for gt, code in ((BF, mkp.MKP_BF16), (F32, mkp.MKP_F32)):
        dz = torch.full((M, N + 5), NAN, dtype=BF, device="cuda")
        dw = torch.full((N, K + pad + 2), NAN, dtype=gt, device="cuda")
        db = torch.full((N + 8,), NAN, device="cuda")
        mkp.mkp_linear_q8_backward(M, N, K, dy, N, mkp.MKP_F32 if t == F32 else mkp.MKP_BF16, x, x.stride(0), xs, z,
                                   z.stride(0), zs, zs.stride(0), 32, mkp.MKP_ACT_SILU, dz, N + 5, dw, K + pad + 2, code, db, ws, n)
        want = oracle.backward(dy, x, xs, z, zs, 32, "silu", gt)
        within(dz[:, :N], *want["dz"], "dz in a wider array")
        within(dw[:, :K], *want["dw"], "dw in a wider array")
        within(db[:N], *want["dbias"], "dbias")
        assert torch.isnan(dz[:, N:]).all() and torch.isnan(dw[:, K:]).all() and torch.isnan(db[N:]).all()


def test_backward_of_no_tokens(mkp):
    e = lambda *s, t=F32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    dz, dw, db = mkp.linear_q8_backward(e(0, 24, t=BF), e(0, 40, t=I8), e(0), e(0, 24, t=I8), e(0), act="gelu")
    assert dz.shape == (0, 24) and (dw == 0).all() and dw.shape == (24, 40) and (db == 0).all()
    dz, dw, db = mkp.linear_q8_backward(torch.ones(3, 24, device="cuda"), e(3, 0, t=I8), torch.ones(3, device="cuda"))
    assert dw.shape == (24, 0) and (db == 3).all() and (dz == 1).all()


def test_rows_of_nan_scale(mkp):
    """A token whose input could not be kept makes every weight gradient NaN; one
    whose pre-activation could not, those of its own channels."""
    dy, x, xs, z, zs = kept(gen(4), 90, 64, 48, 32)
    bad = zs.clone()
    bad[7, 1] = NAN
    dz, dw, db = mkp.linear_q8_backward(dy, x, xs, z, bad, z_group=32, act="gelu")
    assert torch.isnan(dz[7, 32:]).all() and int(torch.isnan(dz).sum()) == 32
    assert torch.isnan(dw[32:]).all() and not torch.isnan(dw[:32]).any() and int(torch.isnan(db).sum()) == 32
    xs[5] = NAN
    _, dw, db = mkp.linear_q8_backward(dy, x, xs, z, zs, z_group=32, act="gelu")
    assert torch.isnan(dw).all() and not torch.isnan(db).any()


# ---- together ----------------------------------------------------------------------

def test_serving_run(mkp):
    """Two layers on one quantised input, then two in a row, as a decoder's block
    runs them: for a prompt and for single tokens, the same numbers."""
    g = gen(11)
    x = features(g, 70, 512)
    (w1, s1), (w2, s2), (w3, s3) = (mkp.quantize_rows(torch.randn(n, k, generator=g, device="cuda").to(BF) / math.sqrt(k))
                                    for n, k in ((1100, 512), (1100, 512), (512, 1100)))
    q, qs = mkp.quantize_rows(x)
    gate = check_linear(mkp, q, w1, s1, None, "silu", F32, qs, "gate")
    up = check_linear(mkp, q, w2, s2, None, "none", F32, qs, "up")
    same(mkp.linear_i8(x, w2, s2), up, "quantised within the call or before it")
    h = gate * up
    y = check_linear(mkp, h, w3, s3, None, "none", BF, what="down")
    for m in (0, 33, 69):   # a token at a time
        one = x[m:m + 1]
        hm = mkp.linear_i8(one, w1, s1, act="silu") * mkp.linear_i8(one, w2, s2)
        same(mkp.linear_i8(hm, w3, s3, dtype=BF), y[m:m + 1], "a single token")


def test_training_run(mkp):
    """A layer's forward pass through the library, its input and pre-activation
    kept in 8 bits, and its whole backward pass, against autograd in 64 bits on
    the kept values."""
    g = gen(12)
    M, N, K = 260, 384, 200
    x = features(g, M, K)
    w = (torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)).to(BF)
    b = torch.randn(N, generator=g, device="cuda")
    z = mkp.linear(x, w, b)
    xq, xs = mkp.quantize_rows(x)
    zq, zs = mkp.quantize_rows(z, group=64)
    dy = torch.randn(M, N, generator=g, device="cuda")
    dz, dw, db = check_backward(mkp, dy, xq, xs, zq, zs, 64, "gelu", what="training")
    dx = mkp.gemm(dz, w)
    leaf = [t.to(F64).requires_grad_() for t in (oracle.values(xq, xs), w, b)]
    kept_z = oracle.values(zq, zs, 64)
    zz = leaf[0] @ leaf[1].t() + leaf[2]
    out = oracle.act("gelu", zz + (kept_z - zz).detach())
    out.backward(dy.to(F64))
    ref = oracle.backward(dy, xq, xs, zq, zs, 64, "gelu", BF)
    within(dw, leaf[1].grad, ref["dw"][1], "dw by autograd")
    within(db, leaf[2].grad, ref["dbias"][1], "dbias by autograd")
    terms = ref["dz"][0].abs() @ w.to(F64).abs()
    within(dx, leaf[0].grad, (2.0 ** -8 + 2 * N * 2.0 ** -24) * 1.02 * terms + ref["dz"][1] @ w.to(F64).abs(), "dx by autograd")


def calls(mkp, M=60, N=300, K=320):
    """One call of each operator on inputs of its own: (name, inputs, call)."""
    x, w, ws, b = layer(gen(M), M, N, K)
    q, s = mkp.quantize_rows(x, group=64)
    back = kept(gen(M + 1), M, N, K, 64)
    return [("quantize", [x], lambda x, **o: mkp.quantize_rows(x, group=64, **o)),
            ("dequantize", [q, s], lambda q, s, **o: (mkp.dequantize_rows(q, s, group=64, **o),)),
            ("linear", [x, w, ws, b], lambda x, w, ws, b, **o: (mkp.linear_i8(x, w, ws, b, act="gelu", **o),)),
            ("backward", list(back), lambda *a, **o: mkp.linear_q8_backward(*a, z_group=64, act="silu", **o))]


def test_streams(mkp):
    """From torch's current stream and from the stream argument, two at once,
    inputs dropped as soon as the call returns."""
    for M in (4, 60, 700):
        for name, inputs, call in calls(mkp, M):
            ref = [t.clone() for t in call(*inputs)]
            torch.cuda.synchronize()
            streams = [torch.cuda.Stream() for _ in range(2)]
            for rep in range(3):
                got = []
                for st in streams:
                    mine = [t.clone() for t in inputs]
                    st.wait_stream(torch.cuda.current_stream())
                    if rep == 0:
                        with torch.cuda.stream(st):
                            got.append(call(*mine))
                            for t in mine:
                                t.record_stream(st)
                    else:
                        got.append(call(*mine, stream=st if rep == 1 else st.cuda_stream))
                    shapes = [(t.shape, t.dtype) for t in mine]
                    del mine
                    junk = [torch.full(sh, 99, device="cuda", dtype=dt) for sh, dt in shapes]
                torch.cuda.synchronize()
                for outs in got:
                    for o, r in zip(outs, ref):
                        same(o, r, f"{name} on a stream")
                del junk


@pytest.mark.parametrize("M", [1, 30, 300])
def test_captured_into_graphs(mkp, M):
    """Two graphs with a workspace each, replayed with new inputs and eager calls
    between, bit for bit as eager calls."""
    for name, inputs, call in calls(mkp, M):
        call(*inputs)
        torch.cuda.synchronize()
        graphs = []
        for k in range(2):
            mine = [t.clone() for t in inputs]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs = call(*mine)
            graphs.append((graph, mine, outs))
        for rep in range(4):
            for k, (graph, mine, outs) in enumerate(graphs):
                for t in mine:
                    t.copy_(t.flip(0).clone())
                graph.replay()
                want = call(*mine)
                torch.cuda.synchronize()
                for o, r in zip(outs, want):
                    same(o, r, f"{name} replay {rep} of graph {k}")


def test_same_bits_again(mkp):
    for M in (1, 33, 1500):
        for name, inputs, call in calls(mkp, M, 520, 1111):
            first = [t.clone() for t in call(*inputs)]
            for _ in range(3):
                for o, r in zip(call(*inputs), first):
                    same(o, r, f"{name} again")


def test_guarded_workspace(mkp):
    """Every call inside a workspace of exactly the reported bytes, whatever it
    held before."""
    for M, N, K in ((1, 40, 1000), (20, 300, 4096), (100, 1024, 1500), (300, 260, 96), (2000, 3000, 144)):
        x, w, ws, b = layer(gen(M), M, N, K)
        for xx, xt in ((x, mkp.MKP_BF16), (placed(oracle.quantize(x)[0], 1), mkp.MKP_I8)):
            sx = torch.rand(M, device="cuda")
            for ww in (placed(w, (-K) % 16), placed(w, 1)):
                n = mkp.mkp_linear_i8_workspace(M, N, K, xx, xx.stride(0), xt, ww, ww.stride(0))
                buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
                y = torch.empty((M, N), device="cuda")
                mkp.mkp_linear_i8(M, N, K, xx, xx.stride(0), xt, sx, ww, ww.stride(0), ws, b, 0, y, N, mkp.MKP_F32,
                                  buf.data_ptr() + 256, n)
                assert (buf[:256] == 0xA5).all() and (buf[256 + n:] == 0xA5).all()
                q, s = (xx, sx) if xt == mkp.MKP_I8 else oracle.quantize(x)
                within(y, *oracle.linear(q, s, w, ws, b, "none", F32), "guarded")
        dy, x, xs, z, zs = kept(gen(M), M, N, K, 0)
        n = mkp.mkp_linear_q8_backward_workspace(M, N, K, True, True)
        buf = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")
        dw, db = torch.empty((N, K), device="cuda"), torch.empty(N, device="cuda")
        mkp.mkp_linear_q8_backward(M, N, K, dy, N, mkp.MKP_BF16, x, x.stride(0), xs, z, z.stride(0), zs, 1, 0, mkp.MKP_ACT_RELU,
                                   None, 0, dw, K, mkp.MKP_F32, db, buf.data_ptr() + 256, n)
        assert (buf[:256] == 0xFF).all() and (buf[256 + n:] == 0xFF).all()
        ref = oracle.backward(dy, x, xs, z, zs, 0, "relu", F32)
        within(dw, *ref["dw"], "guarded dw")
        within(db, *ref["dbias"], "guarded dbias")


def test_helpers_own_way(mkp, monkeypatch):
    """The helpers without their C++ form: the same bits, and the same refusals."""
    with_it = [(name, [t.clone() for t in call(*inputs)]) for M in (1, 30, 300) for name, inputs, call in calls(mkp, M)]
    assert mkp._direct is not None
    x, w, ws, b = layer(gen(1), 4, 10, 64)
    q, s = mkp.quantize_rows(x)
    refused = [(TypeError, lambda: mkp.quantize_rows(x.half())), (ValueError, lambda: mkp.quantize_rows(x, group=48)),
               (ValueError, lambda: mkp.quantize_rows(x.t())), (ValueError, lambda: mkp.quantize_rows(x.cpu())),
               (ValueError, lambda: mkp.quantize_rows(x[0])), (mkp.MkpError, lambda: mkp.quantize_rows(x[:1].expand(4, 64))),
               (TypeError, lambda: mkp.dequantize_rows(q, s, dtype=torch.int8)), (ValueError, lambda: mkp.dequantize_rows(q, s[:3])),
               (ValueError, lambda: mkp.dequantize_rows(q, s, group=32)), (ValueError, lambda: mkp.linear_i8(x, w, ws[:9])),
               (ValueError, lambda: mkp.linear_i8(x, w.cpu(), ws)), (TypeError, lambda: mkp.linear_i8(x, w, ws, b.double())),
               (ValueError, lambda: mkp.linear_i8(x, w, ws, act="abs")), (TypeError, lambda: mkp.linear_i8(x, w, ws, x_scale=s)),
               (TypeError, lambda: mkp.linear_i8(q, w, ws)), (TypeError, lambda: mkp.linear_i8(x, w, ws, dtype=torch.float16)),
               (ValueError, lambda: mkp.linear_q8_backward(x, q, s, act="relu")),
               (ValueError, lambda: mkp.linear_q8_backward(x, q, s, q, s, z_group=32, act="relu")),
               (TypeError, lambda: mkp.linear_q8_backward(x, x, s)), (ValueError, lambda: mkp.linear_q8_backward(x, q[:3], s)),
               (TypeError, lambda: mkp.linear_q8_backward(x, q, s, grad_dtype=torch.float16))]

    def refuse():
        for i, (kind, call) in enumerate(refused):
            with pytest.raises(kind):
                call()
                raise AssertionError(f"call {i} was not refused")

    refuse()
    monkeypatch.setattr(mkp, "_direct", None)
    refuse()
    again = [(name, call(*inputs)) for M in (1, 30, 300) for name, inputs, call in calls(mkp, M)]
    for (name, first), (_, second) in zip(with_it, again):
        for o, r in zip(second, first):
            same(o, r, name)
            assert o.stride() == r.stride()


def test_outputs_beyond_the_caches(mkp):
    """Outputs larger than the caches, with odd rows: binary32 and bf16."""
    M, K = 5003, 12007
    x = features(gen(1), M, K)
    for group in (0, 256):
        q, s = mkp.quantize_rows(x, group=group)
        for t in (BF, F32):
            y = mkp.dequantize_rows(q, s, group=group, dtype=t)
            for m in (slice(0, 40), slice(M // 2, M // 2 + 40), slice(M - 40, M)):
                same(y[m], oracle.values(q[m], s[m], group).to(F32).to(t), "values past the caches")
    M, N, K = 12001, 12003, 96
    x, w, ws, b = layer(gen(2), M, N, K)
    for t in (BF, F32):
        y = mkp.linear_i8(x, w, ws, b, act="relu", dtype=t)
        for m in (slice(0, 300), slice(M - 300, M)):
            q, s = oracle.quantize(x[m])
            within(y[m], *oracle.linear(q, s, w, ws, b, "relu", t), "a layer past the caches")


# tokens of linear_i8's forms: (M, N, K) of the streaming product with X quantised by it,
# by a launch before it, tiles of each size, and tiles with parts of K
FORMS = [(3, 100, 300), (30, 100, 4096), (60, 100, 300), (400, 300, 300), (4100, 4000, 130), (100, 64, 4096)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", FORMS)
def test_not_finite_through_activations(mkp, M, N, K, t, act):
    """A token or a channel of scale NaN is NaN after every activation, and
    nothing else is."""
    x, w, ws, b = layer(gen(M + K), M, N, K)
    x[0, 5], x[M // 2, K - 1], x[M - 1, 0] = NAN, math.inf, -math.inf
    ws[[2, N - 1]] = NAN
    want = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    want[[0, M // 2, M - 1]] = True
    want[:, [2, N - 1]] = True
    q, s = oracle.quantize(x)
    for xx, xs in ((x, None), (placed(q, (-K) % 16), s)):
        y = check_linear(mkp, xx, w, ws, b, act, t, xs, "not finite")
        assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_empty_sums_of_every_few_tokens(mkp, t):
    """No features: act(bias) for every number of tokens, whatever a kernel before
    left in its workgroups' memory (here NaN, in the outputs that its tiles stage)."""
    N = 5000
    b = torch.randn(N, device="cuda")
    one = torch.ones(4096, device="cuda")
    bad = torch.full((4096, 64), NAN, device="cuda", dtype=t)
    w = torch.ones((4096, 64), dtype=I8, device="cuda")
    for M in range(1, 34):
        assert torch.isnan(mkp.linear_i8(bad, w, one, dtype=BF)).all()
        y = mkp.linear_i8(bad[:M, :0], torch.empty((N, 0), dtype=I8, device="cuda"), torch.ones(N, device="cuda"), b)
        same(y, b.repeat(M, 1), f"{M} tokens of no features")


@pytest.mark.parametrize("own_way", [False, True])
def test_rows_of_no_columns(mkp, own_way, monkeypatch):
    """A scale for each row of no columns too, the least one; nothing to sum gives act(bias)."""
    if own_way:
        monkeypatch.setattr(mkp, "_direct", None)
    b = torch.randn(9, device="cuda")
    for M in (1, 12, 300):
        for stream in (None, torch.cuda.Stream()):
            del [torch.full((M,), NAN, device="cuda") for _ in range(4)][:]
            q, s = mkp.quantize_rows(torch.empty((M, 0), dtype=BF, device="cuda"), stream=stream)
            torch.cuda.synchronize()
            assert q.shape == (M, 0) and q.dtype == I8
            same(s, torch.full((M,), 2.0 ** -126, device="cuda"), "scales of no columns")
            assert mkp.dequantize_rows(q, s).shape == (M, 0)
            y = mkp.linear_i8(q, torch.empty((9, 0), dtype=I8, device="cuda"), torch.ones(9, device="cuda"), b, x_scale=s)
            same(y, b.repeat(M, 1), "a layer of no features")
        q, s = mkp.quantize_rows(torch.empty((M, 0), device="cuda"), group=64)
        assert q.shape == (M, 0) and s.shape == (M, 0)


@pytest.mark.parametrize("own_way", [False, True])
def test_scales_broadcast_over_rows_are_refused(mkp, own_way, monkeypatch):
    """A scale with one place for all rows has a leading dimension of 0: the library says so
    instead of reading past it."""
    if own_way:
        monkeypatch.setattr(mkp, "_direct", None)
    dy, x, xs, z, zs = kept(gen(2), 40, 64, 48, 64)
    one = torch.ones((1, 1), device="cuda")
    for bad in (one.expand(40, 1), one[0].expand(40, 1)):
        assert bad.stride(0) == 0
        with pytest.raises(mkp.MkpError):
            mkp.dequantize_rows(z, bad, group=64)
        with pytest.raises(mkp.MkpError):
            mkp.linear_q8_backward(dy, x, xs, z, bad, z_group=64, act="gelu")
    for bad in (one[0].expand(40),):
        with pytest.raises(ValueError):
            mkp.dequantize_rows(z, bad)
        with pytest.raises(ValueError):
            mkp.linear_q8_backward(dy, x, bad, z, zs, z_group=64, act="gelu")
    # (one row is all rows; without an activation z's scales are not looked at)
    same(mkp.dequantize_rows(z[:1], one, group=64), z[:1].to(BF), "one row")
    mkp.linear_q8_backward(dy, x, xs, z, one.expand(40, 1), z_group=64)


@pytest.mark.parametrize("K,t", [(8200, BF), (8193, F32), (16400, BF)], ids=["bf16", "f32", "bf16_wide"])
def test_more_long_rows_than_workgroups_of_1024(mkp, K, t):
    """2^22 rows of more than 8192 columns: 2^32 threads, were a workgroup of 1024 a row's."""
    M = 1 << 22
    torch.cuda.empty_cache()
    size = M * K * (2 if t == BF else 4) + M * (K + 32)
    if torch.cuda.mem_get_info()[0] < size + (8 << 30):
        pytest.skip(f"{size >> 30} GiB and some are not free")
    x = torch.empty((M, K), dtype=t, device="cuda")
    x.fill_(1.0)
    rows = [0, 1, 12345, M // 2, M - 2, M - 1]
    some = features(gen(K), len(rows), K, t)
    for i, m in enumerate(rows):
        x[m] = some[i]
    wq, ws = oracle.quantize(some)
    q, s = mkp.quantize_rows(x)
    same(q[rows], wq, "integers")
    same(s[rows], ws, "scales")
    assert int((s == torch.tensor(1.0 / 127.0, dtype=F32, device="cuda")).sum()) == M - len(rows)
    y = mkp.dequantize_rows(q[M - 2:], s[M - 2:])
    same(y, oracle.values(wq[4:], ws[4:]).to(F32).to(BF), "values")
    del q
    torch.cuda.empty_cache()
    w, sw = oracle.quantize(torch.randn(16, K, generator=gen(1), device="cuda"))
    y = mkp.linear_i8(x, w, sw)
    within(y[rows], *oracle.linear(wq, ws, w, sw, None, "none", F32), "a layer of as many tokens")
    del x, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_are_exact_to_their_bound(mkp, act):
    """One token whose gradient is 1: dbias is the slope itself, in binary32.  Scales
    of 0.01 to 0.98 bring |z| from 0.01 to 124, every place of each slope."""
    z = (torch.arange(254, device="cuda", dtype=torch.int32) % 127 + 1).to(I8)
    z[127:] *= -1
    one = torch.ones((1, 254), device="cuda")
    worst = 0.0
    for i in range(200):
        zs = torch.tensor([0.01 * 1.0233 ** i], device="cuda")
        _, _, db = mkp.linear_q8_backward(one, torch.zeros((1, 16), dtype=I8, device="cuda"), one[0, :1], z[None], zs, act=act,
                                          need_dz=False, need_dw=False)
        ref = oracle.slope(act, oracle.values(z[None], zs))[0]
        within(db, ref, torch.full_like(ref, oracle.SLOPE), f"slope of {act}, scale {i}")
        worst = max(worst, float((db.double() - ref).abs().max()))
    print(f"[slope] {act} {worst:.3e}", flush=True)


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("N,K", [(256, 256), (2304, 768), (333, 517), (1003, 2050), (4100, 3000)])
@pytest.mark.parametrize("M", [65, 1000, 4097, 8191, 8192])
def test_backward_in_whole_numbers(mkp, M, N, K, act):
    """Gradients and inputs of small whole numbers, scales of powers of two: every
    product and every sum, in any order, is exact in binary32 (at most 8192 * 3 * 7 =
    2^17.4, in quarters), so a row that is left out, or taken twice, shows in each element."""
    g = gen(M + N)

    def whole(hi, *shape):
        return torch.randint(-hi, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)

    dy = whole(3, M, N)
    x, z = whole(7, M, K).to(I8), whole(5, M, N).to(I8)
    xs = torch.exp2(whole(1, M).to(F32) - 1)
    dz = dy * (z > 0) if act == "relu" else dy
    want = dz.to(F64).t() @ (x.to(F64) * xs.to(F64)[:, None])
    for t, gt in ((BF, F32), (F32, BF)):
        got = mkp.linear_q8_backward(dy.to(t), placed(x, (-K) % 8), xs, z, torch.ones(M, device="cuda"), act=act, grad_dtype=gt)
        same(got[0], dz.to(BF), "dz")
        same(got[1], want.to(F32).to(gt), "dw")
        same(got[2], dz.sum(0, dtype=torch.int64).to(F32), "dbias")


@pytest.mark.parametrize("M,N,K", [(3, 40, 24), (333, 768, 768), (8192, 300, 130), (700, 2900, 3000)])
def test_binary32_weight_gradients(mkp, M, N, K):
    """Two passes over one workspace: as exact as their bound whatever else is asked for,
    the same bits again, from a graph and from another stream."""
    a = kept(gen(M + K), M, N, K, 64, F32)
    first = check_backward(mkp, *a, 64, "silu", F32)
    for need in (dict(need_dz=False), dict(need_dbias=False), dict(need_dz=False, need_dbias=False)):
        same(check_backward(mkp, *a, 64, "silu", F32, **need)[1], first[1], "dw alone")

    def call(**o):
        return mkp.linear_q8_backward(*a, z_group=64, act="silu", grad_dtype=F32, **o)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    on = call(stream=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for rep in range(3):
        for o in outs:
            o.fill_(NAN)
        graph.replay()
        again = call()
        torch.cuda.synchronize()
        for name, f, *others in zip(("dz", "dw", "dbias"), first, on, outs, again):
            for o in others:
                same(o, f, name)


@pytest.mark.parametrize("gt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(70, 48), (2900, 3000)])
def test_gradients_that_are_not_finite(mkp, N, K, gt):
    """An infinite gradient makes its channel's weight gradient infinite, of x's sign; a
    NaN, NaN; other channels are what they were."""
    M = 200
    dy, x, xs, _, _ = kept(gen(N), M, N, K, 0, F32)
    x[x == 0] = 1
    ref = mkp.linear_q8_backward(dy, x, xs, grad_dtype=gt)[1]
    dy[7, 3], dy[199, 20], dy[64, N - 1] = math.inf, -math.inf, NAN
    dw = mkp.linear_q8_backward(dy, x, xs, grad_dtype=gt)[1]
    same(dw[3], torch.where(x[7] > 0, math.inf, -math.inf).to(gt), "an infinity")
    same(dw[20], torch.where(x[199] > 0, -math.inf, math.inf).to(gt), "a negative one")
    assert torch.isnan(dw[N - 1]).all()
    rest = [n for n in range(N) if n not in (3, 20, N - 1)]
    same(dw[rest], ref[rest], "the others")
