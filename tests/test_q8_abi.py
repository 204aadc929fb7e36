"""Refusals of the 8-bit entry points: each comes back before anything is
launched, so none needs a GPU (addresses are never followed)."""
import pytest
import torch

A = 1 << 20   # an aligned address that is never read


@pytest.fixture(scope="module")
def mkp():
    import dynamic_shape_gemm_amd as m
    return m


def quantize(mkp, **over):
    a = dict(M=4, K=64, X=A, ldx=64, x_type=0, group=0, Q=A, ldq=64, S=A, lds=1, stream=0)
    a.update(over)
    return mkp.mkp_quantize_rows_raw(**a)


def dequantize(mkp, **over):
    a = dict(M=4, K=64, Q=A, ldq=64, S=A, lds=1, group=0, Y=A, ldy=64, y_type=0, stream=0)
    a.update(over)
    return mkp.mkp_dequantize_rows_raw(**a)


def linear(mkp, **over):
    a = dict(M=4, N=10, K=64, X=A, ldx=64, x_type=0, x_scale=0, W=A, ldw=64, w_scale=A, bias=0, act=0, Y=A, ldy=10, y_type=1,
             workspace=A, workspace_bytes=0, stream=0)
    a.update(over)
    return mkp.mkp_linear_i8_raw(**a)


def backward(mkp, **over):
    a = dict(M=4, N=10, K=64, dY=A, lddy=10, dy_type=0, X=A, ldx=64, x_scale=A, Z=A, ldz=10, z_scale=A, ldzs=1, z_group=0, act=2,
             dZ=A, lddz=10, dW=A, lddw=64, dw_type=0, dbias=A, workspace=A, workspace_bytes=0, stream=0)
    a.update(over)
    return mkp.mkp_linear_q8_backward_raw(**a)


CONVERT = [dict(M=-1), dict(K=-1), dict(ldq=63), dict(S=0), dict(Q=0), dict(group=16), dict(group=-32), dict(group=512),
           dict(group=32, lds=1), dict(lds=0)]
CASES = [
    (quantize, CONVERT + [dict(X=0), dict(ldx=63), dict(x_type=2), dict(x_type=-1)]),
    (dequantize, CONVERT + [dict(Y=0), dict(ldy=63), dict(y_type=2)]),
    (linear, [dict(M=-1), dict(N=-1), dict(K=-1), dict(X=0), dict(W=0), dict(w_scale=0), dict(Y=0), dict(ldx=63), dict(ldw=63),
              dict(ldy=9), dict(x_type=3), dict(x_type=2), dict(y_type=2), dict(act=5), dict(act=-1)]),
    (backward, [dict(M=-1), dict(N=-1), dict(K=-1), dict(dY=0), dict(X=0), dict(x_scale=0), dict(Z=0), dict(z_scale=0),
                dict(lddy=9), dict(ldx=63), dict(ldz=9), dict(ldzs=0), dict(lddz=9), dict(lddw=63), dict(dy_type=2),
                dict(dw_type=2), dict(act=7), dict(z_group=48)]),
]


@pytest.mark.parametrize("fn,cases", CASES, ids=lambda v: getattr(v, "__name__", ""))
def test_bad_arguments(mkp, fn, cases):
    for over in cases:
        assert fn(mkp, **over) == mkp.MKP_ERR_INVALID_ARG, over
        assert mkp.last_error() and "workspace" not in mkp.last_error(), over


def test_what_a_launch_cannot_count(mkp):
    for fn, over in ((quantize, dict(M=1 << 24)), (quantize, dict(K=1 << 23, ldx=1 << 23, ldq=1 << 23)),
                     (dequantize, dict(M=1 << 24)), (quantize, dict(ldx=1 << 25)), (linear, dict(M=1 << 24)),
                     (linear, dict(N=1 << 23, ldy=1 << 23)), (linear, dict(K=131072, ldx=131072, ldw=131072)),
                     (backward, dict(M=1 << 24))):
        assert fn(mkp, **over) == mkp.MKP_ERR_UNSUPPORTED, over
    big = dict(M=(1 << 24) - 1, N=1 << 22)
    need = mkp.mkp_linear_i8_workspace(big["M"], big["N"], 64, A, 64, 2, A, 64)
    assert linear(mkp, x_type=2, x_scale=A, ldy=1 << 22, workspace_bytes=need, **big) == mkp.MKP_ERR_UNSUPPORTED
    need = mkp.mkp_linear_q8_backward_workspace(big["M"], big["N"], 64, 1, 1)
    assert backward(mkp, lddy=1 << 22, ldz=1 << 22, lddz=1 << 22, workspace_bytes=need, **big) == mkp.MKP_ERR_UNSUPPORTED


def test_workspace_is_checked(mkp):
    M, N, K = 300, 100, 640
    ext = dict(M=M, N=N, K=K, ldx=K)
    need = mkp.mkp_linear_i8_workspace(M, N, K, A, K, 0, A, K)
    assert need > 0
    more = dict(ext, ldw=K, ldy=N)
    for bad in (dict(workspace=0, workspace_bytes=need), dict(workspace_bytes=need - 1), dict(workspace_bytes=-1),
                dict(workspace=A + 8, workspace_bytes=need)):
        assert linear(mkp, **more, **bad) == mkp.MKP_ERR_INVALID_ARG and "workspace" in mkp.last_error(), bad
    need = mkp.mkp_linear_q8_backward_workspace(M, N, K, 1, 1)
    more = dict(ext, lddy=N, ldz=N, lddz=N, lddw=K)
    for bad in (dict(workspace=0, workspace_bytes=need), dict(workspace_bytes=need - 1), dict(workspace_bytes=-1),
                dict(workspace=A + 8, workspace_bytes=need)):
        assert backward(mkp, **more, **bad) == mkp.MKP_ERR_INVALID_ARG and "workspace" in mkp.last_error(), bad
    # copies of unaligned operands need room
    plain = mkp.mkp_linear_i8_workspace(M, N, K, A, K, 2, A, K)
    assert mkp.mkp_linear_i8_workspace(M, N, K, A + 1, K, 2, A, K) > plain
    assert mkp.mkp_linear_i8_workspace(M, N, K, A, K, 2, A, K + 1) > plain
    assert mkp.mkp_linear_q8_backward_workspace(M, N, K, 0, 0) == 0
    for bad in ((-1, 10, 8, A, 8, 0, A, 8), (4, 10, 8, A, 7, 0, A, 8), (4, 10, 8, A, 8, 0, A, 7), (4, 10, 8, A, 8, 9, A, 8)):
        with pytest.raises(mkp.MkpError):
            mkp.mkp_linear_i8_workspace(*bad)
    with pytest.raises(mkp.MkpError):
        mkp.mkp_linear_q8_backward_workspace(-1, 4, 4, 1, 1)


def test_nothing_to_do(mkp):
    assert quantize(mkp, M=0, X=0, Q=0, S=0) == mkp.MKP_OK
    assert quantize(mkp, K=0, X=0, Q=0, S=0) == mkp.MKP_OK
    assert dequantize(mkp, M=0, Y=0, Q=0, S=0) == mkp.MKP_OK
    assert linear(mkp, M=0, X=0, Y=0, workspace=0) == mkp.MKP_OK
    assert linear(mkp, N=0, W=0, w_scale=0, Y=0, workspace=0) == mkp.MKP_OK
    assert backward(mkp, dZ=0, dW=0, dbias=0, workspace=0) == mkp.MKP_OK
    assert backward(mkp, N=0, dY=0, Z=0, workspace=0) == mkp.MKP_OK
    assert backward(mkp, M=0, dY=0, Z=0, X=0, dW=0, dbias=0, workspace=0) == mkp.MKP_OK


def test_helpers_refuse(mkp):
    bf, i8 = torch.bfloat16, torch.int8
    x, w, s = torch.zeros(3, 64, dtype=bf), torch.zeros(5, 64, dtype=i8), torch.zeros(5)
    cases = [
        (TypeError, lambda: mkp.quantize_rows(x.half())),
        (ValueError, lambda: mkp.quantize_rows(x)),                       # not on a GPU
        (ValueError, lambda: mkp.quantize_rows(x[0])),
        (ValueError, lambda: mkp.quantize_rows(x, group=48)),
        (ValueError, lambda: mkp.dequantize_rows(w, s)),
        (TypeError, lambda: mkp.dequantize_rows(w, s, dtype=torch.float16)),
        (TypeError, lambda: mkp.dequantize_rows(x, s)),
        (ValueError, lambda: mkp.linear_i8(x[:, :60], w, s)),
        (TypeError, lambda: mkp.linear_i8(x.half(), w, s)),
        (ValueError, lambda: mkp.linear_i8(x, w, s)),
        (ValueError, lambda: mkp.linear_i8(x, w, s, act="swish")),
        (ValueError, lambda: mkp.linear_q8_backward(x, w, s)),
        (ValueError, lambda: mkp.linear_q8_backward(x, w[:3], s[:3], act="abs")),
        (TypeError, lambda: mkp.linear_q8_backward(x, w[:3], s[:3], grad_dtype=torch.float16)),
    ]
    for i, (kind, call) in enumerate(cases):
        with pytest.raises(kind):
            call()
            raise AssertionError(f"case {i} was not refused")
