"""Refusals of the vocabulary losses' entry points: each comes back before
anything is launched, so none needs a GPU (addresses are never followed)."""
import pytest
import torch

A = 1 << 20   # an aligned address that is never read


@pytest.fixture(scope="module")
def mkp():
    import dynamic_shape_gemm_amd as m
    return m


def xent(mkp, **over):
    a = dict(M=4, V=10, K=8, X=A, ldx=8, W=A, ldw=8, bias=0, labels=A, scale=1.0, softcap=0.0, smoothing=0.0, z_loss=0.0,
             loss=A, lse=A, workspace=A, workspace_bytes=0, stream=0)
    a.update(over)
    return mkp.mkp_linear_xent_raw(**a)


def xent_bwd(mkp, **over):
    a = dict(M=4, V=10, K=8, X=A, ldx=8, W=A, ldw=8, bias=0, labels=A, scale=1.0, softcap=0.0, smoothing=0.0, z_loss=0.0,
             lse=A, dloss=A, dX=A, lddx=8, dW=A, lddw=8, dbias=0, grad_type=0, workspace=A, workspace_bytes=0, stream=0)
    a.update(over)
    return mkp.mkp_linear_xent_backward_raw(**a)


def distill(mkp, **over):
    a = dict(M=4, V=10, K=8, X=A, ldx=8, W=A, ldw=8, bias=0, k=3, ids=A, ldids=3, teacher=A, ldt=3, teacher_lse=0,
             temperature=1.0, scale=1.0, softcap=0.0, loss=A, lse=A, workspace=A, workspace_bytes=0, stream=0)
    a.update(over)
    return mkp.mkp_linear_distill_raw(**a)


def distill_bwd(mkp, **over):
    a = dict(M=4, V=10, K=8, X=A, ldx=8, W=A, ldw=8, bias=0, k=3, ids=A, ldids=3, teacher=A, ldt=3, teacher_lse=0,
             temperature=1.0, scale=1.0, softcap=0.0, lse=A, dloss=A, dX=A, lddx=8, dW=A, lddw=8, dbias=0, grad_type=0,
             workspace=A, workspace_bytes=0, stream=0)
    a.update(over)
    return mkp.mkp_linear_distill_backward_raw(**a)


COMMON = [dict(M=-1), dict(V=0), dict(K=0), dict(V=-3), dict(K=1 << 22, ldx=1 << 22, ldw=1 << 22), dict(M=1 << 31),
          dict(V=1 << 31), dict(ldx=7), dict(ldw=7), dict(X=0), dict(W=0), dict(lse=0), dict(scale=float("nan")),
          dict(scale=float("inf")), dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=1e-39)]
BWD = [dict(dloss=0), dict(grad_type=2), dict(lddx=7), dict(lddw=7)]
DISTILL = [dict(k=0), dict(k=-1), dict(k=1025, ldids=1025, ldt=1025), dict(ids=0), dict(teacher=0), dict(ldids=2),
           dict(ldt=2), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("inf")),
           dict(temperature=1e-39)]
XENT = [dict(labels=0), dict(smoothing=-0.1), dict(smoothing=1.1), dict(smoothing=float("nan")),
        dict(z_loss=float("inf"))]


@pytest.mark.parametrize("fn,cases", [(xent, COMMON + XENT + [dict(loss=0)]), (xent_bwd, COMMON + XENT + BWD),
                                      (distill, COMMON + DISTILL + [dict(loss=0)]),
                                      (distill_bwd, COMMON + DISTILL + BWD)])
def test_bad_arguments(mkp, fn, cases):
    for over in cases:
        assert fn(mkp, **over) == mkp.MKP_ERR_INVALID_ARG, over
        assert mkp.last_error() and "workspace" not in mkp.last_error(), over


@pytest.mark.parametrize("fn,k,back", [(xent, 0, 0), (xent_bwd, 0, 1), (distill, 3, 0), (distill_bwd, 3, 1)])
def test_workspace_is_checked(mkp, fn, k, back):
    need = mkp.mkp_linear_loss_workspace(4, 10, 8, k, A, 8, back)
    assert need > 0
    for over in (dict(workspace=0, workspace_bytes=need), dict(workspace_bytes=need - 1), dict(workspace_bytes=-1),
                 dict(workspace=A + 8, workspace_bytes=need)):
        assert fn(mkp, **over) == mkp.MKP_ERR_INVALID_ARG, over
        assert "workspace" in mkp.last_error()
    # an unaligned weight needs room for its copy
    assert mkp.mkp_linear_loss_workspace(4, 1000, 8, k, A + 2, 8, back) > mkp.mkp_linear_loss_workspace(4, 1000, 8, k, A, 8, back)
    for bad in ((-1, 10, 8, 0), (4, 0, 8, 0), (4, 10, 0, 0), (4, 10, 8, -1), (4, 10, 8, 1025)):
        with pytest.raises(mkp.MkpError):
            mkp.mkp_linear_loss_workspace(*bad, A, 8, back)


def test_too_large_for_a_launch(mkp):
    """Extents whose tiles a launch cannot count, with a workspace to match."""
    M = V = 1 << 29
    need = mkp.mkp_linear_loss_workspace(M, V, 64, 0, A, 64, 0)
    assert xent(mkp, M=M, V=V, K=64, ldx=64, ldw=64, workspace_bytes=need) == mkp.MKP_ERR_UNSUPPORTED
    M, K = (1 << 30) - 1, 1 << 21
    need = mkp.mkp_linear_loss_workspace(M, 10, K, 0, A, K, 1)
    assert xent_bwd(mkp, M=M, K=K, ldx=K, ldw=K, lddx=K, lddw=K, workspace_bytes=need) == mkp.MKP_ERR_UNSUPPORTED
    # a workgroup per row, tiles of 512 threads, chunks of a padded weight: 2^32 threads each
    for fn, back, W, ext in ((xent, 0, A, dict(M=1 << 24)), (xent_bwd, 1, A, dict(M=1 << 24)),
                             (xent, 0, A, dict(M=1 << 20, V=1 << 19)),
                             (xent, 0, A + 2, dict(V=1 << 29, K=64, ldx=64, ldw=64))):
        a = dict(dict(M=4, V=10, K=8, ldw=8), **ext)
        need = mkp.mkp_linear_loss_workspace(a["M"], a["V"], a["K"], 0, W, a["ldw"], back)
        assert fn(mkp, W=W, workspace_bytes=need, **ext) == mkp.MKP_ERR_UNSUPPORTED, ext


def test_nothing_to_do(mkp):
    assert xent(mkp, M=0, X=0, labels=0, loss=0, lse=0, workspace=0) == mkp.MKP_OK
    assert distill(mkp, M=0, X=0, ids=0, teacher=0, loss=0, lse=0, workspace=0) == mkp.MKP_OK
    assert xent_bwd(mkp, dX=0, dW=0, workspace=0) == mkp.MKP_OK
    assert xent_bwd(mkp, M=0, X=0, labels=0, lse=0, dloss=0, dW=0, workspace=0) == mkp.MKP_OK


def test_workspace_does_not_hold_the_logits(mkp):
    """Well below four bytes a logit: a piece of the gradient, and statistics."""
    M, V, K = 8192, 128256, 4096
    assert mkp.mkp_linear_loss_workspace(M, V, K, 0, A, K, 0) < M * V // 4
    assert mkp.mkp_linear_loss_workspace(M, V, K, 0, A, K, 1) < M * V


def test_helpers_refuse(mkp):
    bf = torch.bfloat16
    x, w, y = torch.zeros(3, 8, dtype=bf), torch.zeros(5, 8, dtype=bf), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError):
        mkp.linear_xent(x.float(), w, y)
    with pytest.raises(ValueError):
        mkp.linear_xent(x, w[:, :7], y)
    with pytest.raises(ValueError):
        mkp.linear_xent(x, w, y)                       # not on a GPU
    with pytest.raises(TypeError):
        mkp.linear_xent(x, w, y.int())
    with pytest.raises(ValueError):
        mkp.linear_xent(x, w, y[:2])
    with pytest.raises(ValueError):
        mkp.linear_xent(x.t().contiguous().t(), w, y)
    ids, t = torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2)
    with pytest.raises(ValueError):
        mkp.linear_distill(x, w, ids[:, :0], t[:, :0])
    with pytest.raises(ValueError):
        mkp.linear_distill(x, w, ids, t[:, :1])
    with pytest.raises(TypeError):
        mkp.linear_distill(x, w, ids, t.double())


def test_build_refuses_tiles_that_fill_a_cu_alone():
    """A loss tile of 269 registers (one wave a SIMD) is named, one of 239 not."""
    import importlib.util
    import os

    import dynamic_shape_gemm_amd as m
    path = os.path.join(os.path.dirname(m.__file__), "build.py")
    spec = importlib.util.spec_from_file_location("mkp_build", path)
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    remark = ("x.hip:1:0: remark: Function Name: {} [-R]\nx.hip:1:0: remark:     VGPRs: {} [-R]\n"
              "x.hip:1:0: remark:     Occupancy [waves/SIMD]: {} [-R]\n")
    usage = build.parse_resource_usage(remark.format("a_loss_grad_kernel", 173, 1) +
                                       remark.format("b_loss_grad_kernel", 143, 2) +
                                       remark.format("loss_stream_kernel", 62, 1))
    assert build.too_few_waves(usage) == ["a_loss_grad_kernel"]
    if os.path.exists(build.RESOURCE_REPORT):   # what was built
        with open(build.RESOURCE_REPORT) as f:
            built = {line.split()[0]: dict(p.split("=") for p in line.split()[1:]) for line in f}
        tiles = [u for k, u in built.items() if "loss_grad_kernel" in k or "loss_forward_kernel" in k]
        assert tiles and all(int(u["occupancy"]) >= 2 for u in tiles)


@pytest.mark.parametrize("fn", [distill, distill_bwd])
def test_temperatures_whose_square_is_no_number(mkp, fn):
    """T^2 times the divergence is the loss: infinite or 0 it would be NaN."""
    for T in (1e20, 2e19, 1e-20, 1e-30):
        assert fn(mkp, temperature=T) == mkp.MKP_ERR_INVALID_ARG, T
        assert "temperature" in mkp.last_error(), T
    for T in (1e18, 1e-18):   # what is missing now is the workspace
        assert fn(mkp, temperature=T) == mkp.MKP_ERR_INVALID_ARG and "workspace" in mkp.last_error(), T
