"""Refusals of RMS norm: every bad call returns its error before anything
reaches the GPU (fake addresses, CPU)."""
import pytest

L = pytest.importorskip("linear_cross_entropy_gemm_amd")
torch = pytest.importorskip("torch")


# The base call of each helper is complete except for one refusal that is
# checked last, so no variant with fake addresses can reach a launch.
def _fwd(f=L.flce_rms_norm_fwd, **kw):
    a = dict(x=16, ld_x=8, residual=32, ld_r=8, weight=16, offset=0.0, M=2, H=8, eps=1e-6, y=64, ld_y=8, sum=32,
             ld_s=9, rstd=16, stream=0, dtype=0, w_dtype=0)   # sum in the place of the residual, another stride
    a.update(kw)
    return f(*a.values())


FWD = [
    (dict(dtype=2), L.FLCE_EINVAL), (dict(w_dtype=-1), L.FLCE_EINVAL), (dict(M=-1), L.FLCE_EINVAL),
    (dict(H=0), L.FLCE_EINVAL), (dict(M=1 << 31), L.FLCE_EUNSUPPORTED), (dict(H=(1 << 21) + 1), L.FLCE_EUNSUPPORTED),
    (dict(H=(1 << 32) + 8), L.FLCE_EUNSUPPORTED),
    (dict(eps=0.0), L.FLCE_EINVAL), (dict(eps=-1.0), L.FLCE_EINVAL), (dict(eps=float("nan")), L.FLCE_EINVAL),
    (dict(eps=float("inf")), L.FLCE_EINVAL), (dict(offset=float("inf")), L.FLCE_EINVAL),
    (dict(offset=float("nan")), L.FLCE_EINVAL), (dict(x=None), L.FLCE_EINVAL), (dict(y=None), L.FLCE_EINVAL),
    (dict(x=17), L.FLCE_EINVAL), (dict(weight=17), L.FLCE_EINVAL), (dict(residual=33), L.FLCE_EINVAL),
    (dict(sum=33), L.FLCE_EINVAL), (dict(residual=None), L.FLCE_EINVAL), (dict(sum=None), L.FLCE_EINVAL),
    (dict(rstd=18), L.FLCE_EINVAL), (dict(ld_x=-1), L.FLCE_EINVAL), (dict(ld_r=-1), L.FLCE_EINVAL),
    (dict(ld_y=7), L.FLCE_EINVAL), (dict(ld_s=7), L.FLCE_EINVAL), (dict(y=32), L.FLCE_EINVAL),
    (dict(), L.FLCE_EINVAL), (dict(M=0, x=None, y=None), L.FLCE_OK),
]


@pytest.mark.parametrize("kw,code", FWD + [(dict(y=65), L.FLCE_EINVAL), (dict(sum=48, y=16, ld_y=9), L.FLCE_EINVAL)])
def test_rms_norm_fwd_rejects_before_launch(kw, code):
    assert _fwd(**kw) == code


def _mx(x, ld_x, residual, ld_r, weight, offset, M, H, eps, y, ld_y, sum, ld_s, rstd, stream, dtype, w_dtype,
        scales=128, ld_scales=1):
    return L.flce_rms_norm_mx(x, ld_x, residual, ld_r, weight, offset, M, H, eps, y, ld_y, scales, ld_scales, sum, ld_s,
                              rstd, stream, dtype, w_dtype)


@pytest.mark.parametrize("kw,code", FWD + [
    (dict(scales=None), L.FLCE_EINVAL), (dict(ld_scales=0), L.FLCE_EINVAL), (dict(y=16, sum=48), L.FLCE_EINVAL),
    (dict(y=32, sum=48), L.FLCE_EINVAL)])
def test_rms_norm_mx_rejects_before_launch(kw, code):
    assert _fwd(_mx, **kw) == code


def _bwd(**kw):
    a = dict(grad_y=16, ld_gy=8, s=32, ld_s=8, grad_s=48, ld_gs=8, weight=16, offset=0.0, rstd=16, M=2, H=8, grad_x=64,
             ld_gx=8, grad_weight=16, stream=0, dtype=0, w_dtype=0, workspace=256, workspace_bytes=0)
    a.update(kw)
    return L.flce_rms_norm_bwd(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), L.FLCE_EINVAL), (dict(w_dtype=2), L.FLCE_EINVAL), (dict(M=-1), L.FLCE_EINVAL),
    (dict(H=0), L.FLCE_EINVAL), (dict(H=(1 << 21) + 1), L.FLCE_EUNSUPPORTED), (dict(offset=float("nan")), L.FLCE_EINVAL),
    (dict(grad_y=None), L.FLCE_EINVAL), (dict(s=None), L.FLCE_EINVAL), (dict(rstd=None), L.FLCE_EINVAL),
    (dict(grad_y=17), L.FLCE_EINVAL), (dict(s=33), L.FLCE_EINVAL), (dict(grad_s=49), L.FLCE_EINVAL),
    (dict(grad_x=65), L.FLCE_EINVAL), (dict(weight=17), L.FLCE_EINVAL), (dict(grad_weight=17), L.FLCE_EINVAL),
    (dict(rstd=18), L.FLCE_EINVAL), (dict(ld_gy=-1), L.FLCE_EINVAL), (dict(ld_s=-1), L.FLCE_EINVAL),
    (dict(ld_gs=-1), L.FLCE_EINVAL), (dict(ld_gx=7), L.FLCE_EINVAL), (dict(grad_x=16), L.FLCE_EINVAL),
    (dict(grad_x=32), L.FLCE_EINVAL), (dict(grad_x=48), L.FLCE_EINVAL), (dict(workspace=None), L.FLCE_EINVAL),
    (dict(workspace=128), L.FLCE_EINVAL), (dict(), L.FLCE_EWORKSPACE), (dict(M=0, grad_weight=None), L.FLCE_OK),
])
def test_rms_norm_bwd_rejects_before_launch(kw, code):
    assert _bwd(**kw) == code


def test_rms_norm_bwd_workspace_size():
    for M, H, dt in [(1, 1, 0), (8192, 6656, 0), (4099, 5003, 1), (100000, 64, 0), (3, 1 << 21, 1), (0, 8, 0)]:
        b = L.flce_rms_norm_bwd_workspace_size(M, H, dt)
        assert b % 256 == 0 and 4 * H <= b <= 1024 * 4 * H + 256
    assert L.flce_rms_norm_bwd_workspace_size(-1, 8, 0) == 0
    assert L.flce_rms_norm_bwd_workspace_size(1, (1 << 21) + 1, 0) == 0
    assert L.flce_rms_norm_bwd_workspace_size(1, 8, 3) == 0


def test_wrappers_refuse_bad_tensors():
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    for f in (lambda: L.rms_norm_fwd(x), lambda: L.rms_norm(x), lambda: L.rms_norm_mx8(x),
              lambda: L.rms_norm_bwd(x, x, None, x)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(TypeError):
        L.rms_norm_fwd(x.half())
    W, lab = torch.zeros(5, 8), torch.zeros(2, dtype=torch.int64)
    for kw in (dict(norm="batch"), dict(norm="rms", norm_bias=torch.zeros(8)), dict(norm_offset=1.0)):
        with pytest.raises(ValueError, match="norm"):
            L.lm_head_loss(x, W, lab, None, **kw)


@pytest.mark.parametrize("where", ["x", "weight", "residual", "lm_head_loss"])
def test_forward_mode_tangents_are_refused_not_dropped(where, monkeypatch):
    import torch.autograd.forward_ad as fw
    from linear_cross_entropy_gemm_amd import head

    def fwd(x, w, eps, residual, offset, stats, mx8=False):
        return x.detach().clone(), None if residual is None else x.detach().clone(), torch.ones(3)
    monkeypatch.setattr(head, "_rms_norm_fwd", fwd)
    x, w, r = torch.randn(3, 4), torch.randn(4), torch.randn(3, 4)
    calls = {"x": (x, lambda d: L.rms_norm(d, w)), "weight": (w, lambda d: L.rms_norm(x, d)),
             "residual": (r, lambda d: L.rms_norm(x, w, residual=d)),
             "lm_head_loss": (x, lambda d: L.lm_head_loss(d, torch.randn(5, 4), torch.zeros(3, dtype=torch.int64), w,
                                                          residual=r, norm="rms"))}
    t, call = calls[where]
    with fw.dual_level():
        with pytest.raises(NotImplementedError, match="jvp"):
            call(fw.make_dual(t.clone(), torch.ones_like(t)))
    assert torch.equal(L.rms_norm(x, w), x)
