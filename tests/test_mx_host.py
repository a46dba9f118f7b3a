"""Refusals of the 4-bit projection: every bad call returns its error before
anything reaches the GPU (fake addresses, CPU)."""
import pytest

L = pytest.importorskip("linear_cross_entropy_gemm_amd")
torch = pytest.importorskip("torch")


# The base call of each helper is complete except for one refusal that is
# checked last, so no variant with fake addresses can reach a launch.
def _pack(**kw):
    a = dict(W=16, ld_w=-1, V=4, H=8, packed=16, scales=16, stream=0, dtype=0)
    a.update(kw)
    return L.flce_pack_mx(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), L.FLCE_EINVAL), (dict(V=-1), L.FLCE_EINVAL), (dict(H=0), L.FLCE_EINVAL),
    (dict(V=(1 << 24) + 1), L.FLCE_EUNSUPPORTED), (dict(H=(1 << 21) + 1), L.FLCE_EUNSUPPORTED),
    (dict(V=1 << 20, H=1 << 16), L.FLCE_EUNSUPPORTED), (dict(W=None), L.FLCE_EINVAL),
    (dict(packed=None), L.FLCE_EINVAL), (dict(scales=None), L.FLCE_EINVAL), (dict(W=17), L.FLCE_EINVAL),
    (dict(W=18, dtype=1), L.FLCE_EINVAL), (dict(packed=24), L.FLCE_EINVAL), (dict(scales=18), L.FLCE_EINVAL), (dict(), L.FLCE_EINVAL),
    (dict(V=0, W=None, packed=None, scales=None), L.FLCE_OK),
])
def test_pack_rejects_before_launch(kw, code):
    assert _pack(**kw) == code


def _logits(**kw):
    a = dict(x=16, ld_x=8, x_scales=None, ld_xs=0, packed=16, scales=16, N=2, H=8, V=8, softcap_T=0.0, multiplier=1.0,
             logits=16, ld_logits=8, stream=0, x_dtype=0, dtype=0, workspace=256, workspace_bytes=0)
    a.update(kw)   # no workspace bytes: refused last
    return L.flce_logits_mx(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=3), L.FLCE_EINVAL), (dict(dtype=2), L.FLCE_EINVAL), (dict(dtype=-1), L.FLCE_EINVAL),
    (dict(N=-1), L.FLCE_EINVAL), (dict(H=0), L.FLCE_EINVAL), (dict(V=0), L.FLCE_EINVAL),
    (dict(softcap_T=float("nan")), L.FLCE_EINVAL), (dict(softcap_T=float("inf")), L.FLCE_EINVAL),
    (dict(softcap_T=1e-45), L.FLCE_EINVAL), (dict(softcap_T=1e-30, multiplier=1e10), L.FLCE_EINVAL),
    (dict(multiplier=float("inf")), L.FLCE_EINVAL), (dict(N=(1 << 20) + 1), L.FLCE_EUNSUPPORTED),
    (dict(V=(1 << 24) + 1), L.FLCE_EUNSUPPORTED), (dict(H=(1 << 21) + 1), L.FLCE_EUNSUPPORTED),
    (dict(x=None), L.FLCE_EINVAL), (dict(packed=None), L.FLCE_EINVAL), (dict(scales=None), L.FLCE_EINVAL),
    (dict(logits=None), L.FLCE_EINVAL), (dict(x_scales=16), L.FLCE_EINVAL), (dict(x_dtype=2), L.FLCE_EINVAL),
    (dict(x=17), L.FLCE_EINVAL), (dict(x=18, x_dtype=1), L.FLCE_EINVAL), (dict(packed=24), L.FLCE_EINVAL),
    (dict(logits=17), L.FLCE_EINVAL), (dict(logits=18, dtype=1), L.FLCE_EINVAL), (dict(ld_x=-1), L.FLCE_EINVAL),
    (dict(x_dtype=2, x_scales=16, ld_xs=-1), L.FLCE_EINVAL), (dict(ld_logits=7), L.FLCE_EINVAL),
    (dict(scales=18), L.FLCE_EINVAL), (dict(workspace=None), L.FLCE_EINVAL), (dict(workspace=128), L.FLCE_EINVAL),
    (dict(N=1 << 20, H=1 << 20), L.FLCE_EUNSUPPORTED), (dict(), L.FLCE_EWORKSPACE),
    (dict(N=1 << 18, V=(1 << 17) + 1), L.FLCE_EUNSUPPORTED),
    (dict(N=0, x=None, logits=None), L.FLCE_OK),
])
def test_logits_reject_before_launch(kw, code):
    assert _logits(**kw) == code


def test_workspace_size():
    for N, H, dt in [(1, 1, 0), (320, 4096, 0), (33, 1001, 1), (5, 7168, 2), (0, 8, 0), (1 << 20, 128, 0)]:
        b = L.flce_logits_mx_workspace_size(N, H, dt)
        assert b >= 256 and b % 256 == 0 and b >= N * H * (2, 5, 1)[dt]   # bytes of parts
    for bad in [(-1, 8, 0), (1, 0, 0), (1, 8, 3), ((1 << 20) + 1, 8, 0), (1, (1 << 21) + 1, 0)]:
        assert L.flce_logits_mx_workspace_size(*bad) == 0


def test_wrappers_refuse_bad_tensors():
    W = torch.zeros(8, 100)
    with pytest.raises(ValueError, match="GPU"):
        L.mx4_pack(W)
    with pytest.raises(TypeError):
        L.mx4_pack(W.half())
    q = L.Mx4Weight(torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 4, dtype=torch.uint8).view(
        torch.float8_e8m0fnu), 100)
    with pytest.raises(ValueError, match="GPU"):
        L.logits_mx4(torch.zeros(2, 100), q)
    with pytest.raises(TypeError):
        L.logits_mx4(torch.zeros(2, 100).half(), q)
    with pytest.raises(TypeError):
        L.logits_mx4(L.Mx8Rows(torch.zeros(2, 100), torch.zeros(2, 4)), q)
    from linear_cross_entropy_gemm_amd import mx
    mx._check_weight(q)
    for bad in (L.Mx4Weight(q.data, q.scales, 129), L.Mx4Weight(q.data[:, :63], q.scales, 100),
                L.Mx4Weight(q.data, q.scales[:7], 100), L.Mx4Weight(q.data, q.scales.view(torch.uint8), 100),
                L.Mx4Weight(q.data.int(), q.scales, 100)):
        with pytest.raises(ValueError, match="weight"):
            mx._check_weight(bad)
    x, u = torch.zeros(2, 100), torch.zeros(2)
    for kw in (dict(mx8=True), dict(norm="rms", mx8=True), dict(residual=x), dict(norm="none")):
        with pytest.raises(ValueError):
            L.lm_head_sample(x, W, u, None, **kw)
