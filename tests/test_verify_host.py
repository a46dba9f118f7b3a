"""Refusals of draft verification: every bad call returns its error before
anything reaches the GPU (fake addresses, CPU)."""
import pytest

L = pytest.importorskip("linear_cross_entropy_gemm_amd")
torch = pytest.importorskip("torch")


# The base call is complete except for one refusal that is checked last (no
# workspace bytes), so no variant with fake addresses can reach a launch.
def _verify(prm=None, prm2=None, **kw):
    def params(d):
        p = L.flce_sample_params_t(temperature=1.0, top_p=1.0)
        for k, v in d.items():
            setattr(p, k, v)
        return p
    a = dict(target=16, ld_target=8, draft=16, ld_draft=8, draft_tokens=16, draft_lens=16, u=16, u_draw=16, B=2, K=3,
             V=8, params=params(prm or {}), draft_params=None if prm2 is None else params(prm2), tokens=16, accepted=16,
             logprobs=16, stream=0, dtype=0, workspace=256, workspace_bytes=0)
    a.update(kw)
    return L.flce_verify(*a.values())


@pytest.mark.parametrize("prm,kw,code", [
    ({}, dict(dtype=2), L.FLCE_EINVAL), ({}, dict(B=-1), L.FLCE_EINVAL), ({}, dict(K=-1), L.FLCE_EINVAL),
    ({}, dict(V=0), L.FLCE_EINVAL), ({}, dict(params=None), L.FLCE_EINVAL),
    (dict(temperature=-1.0), {}, L.FLCE_EINVAL), (dict(temperature=float("nan")), {}, L.FLCE_EINVAL),
    (dict(top_k=-1), {}, L.FLCE_EINVAL), (dict(top_p=0.0), {}, L.FLCE_EINVAL), (dict(top_p=1.5), {}, L.FLCE_EINVAL),
    (dict(min_p=-0.5), {}, L.FLCE_EINVAL), (dict(min_p=1.5), {}, L.FLCE_EINVAL),
    (dict(temperature_rows=18), {}, L.FLCE_EINVAL), (dict(top_k_rows=20), {}, L.FLCE_EINVAL),
    ({}, dict(target=None), L.FLCE_EINVAL), ({}, dict(target=17), L.FLCE_EINVAL), ({}, dict(draft=17), L.FLCE_EINVAL),
    ({}, dict(draft_tokens=None), L.FLCE_EINVAL), ({}, dict(draft_tokens=20), L.FLCE_EINVAL),
    ({}, dict(draft_lens=20), L.FLCE_EINVAL), ({}, dict(u=None), L.FLCE_EINVAL), ({}, dict(u=18), L.FLCE_EINVAL),
    ({}, dict(u_draw=None), L.FLCE_EINVAL), ({}, dict(u_draw=18), L.FLCE_EINVAL),
    ({}, dict(tokens=None), L.FLCE_EINVAL), ({}, dict(tokens=20), L.FLCE_EINVAL),
    ({}, dict(accepted=None), L.FLCE_EINVAL), ({}, dict(accepted=20), L.FLCE_EINVAL),
    ({}, dict(logprobs=18), L.FLCE_EINVAL), ({}, dict(workspace=None), L.FLCE_EINVAL),
    ({}, dict(workspace=128), L.FLCE_EINVAL), ({}, dict(ld_target=-1), L.FLCE_EINVAL),
    ({}, dict(ld_draft=-1), L.FLCE_EINVAL), ({}, dict(K=1025), L.FLCE_EUNSUPPORTED),
    ({}, dict(B=(1 << 21) + 1, K=0), L.FLCE_EUNSUPPORTED), ({}, dict(B=1 << 20, K=1), L.FLCE_EUNSUPPORTED),
    ({}, dict(V=(1 << 24) + 1), L.FLCE_EUNSUPPORTED), ({}, dict(B=4096, K=1, V=1 << 24), L.FLCE_EUNSUPPORTED),
    ({}, {}, L.FLCE_EWORKSPACE), ({}, dict(K=0, draft_tokens=None, u=None, draft=None), L.FLCE_EWORKSPACE),
    ({}, dict(B=0, target=None, draft=None, draft_tokens=None, u=None, u_draw=None, tokens=None, accepted=None,
              workspace=None), L.FLCE_OK),
])
def test_verify_rejects_before_launch(prm, kw, code):
    assert _verify(prm, **kw) == code


@pytest.mark.parametrize("prm2", [dict(temperature=-1.0), dict(top_p=0.0), dict(top_k=-3), dict(min_p_rows=17)])
def test_verify_rejects_the_drafts_parameters(prm2):
    assert _verify({}, prm2) == L.FLCE_EINVAL
    assert _verify({}, {}) == L.FLCE_EWORKSPACE


def test_verify_workspace_size():
    for B, K, V, dt, d in [(1, 4, 202048, 0, 1), (64, 4, 129279, 1, 1), (3, 0, 8, 0, 0), (0, 4, 8, 0, 1), (5, 7, 2048, 1, 0)]:
        b = L.flce_verify_workspace_size(B, K, V, dt, d)
        assert b >= 256 and b % 256 == 0
        assert b >= L.flce_sample_workspace_size(B * (2 * K + 1 if d else K + 1), V, dt)
    for bad in [(-1, 4, 8, 0, 1), (1, -1, 8, 0, 1), (1, 1, 0, 0, 1), (1, 1, 8, 2, 1), (1, 1025, 8, 0, 1),
                (1 << 20, 0, 1 << 16, 0, 0)]:
        assert L.flce_verify_workspace_size(*bad) == 0


def test_wrapper_refuses_bad_tensors():
    z = torch.zeros(2, 4, 8)
    x, u, ud = torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3), torch.zeros(2)
    with pytest.raises(ValueError, match="GPU"):
        L.verify(z, x, u, ud)
    with pytest.raises(TypeError):
        L.verify(z.half(), x, u, ud)
