"""Refusals of the operators around the projection: every bad call returns
its error before anything reaches the GPU (fake addresses, CPU)."""
import pytest

L = pytest.importorskip("linear_cross_entropy_gemm_amd")
torch = pytest.importorskip("torch")


# The base call of each helper is complete except for one refusal that is
# checked last, so no variant with fake addresses can reach a launch.
def _ln_fwd(**kw):
    a = dict(x=16, ld_x=8, weight=16, bias=16, M=2, H=8, eps=1e-5, y=16, ld_y=9, mean=16, rstd=16, stream=0, dtype=0,
             w_dtype=0)   # x == y with different strides: refused last
    a.update(kw)
    return L.flce_layer_norm_fwd(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), L.FLCE_EINVAL), (dict(w_dtype=-1), L.FLCE_EINVAL), (dict(M=-1), L.FLCE_EINVAL),
    (dict(H=0), L.FLCE_EINVAL), (dict(M=1 << 31), L.FLCE_EUNSUPPORTED), (dict(H=(1 << 21) + 1), L.FLCE_EUNSUPPORTED),
    (dict(eps=0.0), L.FLCE_EINVAL), (dict(eps=-1.0), L.FLCE_EINVAL), (dict(eps=float("nan")), L.FLCE_EINVAL),
    (dict(eps=float("inf")), L.FLCE_EINVAL), (dict(x=None), L.FLCE_EINVAL), (dict(y=None), L.FLCE_EINVAL),
    (dict(x=17), L.FLCE_EINVAL), (dict(y=17), L.FLCE_EINVAL), (dict(weight=17), L.FLCE_EINVAL),
    (dict(bias=18, w_dtype=1), L.FLCE_EINVAL), (dict(mean=18), L.FLCE_EINVAL), (dict(rstd=18), L.FLCE_EINVAL),
    (dict(ld_x=-1), L.FLCE_EINVAL), (dict(ld_y=7), L.FLCE_EINVAL), (dict(), L.FLCE_EINVAL),
    (dict(M=0, x=None, y=None), L.FLCE_OK),
])
def test_layer_norm_fwd_rejects_before_launch(kw, code):
    assert _ln_fwd(**kw) == code


def _ln_bwd(**kw):
    a = dict(grad_y=16, ld_gy=8, x=32, ld_x=8, weight=16, mean=16, rstd=16, M=2, H=8, grad_x=64, ld_gx=8,
             grad_weight=16, grad_bias=16, stream=0, dtype=0, w_dtype=0, workspace=256, workspace_bytes=0)
    a.update(kw)
    return L.flce_layer_norm_bwd(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), L.FLCE_EINVAL), (dict(w_dtype=2), L.FLCE_EINVAL), (dict(M=-1), L.FLCE_EINVAL),
    (dict(H=0), L.FLCE_EINVAL), (dict(H=(1 << 21) + 1), L.FLCE_EUNSUPPORTED),
    (dict(grad_y=None), L.FLCE_EINVAL), (dict(x=None), L.FLCE_EINVAL), (dict(mean=None), L.FLCE_EINVAL),
    (dict(rstd=None), L.FLCE_EINVAL), (dict(grad_y=17), L.FLCE_EINVAL), (dict(x=33), L.FLCE_EINVAL),
    (dict(grad_x=65), L.FLCE_EINVAL), (dict(weight=17), L.FLCE_EINVAL), (dict(grad_weight=17), L.FLCE_EINVAL),
    (dict(grad_bias=17), L.FLCE_EINVAL), (dict(mean=18), L.FLCE_EINVAL), (dict(ld_gy=-1), L.FLCE_EINVAL),
    (dict(ld_x=-1), L.FLCE_EINVAL), (dict(ld_gx=7), L.FLCE_EINVAL), (dict(grad_x=16), L.FLCE_EINVAL),
    (dict(grad_x=32), L.FLCE_EINVAL), (dict(workspace=None), L.FLCE_EINVAL), (dict(workspace=128), L.FLCE_EINVAL),
    (dict(), L.FLCE_EWORKSPACE),
    (dict(M=0, grad_weight=None, grad_bias=None), L.FLCE_OK),
])
def test_layer_norm_bwd_rejects_before_launch(kw, code):
    assert _ln_bwd(**kw) == code


def test_layer_norm_bwd_workspace_size():
    for M, H, dt in [(1, 1, 0), (8192, 6656, 0), (4099, 5003, 1), (100000, 64, 0), (3, 1 << 21, 1), (0, 8, 0)]:
        b = L.flce_layer_norm_bwd_workspace_size(M, H, dt)
        # at least one partial of both gradients, at most 1024 of them
        assert b % 256 == 0 and 8 * H <= b <= 1024 * 8 * H + 256
    assert L.flce_layer_norm_bwd_workspace_size(-1, 8, 0) == 0
    assert L.flce_layer_norm_bwd_workspace_size(1, (1 << 21) + 1, 0) == 0
    assert L.flce_layer_norm_bwd_workspace_size(1, 8, 3) == 0


def _drop(**kw):
    a = dict(x=16, residual=None, y=18, n=8, p=0.5, seed=1, offset=0, offset_dev=None, stream=0, dtype=0)
    a.update(kw)     # y overlaps x partly: refused last
    return L.flce_dropout(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), L.FLCE_EINVAL), (dict(n=-1), L.FLCE_EINVAL), (dict(p=-0.1), L.FLCE_EINVAL),
    (dict(p=1.0000001), L.FLCE_EINVAL), (dict(p=float("nan")), L.FLCE_EINVAL), (dict(x=None), L.FLCE_EINVAL),
    (dict(y=None), L.FLCE_EINVAL), (dict(x=17), L.FLCE_EINVAL), (dict(y=19), L.FLCE_EINVAL),
    (dict(residual=33), L.FLCE_EINVAL), (dict(offset_dev=12), L.FLCE_EINVAL), (dict(), L.FLCE_EINVAL),
    (dict(n=(1 << 33) + 1), L.FLCE_EUNSUPPORTED),
    (dict(y=16, residual=18), L.FLCE_EINVAL), (dict(n=0, x=None, y=None), L.FLCE_OK),
])
def test_dropout_rejects_before_launch(kw, code):
    assert _drop(**kw) == code


def test_wrappers_refuse_bad_tensors():
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    for f in (lambda: L.layer_norm_fwd(x), lambda: L.layer_norm(x), lambda: L.dropout(x, 0.5, 1),
              lambda: L.layer_norm_bwd(x, x, None, x, x)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    for f in (lambda: L.layer_norm_fwd(x.half()), lambda: L.dropout(x.long(), 0.5, 1)):
        with pytest.raises(TypeError):
            f()


def _sample(prm=None, rows=None, **kw):
    p = L.flce_sample_params_t(temperature=1.0, top_p=1.0)
    for k, v in (prm or {}).items():
        setattr(p, k, v)
    a = dict(logits=16, ld=8, u=16, N=2, V=8, params=p, tokens=16, logprobs=16, stream=0, dtype=0, workspace=256,
             workspace_bytes=0)   # no workspace bytes: refused last
    a.update(kw)
    return L.flce_sample(*a.values())


@pytest.mark.parametrize("prm,kw,code", [
    ({}, dict(dtype=2), L.FLCE_EINVAL), ({}, dict(N=-1), L.FLCE_EINVAL), ({}, dict(V=0), L.FLCE_EINVAL),
    ({}, dict(params=None), L.FLCE_EINVAL), (dict(temperature=-1.0), {}, L.FLCE_EINVAL),
    (dict(temperature=float("nan")), {}, L.FLCE_EINVAL), (dict(temperature=float("inf")), {}, L.FLCE_EINVAL),
    (dict(top_k=-1), {}, L.FLCE_EINVAL), (dict(top_p=0.0), {}, L.FLCE_EINVAL), (dict(top_p=1.5), {}, L.FLCE_EINVAL),
    (dict(top_p=float("nan")), {}, L.FLCE_EINVAL), (dict(min_p=-0.5), {}, L.FLCE_EINVAL),
    (dict(min_p=1.5), {}, L.FLCE_EINVAL), (dict(temperature_rows=18), {}, L.FLCE_EINVAL),
    (dict(top_k_rows=20), {}, L.FLCE_EINVAL), (dict(top_p_rows=18), {}, L.FLCE_EINVAL),
    (dict(min_p_rows=18), {}, L.FLCE_EINVAL), ({}, dict(logits=None), L.FLCE_EINVAL),
    ({}, dict(u=None), L.FLCE_EINVAL), ({}, dict(tokens=None), L.FLCE_EINVAL),
    ({}, dict(workspace=None), L.FLCE_EINVAL), ({}, dict(logits=17), L.FLCE_EINVAL),
    ({}, dict(logits=18, dtype=1), L.FLCE_EINVAL), ({}, dict(u=18), L.FLCE_EINVAL),
    ({}, dict(tokens=20), L.FLCE_EINVAL), ({}, dict(logprobs=18), L.FLCE_EINVAL),
    ({}, dict(workspace=128), L.FLCE_EINVAL), ({}, dict(ld=-1), L.FLCE_EINVAL),
    ({}, dict(N=(1 << 21) + 1), L.FLCE_EUNSUPPORTED), ({}, dict(V=(1 << 24) + 1), L.FLCE_EUNSUPPORTED),
    ({}, dict(N=1 << 20, V=1 << 20), L.FLCE_EUNSUPPORTED), ({}, {}, L.FLCE_EWORKSPACE), ({}, dict(N=0, logits=None, u=None, tokens=None, workspace=None), L.FLCE_OK),
])
def test_sample_rejects_before_launch(prm, kw, code):
    assert _sample(prm, **kw) == code


def test_sample_workspace_size():
    for N, V, dt in [(1, 1, 0), (64, 129280, 1), (256, 202048, 0), (0, 8, 0), (0, 1 << 20, 0), (1 << 21, 8, 1), (1, 1 << 24, 0)]:
        b = L.flce_sample_workspace_size(N, V, dt)
        assert b >= 256 and b % 256 == 0
    assert L.flce_sample_workspace_size(-1, 8, 0) == 0 and L.flce_sample_workspace_size(1, 0, 0) == 0
    assert L.flce_sample_workspace_size(1, 8, 2) == 0 and L.flce_sample_workspace_size(1, (1 << 24) + 1, 0) == 0


def _identity():
    """A differentiable identity with the package's notes and checks, on the CPU."""
    from linear_cross_entropy_gemm_amd import torch_api

    class F(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, b, n):
            return a * 1

        @staticmethod
        def backward(ctx, g):
            torch_api.check_leaves(ctx, g)
            return g, None, None

    def call(x):
        y = F.apply(x, None, 3)
        torch_api.note_leaves(y)
        return y
    return call


def test_captured_backward_is_refused_beside_a_live_graph_of_another_stream(monkeypatch):
    """The streams and the capture are played by stand-ins: a leaf whose graph
    from stream 1 is alive refuses a backward pass captured on stream 2, and
    is accepted uncaptured, on stream 1, and once that graph is gone."""
    import gc
    import types
    state = {"stream": 1, "capturing": False}
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda dev=None: types.SimpleNamespace(cuda_stream=state["stream"]))
    f = _identity()
    x, one = torch.ones(3, requires_grad=True), torch.ones(3)

    def grad():
        return torch.autograd.grad(f(x), x, one)[0]

    alive = f(x)
    assert torch.equal(grad(), one)
    state.update(stream=2)
    assert torch.equal(grad(), one)
    state.update(capturing=True)
    with pytest.raises(RuntimeError, match="cannot be captured"):
        grad()
    state.update(stream=1)
    assert torch.equal(grad(), one)
    state.update(stream=2)
    del alive
    gc.collect()
    assert torch.equal(grad(), one)
    assert torch.equal(torch.autograd.grad(f(f(x)), x, one)[0], one)   # a node in between has no mark


@pytest.mark.parametrize("k", [-(1 << 63) - 1, 1 << 63, (1 << 64) + 5])
def test_top_k_outside_the_parameter_block_is_refused(k):
    from linear_cross_entropy_gemm_amd import head
    prm = L.flce_sample_params_t()
    with pytest.raises(ValueError):
        head._sample_param("top_k", k, torch.int64, 1, torch.device("cpu"), prm)
    with pytest.raises(TypeError):
        head._sample_param("top_k", 2.5, torch.int64, 1, torch.device("cpu"), prm)
    head._sample_param("top_k", (1 << 63) - 1, torch.int64, 1, torch.device("cpu"), prm)
    assert prm.top_k == (1 << 63) - 1
