"""The torch wrappers around the head's operators where no GPU is needed: the
calls of the library are played by stand-ins."""
import pytest

L = pytest.importorskip("linear_cross_entropy_gemm_amd")
torch = pytest.importorskip("torch")

from linear_cross_entropy_gemm_amd import head  # noqa: E402


def _stand_ins(monkeypatch):
    """layer_norm and dropout without their kernels: plain copies, as far as
    autograd can see (an operator's output comes from outside of torch)."""
    def copy(x):
        y = torch.empty(x.shape)
        y.detach().numpy()[...] = x.detach().numpy()
        return y
    monkeypatch.setattr(head, "_check_tensor", lambda name, x: None)
    monkeypatch.setattr(head, "_layer_norm_fwd", lambda x, w, b, eps, stats: (copy(x), torch.ones(3), torch.ones(3)))
    monkeypatch.setattr(head, "_dropout", lambda x, p, seed, offset, residual: copy(x))


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("grad_mode", [False, True])
@pytest.mark.parametrize("where", ["x", "weight", "bias", "dropout", "residual", "lm_head_loss"])
def test_forward_mode_tangents_are_refused_not_dropped(where, grad_mode, grad, monkeypatch):
    import torch.autograd.forward_ad as fw
    _stand_ins(monkeypatch)
    x, w, b, r = torch.randn(3, 4), torch.randn(4), torch.randn(4), torch.randn(3, 4)
    calls = {
        "x": (x, lambda d: L.layer_norm(d, w, b)),
        "weight": (w, lambda d: L.layer_norm(x, d, b)),
        "bias": (b, lambda d: L.layer_norm(x, w, d)),
        "dropout": (x, lambda d: L.dropout(d, 0.5, 1)),
        "residual": (r, lambda d: L.dropout(x, 0.5, 1, residual=d)),
        "lm_head_loss": (x, lambda d: L.lm_head_loss(d, torch.randn(5, 4), torch.zeros(3, dtype=torch.int64), w, b)),
    }
    t, call = calls[where]
    with fw.dual_level(), torch.set_grad_enabled(grad_mode):
        d = fw.make_dual(t.clone().requires_grad_(grad), torch.ones_like(t))
        with pytest.raises(NotImplementedError, match="jvp"):
            call(d)
        # tensors without a tangent are none of this
        assert torch.equal(L.layer_norm(x, w, b), x) and torch.equal(L.dropout(x, 0.5, 1, residual=r), x)
    assert torch.equal(L.layer_norm(x, w, b), x) and torch.equal(L.dropout(x, 0.5, 1), x)


def test_a_tangent_of_the_upstream_gradient_is_refused(monkeypatch):
    import torch.autograd.forward_ad as fw
    from linear_cross_entropy_gemm_amd import torch_api
    _stand_ins(monkeypatch)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(head, "layer_norm_bwd", lambda g, x, *a, **k: L.LayerNormGrads(x * 1, None, None))
    monkeypatch.setattr(torch_api, "fwd_bwd", lambda h, W, *a, **k: L.FlceOutputs(
        torch.zeros(()), torch.zeros_like(h), torch.zeros_like(W), torch.zeros((), dtype=torch.int64), None))
    monkeypatch.setattr(torch_api, "scale_grads", lambda g, gh, gW, d: (gh, gW))
    monkeypatch.setattr(torch_api, "note_leaves", lambda out: None)
    monkeypatch.setattr(head, "note_leaves", lambda out: None)
    x = torch.randn(3, 4, requires_grad=True)
    for y in (L.layer_norm(x), L.dropout(x, 0.5, 1),
              L.linear_cross_entropy(x, torch.randn(5, 4), torch.zeros(3, dtype=torch.int64))[0]):
        one = torch.ones_like(y)
        with fw.dual_level():
            with pytest.raises(NotImplementedError, match="jvp"):
                torch.autograd.grad(y, x, fw.make_dual(one, one), retain_graph=True)
            torch.autograd.grad(y, x, one)


def test_captured_backward_beside_live_graphs_of_each_kind_of_stream(monkeypatch):
    """A warm-up's graph from a side stream of torch's own pool (odd ids) may be
    alive when a backward pass is captured on another; one from the default
    stream (id 0) or a foreign stream (its address, even) may not."""
    import types
    from test_head_host import _identity
    now = {}
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(
        cuda_stream=now["handle"], stream_id=now["id"]))
    f, one = _identity(), torch.ones(3)
    for warm, ident, refused in ((0x1000, 33, False), (0, 0, True), (0x2000, 0x2000, True)):
        x = torch.ones(3, requires_grad=True)
        now.update(handle=warm, id=ident, capturing=False)
        alive = f(x)
        alive.backward(one, retain_graph=True)
        now.update(handle=0x3000, id=65, capturing=True)
        y = f(x)
        if refused:
            with pytest.raises(RuntimeError, match="cannot be captured"):
                torch.autograd.grad(y, x, one)
        else:
            assert torch.equal(torch.autograd.grad(y, x, one)[0], one)
        del alive
