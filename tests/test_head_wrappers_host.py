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


class _OnGpu(torch.Tensor):
    """A CPU tensor that says it is on the GPU."""
    is_cuda = property(lambda self: True)


def _on_gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnGpu)


@pytest.mark.parametrize("kind", ["logits", "lm_head_sample", "linear_cross_entropy", "lm_head_loss", "fwd_bwd",
                                  "forward"])
def test_a_projection_of_another_width_never_reaches_the_kernels(kind, monkeypatch):
    """The kernels read H columns of each row of W: one with fewer, or one that
    is not on the GPU of the hidden states, would be read past its end."""
    from linear_cross_entropy_gemm_amd import torch_api
    calls = []
    _stand_ins(monkeypatch)
    monkeypatch.setattr(torch_api, "_enqueue", lambda dev, call: call(0))
    for name in ("flce_logits", "flce_fwd", "flce_fwd_bwd_ex", "flce_sample"):
        monkeypatch.setattr(torch_api._lib, name, lambda *a, _n=name: calls.append(_n) or 0)
    monkeypatch.setattr(head, "_layer_norm_fwd", lambda x, w, b, eps, stats: (x, None, None))
    x, u, lab = _on_gpu(3, 8), _on_gpu(3), _on_gpu(3, dtype=torch.int64)
    call = {"logits": lambda W: L.logits(x, W), "lm_head_sample": lambda W: L.lm_head_sample(x, W, u, None),
            "linear_cross_entropy": lambda W: L.linear_cross_entropy(x, W, lab),
            "lm_head_loss": lambda W: L.lm_head_loss(x, W, lab, None),
            "fwd_bwd": lambda W: L.fwd_bwd(x, W, lab), "forward": lambda W: L.forward(x, W, lab)}[kind]
    for W in (_on_gpu(20, 7), _on_gpu(20, 9), _on_gpu(20), _on_gpu(2, 20, 8), torch.zeros(20, 8)):
        with pytest.raises(ValueError):
            call(W)
    if kind == "logits":
        for out in (_on_gpu(3, 20, dtype=torch.bfloat16), _on_gpu(3, 16), _on_gpu(2, 20), _on_gpu(60)):
            with pytest.raises(ValueError):
                L.logits(x, _on_gpu(20, 8), out=out)
        assert not calls
        L.logits(x, _on_gpu(20, 8), out=_on_gpu(3, 24))
        assert calls == ["flce_logits"]
    else:
        assert not calls


def test_launches_go_to_the_tensors_device(monkeypatch):
    """The default stream's handle is 0 on every device: a launch on it runs on
    the current one, so that has to be the tensors' own."""
    from linear_cross_entropy_gemm_amd import torch_api
    now = [0]

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            now.append(self.dev.index)

        def __exit__(self, *a):
            now.pop()

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    for i in (0, 1):
        assert torch_api._enqueue(torch.device("cuda", i), lambda s: (s, now[-1])) == (100 + i, i)
    assert now == [0]


@pytest.mark.parametrize("kind", ["fwd_bwd", "forward", "logits", "cross_entropy", "scale_grads", "read_status"])
def test_every_launch_of_the_projection_goes_to_the_tensors_device(kind, monkeypatch):
    from linear_cross_entropy_gemm_amd import torch_api
    inside, seen = [], []

    def enqueue(dev, call):
        inside.append(dev)
        rc = call(7)
        inside.pop()
        return rc

    monkeypatch.setattr(torch_api, "_enqueue", enqueue)
    names = ("flce_logits", "flce_fwd", "flce_fwd_bwd_ex", "flce_cross_entropy", "flce_scale_grads", "flce_read_status")
    for name in names:
        monkeypatch.setattr(torch_api._lib, name, lambda *a, _n=name: seen.append((_n, bool(inside))) or 0)
    x, W, lab = _on_gpu(3, 8), _on_gpu(20, 8), _on_gpu(3, dtype=torch.int64)
    {"fwd_bwd": lambda: L.fwd_bwd(x, W, lab), "forward": lambda: L.forward(x, W, lab),
     "logits": lambda: L.logits(x, W), "cross_entropy": lambda: L.cross_entropy(_on_gpu(3, 20), lab, grad=True),
     "scale_grads": lambda: torch_api.scale_grads(torch.ones(()), x, W, torch.float32),
     "read_status": lambda: L.read_status(torch.zeros(8, dtype=torch.uint8))}[kind]()
    assert seen and all(ok for _, ok in seen), seen


def test_cross_entropy_of_too_few_labels_never_reaches_the_kernels(monkeypatch):
    """One label (and one upstream gradient) is read per row of the logits."""
    from linear_cross_entropy_gemm_amd import torch_api
    calls = []
    monkeypatch.setattr(torch_api, "_enqueue", lambda dev, call: call(0))
    monkeypatch.setattr(torch_api._lib, "flce_cross_entropy", lambda *a: calls.append(a) or 0)
    monkeypatch.setattr(torch_api._lib, "flce_read_status", lambda *a: 0)
    z, lab = _on_gpu(3, 20), _on_gpu(3, dtype=torch.int64)
    for kw in (dict(labels=lab[:2]), dict(labels=_on_gpu(4, dtype=torch.int64)),
               dict(labels=torch.zeros(3, dtype=torch.int64)), dict(z=torch.zeros(3, 20)),
               dict(grad=True, reduction="none", grad_rows=_on_gpu(2))):
        with pytest.raises(ValueError):
            L.cross_entropy(**{"z": z, "labels": lab, **kw})
    assert not calls
    L.cross_entropy(z, lab, grad=True, reduction="none", grad_rows=_on_gpu(3))
    assert len(calls) == 1
