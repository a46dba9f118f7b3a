"""Whole training steps of the head captured after a warm-up on a side stream
whose last loss is still alive, replayed with eager work in between."""
import pytest

from gpu_util import log

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("require_gpu")]


@pytest.mark.parametrize("path", ["linear_cross_entropy", "lm_head_loss"])
def test_step_is_captured_beside_the_warm_up_of_a_side_stream(path):
    import torch
    import linear_cross_entropy_gemm_amd as L
    g = torch.Generator().manual_seed(3)
    N, H, V = 96, 320, 700
    x = torch.randn(N, H, generator=g).bfloat16().cuda().requires_grad_()
    W = (torch.randn(V, H, generator=g) * 0.1).bfloat16().cuda().requires_grad_()
    w = (1 + 0.2 * torch.randn(H, generator=g)).cuda().requires_grad_()
    lab = torch.randint(0, V, (N,), generator=g).cuda()
    leaves = (x, W) if path == "linear_cross_entropy" else (x, W, w)

    def step():
        for t in leaves:
            t.grad = None
        if path == "linear_cross_entropy":
            loss, _ = L.linear_cross_entropy(x, W, lab)
        else:
            loss, _ = L.lm_head_loss(x, W, lab, w, dropout_p=0.1, seed=5)
        loss.backward()
        return loss

    side = torch.cuda.Stream()
    assert side.stream_id % 2 == 1 and torch.cuda.default_stream().stream_id == 0
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            alive = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    log(f"[capture] {path}: warm-up done, its loss alive")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step()
    torch.cuda.synchronize()
    log(f"[capture] {path}: captured")
    grads = [t.grad for t in leaves]
    for rep in range(4):
        with torch.no_grad():
            x.mul_(0.9)
            W.mul_(1.1)
        for t in (loss.detach(), *grads):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [loss.detach().clone(), *(t.clone() for t in grads)]
        with torch.cuda.stream(side):   # the program's own eager work between replays
            want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (want.detach(), *(t.grad for t in leaves)))), rep
    assert alive.grad_fn is not None
