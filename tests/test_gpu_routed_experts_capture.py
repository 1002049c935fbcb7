"""A whole differentiable step (norm, router, experts, a grouped product, their gradients) captured into a CUDA graph
and replayed with other values."""
import pytest
import torch

from tests import synthetic as syn
from tests.test_gpu_routed_experts import BF, layer_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,H,E,k,I", [(40, 256, 8, 2, 128), (300, 384, 12, 1, 256), (700, 4224, 6, 2, 256)])
def test_a_backward_pass_captured_and_replayed(cuda, M, H, E, k, I):
    from invariant_moe_gb300 import routed_experts as rx
    leaves = [t.requires_grad_() for t in layer_of(M, H, E, k, I, 150, cuda)]
    x, router, bias, w13, w2, nw, nb = leaves
    off = torch.linspace(0, M, E + 1, device=cuda).int()

    def step():
        for t in leaves:
            t.grad = None
        y = rx.moe_block(x, nw, nb, router, w13, w2, k, bias=bias)
        (y.float().square().sum() + rx.grouped_linear(x, w13, off).float().square().sum()).backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # its graph is gone before the capture begins
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    kept = [t.grad for t in leaves]
    for seed in (160, 161):
        with torch.no_grad():
            x.copy_(syn.normal((M, H), 1.0, seed, BF))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        step()
        assert all(torch.equal(a, t.grad) for a, t in zip(got, leaves))
