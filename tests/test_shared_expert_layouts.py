"""gated_ffn's second derivatives where an input has to be copied first (no GPU: see
tests/test_shared_expert_host.py)."""
import pytest
import torch

from invariant_moe_gb300 import shared_expert as se
from tests import ffn_reference as ref
from tests.test_shared_expert_host import BF, aligned, formulas, make  # noqa: F401

VIEWS = {"as_it_lies": aligned, "transposed": lambda t: t.t().contiguous().t(),
         "inside": lambda t: torch.cat((t[:, :4], t, t[:, :3]), 1)[:, 4:4 + t.shape[1]]}


@pytest.mark.parametrize("view", list(VIEWS))
@pytest.mark.parametrize("with_addend", [False, True])
def test_second_order_is_refused_in_every_layout(formulas, view, with_addend):
    """dout is a constant and x the only differentiable argument: dx depends on x all the same."""
    x, w13, w2, add = [aligned(t) for t in make(4)]
    x = VIEWS[view](x).detach().requires_grad_()
    out = se.gated_ffn(x, w13, w2, VIEWS[view](add) if with_addend else None)
    (g,) = torch.autograd.grad(out.sum(), x, create_graph=True)
    assert g.requires_grad
    with pytest.raises(RuntimeError, match="second"):
        (g.float().square().sum() + x.float().sum()).backward()


@pytest.mark.parametrize("view", list(VIEWS))
def test_gradients_in_every_layout(formulas, view):
    x, w13, w2, add = [aligned(t) for t in make(5)]
    v = [VIEWS[view](t).detach().requires_grad_() for t in (x, add)]
    w = [t.clone().requires_grad_() for t in (w13, w2)]
    dout = aligned(make(6)[3])
    se.gated_ffn(v[0], *w, v[1]).backward(dout)
    r = ref.ffn(x, w13, w2, dout=dout)
    for t, want in ((v[0], r["dx"]), (w[0], r["dw13"]), (w[1], r["dw2"]), (v[1], dout)):
        assert t.grad.shape == t.shape and torch.equal(t.grad, want.to(BF))
