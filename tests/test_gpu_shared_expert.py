"""The shared expert as it is used: differentiable block, beside the routed
experts, and in 4 bits (invariant_moe_gb300.shared_expert) on a GPU."""
import pytest
import torch

from tests import ffn_reference as ref
from tests import synthetic as syn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def make(M, H, I, seed, dev):
    return (syn.normal((M, H), 1.0, seed, BF).to(dev), syn.normal((2 * I, H), H ** -0.5, seed + 1, BF).to(dev),
            syn.normal((H, I), I ** -0.5, seed + 2, BF).to(dev))


def test_autograd(cuda):
    """The block inside a larger expression: gradients of every argument, views and shared uses among them."""
    from invariant_moe_gb300.shared_expert import gated_ffn
    M, H, I = 45, 160, 96
    x, w13, w2 = make(M, H, I, 1, cuda)
    add = syn.normal((M, H), 0.5, 4, BF).to(cuda)
    wide = torch.zeros(M, H + 32, dtype=BF, device=cuda)
    wide[:, 16:16 + H] = x
    leaves = [t.requires_grad_() for t in (wide, w13, w2, add)]
    out = gated_ffn(wide[:, 16:16 + H], w13, w2, add)
    out.sum().backward()  # an expanded gradient
    r = ref.ffn(x.cpu(), w13.detach().cpu(), w2.detach().cpu(), add.detach().cpu(), torch.ones(M, H))
    assert ref.rel_norm(out.detach().cpu(), r["out"]) <= ref.norm_bound(2)
    assert ref.rel_norm(leaves[0].grad[:, 16:16 + H].cpu(), r["dx"]) <= ref.norm_bound(2)
    assert not leaves[0].grad[:, :16].any() and not leaves[0].grad[:, 16 + H:].any()
    assert ref.rel_norm(leaves[1].grad.cpu(), r["dw13"]) <= ref.norm_bound(2)
    assert ref.rel_norm(leaves[2].grad.cpu(), r["dw2"]) <= ref.norm_bound(2)
    assert torch.equal(leaves[3].grad, torch.ones_like(add))
    with torch.no_grad():
        assert torch.equal(gated_ffn(wide[:, 16:16 + H], w13, w2, add), out)
    # only one gradient asked for
    w2b = w2.detach().clone().requires_grad_()
    gated_ffn(x.detach(), w13.detach(), w2b).sum().backward()
    assert torch.equal(w2b.grad, leaves[2].grad)


def test_beside_the_routed_experts(cuda):
    import invariant_moe_gb300 as bm
    from invariant_moe_gb300.shared_expert import moe_layer_with_shared_expert
    M, H, E, I, k = 150, 256, 16, 128, 4
    w = syn.moe_weights(H, E, I, seed=11, unit=True)
    dev = [t.to(cuda) for t in (w.w_router, w.w13, w.w2)]
    x, s13, s2 = make(M, H, I, 12, cuda)
    out, _, ids, wts = moe_layer_with_shared_expert(x, dev[0], dev[1], dev[2], k, s13, s2)
    base, _, ids2, _ = bm.moe_layer(x, dev[0], dev[1], dev[2], k)
    assert torch.equal(ids, ids2)
    assert torch.equal(out, bm.bi_ffn_forward(x, s13, s2, addend=base))
    r = ref.ffn(x.cpu(), s13.cpu(), s2.cpu(), base.cpu())
    assert ref.rel_norm(out.cpu(), r["out"]) <= ref.norm_bound(2)
    for a, n in ((0, 1), (7, 3), (20, 64), (5, 140)):
        o = moe_layer_with_shared_expert(x[a:a + n], dev[0], dev[1], dev[2], k, s13, s2)[0]
        assert torch.equal(o, out[a:a + n])


def test_in_four_bits(cuda):
    """Each step of the 4-bit expert against the 64-bit product of what its operands stand for."""
    import invariant_moe_gb300 as bm
    from invariant_moe_gb300.shared_expert import Mx4SharedExpert
    M, H, I = 70, 288, 160
    x, w13, w2 = make(M, H, I, 21, cuda)
    add = syn.normal((M, H), 0.5, 24, BF).to(cuda)
    e = Mx4SharedExpert(w13, w2)
    out = e(x, addend=add)

    def values(q, s):
        return bm.bi_mx4_dequantize(q, s, dtype=torch.float32).double().cpu()

    act, _ = ref.mx4_gated(values(*bm.bi_mx4_quantize(x)), values(e.w13, e.s13))
    got = bm.bi_mx4_gate_up(*bm.bi_mx4_quantize(x), e.w13, e.s13)
    assert ref.rel_norm(got.cpu(), act) <= ref.norm_bound(1)
    want, _ = ref.mx4_product(values(*bm.bi_mx4_quantize(got)), values(e.w2, e.s2), add.cpu())
    assert ref.rel_norm(out.cpu(), want) <= ref.norm_bound(1)
    for a, n in ((0, 1), (3, 17), (1, 64)):
        assert torch.equal(e(x[a:a + n], addend=add[a:a + n]), out[a:a + n])
    with pytest.raises(ValueError):
        Mx4SharedExpert(w13[:, :280], w2[:280])


def test_example_runs(cuda, capsys):
    from invariant_moe_gb300 import shared_expert
    shared_expert.main()
    text = capsys.readouterr().out
    losses = [float(line.split()[-1]) for line in text.splitlines() if line.startswith("step")]
    assert losses[-1] < 0.2 * losses[0]
    assert "bit for bit: True" in text


@pytest.mark.parametrize("how", ["sum_rows", "cat", "transposed"])
def test_gradients_of_any_layout(cuda, how):
    """Expanded, misaligned and transposed gradients give the bits of the same gradient laid out plainly."""
    from invariant_moe_gb300.shared_expert import gated_ffn
    M, H, I = 45, 160, 96
    v = syn.normal((H,), 1.0, 41, BF).to(cuda)

    def reduce(o):
        if how == "sum_rows":
            return (o.sum(0) * v).sum()
        if how == "cat":
            z = torch.zeros(M, 4, dtype=BF, device=cuda)
            return (torch.cat((z, o, z), 1) * torch.cat((v[:4], v, v[:4]))).sum()
        return (o.t().contiguous() * v[:, None]).sum()

    leaves = [t.requires_grad_() for t in make(M, H, I, 31, cuda)]
    reduce(gated_ffn(*leaves)).backward()
    got = [t.grad.clone() for t in leaves]
    for t in leaves:
        t.grad = None
    gated_ffn(*leaves).backward(v.expand(M, H).contiguous())
    for a, t in zip(got, leaves):
        assert torch.equal(a, t.grad)


def test_second_order_is_refused(cuda):
    """A gradient penalty raises; the first-order gradients of a graph that was asked for have their bits."""
    from invariant_moe_gb300.shared_expert import gated_ffn
    leaves = [t.requires_grad_() for t in make(37, 144, 112, 51, cuda)]
    out = gated_ffn(*leaves)
    grads = torch.autograd.grad(out.sum(), leaves, create_graph=True)
    want = torch.autograd.grad(gated_ffn(*leaves).sum(), leaves)
    for t, g, w in zip(leaves, grads, want):
        assert torch.equal(g, w) and g.requires_grad
        with pytest.raises(RuntimeError, match="second"):
            torch.autograd.grad(g.float().square().sum(), t, retain_graph=True)
