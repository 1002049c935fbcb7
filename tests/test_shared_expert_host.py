"""gated_ffn's handling of autograd (no GPU): the library's calls are replaced by
their formulas, with the library's own rules for row strides and alignment."""
import pytest
import torch

from invariant_moe_gb300 import shared_expert as se
from tests import ffn_reference as ref

BF = torch.bfloat16
M, H, I = 6, 32, 16


def check_rows(t):
    """What the library asks of a token matrix."""
    if t.shape[0] > 1 and (t.stride(1) != 1 or t.stride(0) % 8 or t.stride(0) < t.shape[1]):
        raise RuntimeError(f"row strides {t.stride()}")
    if t.data_ptr() % 16:
        raise RuntimeError("alignment")


@pytest.fixture
def formulas(monkeypatch):
    def forward_train(x, w13, w2, addend=None):
        check_rows(x)
        if addend is not None:
            check_rows(addend)
        r = ref.ffn(x, w13, w2, addend)
        return r["out"].to(BF), torch.cat((r["g"], r["u"]), 1).float(), r["act"].to(BF)

    def backward(dout, x, w13, w2, gu, act, need=(True, True, True)):
        check_rows(dout)
        check_rows(x)
        r = ref.ffn(x, w13, w2, dout=dout)
        return tuple(r[n].to(BF) if f else None for n, f in zip(("dx", "dw13", "dw2"), need))

    monkeypatch.setattr(se, "bi_ffn_forward_train", forward_train)
    monkeypatch.setattr(se, "bi_ffn_forward", lambda *a, **k: forward_train(*a, **k)[0])
    monkeypatch.setattr(se, "bi_ffn_backward", backward)


def make(seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).to(BF) for s in ((M, H), (2 * I, H), (H, I), (M, H))]


def aligned(t):
    """A copy of t at a 16-byte aligned address."""
    b = torch.empty(t.numel() + 8, dtype=t.dtype)
    k = (-b.data_ptr() // 2) % 8
    return b[k:k + t.numel()].view(t.shape).copy_(t)


# what a gradient looks like after sums, concatenations, transposes, slices
REDUCE = {
    "sum": lambda o: o.sum(),
    "sum_rows": lambda o: (o.sum(0) * torch.arange(H).to(BF)).sum(),
    "sum_columns": lambda o: (o.sum(1) * torch.arange(M).to(BF)).sum(),
    "cat_offset": lambda o: (torch.cat((torch.zeros(M, 4, dtype=BF), o, torch.zeros(M, 4, dtype=BF)), 1)
                             * torch.arange(H + 8).to(BF)).sum(),
    "cat_rows": lambda o: (torch.cat((torch.zeros(1, H, dtype=BF), o)) * torch.arange(H).to(BF)).sum(),
    "transposed": lambda o: (o.t().contiguous() * torch.arange(M).to(BF)).sum(),
    "narrow": lambda o: o[1:3, 5:9].sum(),
}


@pytest.mark.parametrize("how", list(REDUCE))
def test_every_layout_of_a_gradient(formulas, how):
    x, w13, w2, add = [aligned(t).requires_grad_() for t in make()]
    out = se.gated_ffn(x, w13, w2, add)
    REDUCE[how](out).backward()
    o = out.detach().clone().requires_grad_()
    REDUCE[how](o).backward()
    r = ref.ffn(x.detach(), w13.detach(), w2.detach(), dout=o.grad)
    for t, want in ((x, r["dx"]), (w13, r["dw13"]), (w2, r["dw2"]), (add, o.grad)):
        assert torch.equal(t.grad, want.to(BF))


@pytest.mark.parametrize("grad", [False, True])
def test_every_layout_of_the_tokens(formulas, grad):
    """Transposed, misaligned and odd-stride views of x and addend."""
    x, w13, w2, add = [aligned(t) for t in make(1)]
    want = ref.ffn(x, w13, w2, add)["out"].to(BF)

    def inside(more, at):
        return lambda t: aligned(torch.zeros(M, H + more, dtype=BF))[:, at:at + H].copy_(t)

    views = [lambda t: t.t().contiguous().t(), inside(12, 4), inside(16, 4), inside(16, 8)]
    for f in views:
        for a, b in ((f(x), add), (x, f(add))):
            if grad:
                a, b = a.detach().requires_grad_(), b.detach().requires_grad_()
            assert torch.equal(se.gated_ffn(a, w13, w2, b), want)
    # rows that suit the library are handed over as they are
    v = inside(16, 8)(x)
    assert se._rows16(v) is v
    assert se._rows16(x) is x


def test_second_order_is_refused_where_it_is_needed(formulas):
    """A gradient taken with create_graph=True keeps its place in the graph: what would need a second derivative
    of the block raises, instead of losing that term; what does not need one has its value."""
    x, w13, w2, add = [aligned(t).requires_grad_() for t in make(2)]
    loss = se.gated_ffn(x, w13, w2, add).float().square().sum()
    grads = torch.autograd.grad(loss, (x, w13, w2), create_graph=True)
    for t, g in zip((x, w13, w2), grads):
        assert g.requires_grad
        with pytest.raises(RuntimeError, match="second"):
            torch.autograd.grad(loss + g.float().square().sum(), t, retain_graph=True)
    # a sum's gradient is a constant, dx depends on x all the same
    out = se.gated_ffn(x, w13, w2)
    g, = torch.autograd.grad(out.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second"):
        (out.sum() + g.float().square().sum()).backward()
    # first-order terms of a graph that was asked for are right
    for t in (x, w13, w2, add):
        t.grad = None
    se.gated_ffn(x, w13, w2, add).sum().backward(create_graph=True)
    r = ref.ffn(x.detach(), w13.detach(), w2.detach(), dout=torch.ones(M, H))
    for t, n in ((x, "dx"), (w13, "dw13"), (w2, "dw2")):
        assert torch.equal(t.grad.detach(), r[n].to(BF))
    # the addend's gradient is dout itself, differentiable as that is
    v = torch.randn(M, H).to(BF).requires_grad_()
    g, = torch.autograd.grad((se.gated_ffn(x, w13, w2, add) * v).sum(), add, create_graph=True)
    g2, = torch.autograd.grad(g.float().square().sum(), v)
    assert torch.equal(g2, (2 * v.detach().float()).to(BF))


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("no_grad", [False, True])
def test_forward_mode_is_refused(formulas, which, no_grad):
    """A tangent on any argument raises; without one the call is as ever inside a dual level."""
    from torch.autograd import forward_ad
    args = [aligned(t) for t in make(3)]
    want = se.gated_ffn(*args)
    with torch.set_grad_enabled(not no_grad), forward_ad.dual_level():
        assert torch.equal(se.gated_ffn(*args), want)
        dual = list(args)
        dual[which] = forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises((RuntimeError, NotImplementedError), match="forward"):
            se.gated_ffn(*dual)
    with torch.no_grad():
        assert torch.equal(se.gated_ffn(*args), want)
