"""A shared (always active) expert beside the routed experts: trained in bf16,
served in bf16 or in 4 bits.

``gated_ffn`` is the feed-forward block as a differentiable function,
``moe_layer_with_shared_expert`` the routed layer with a shared expert added to
it, and ``Mx4SharedExpert`` the expert with its weights in the microscaled 4-bit
form: quantise the tokens, the gated product, quantise the activations, the down
product added to the routed experts' output.  Everything but autograd's
bookkeeping runs in the library's kernels."""
from __future__ import annotations

import torch
from torch.autograd.forward_ad import unpack_dual

from . import (_on_stream, bi_ffn_backward, bi_ffn_forward, bi_ffn_forward_train, bi_mx4_gate_up, bi_mx4_gemm,
               bi_mx4_quantize, moe_layer, mx4_interleave_gate_up)


def _rows16(t):
    """t [M, cols], or a copy of it where its rows do not lie as the library takes them: unit column stride, a
    row stride of at least cols and a multiple of 8, 16-byte aligned.  (Autograd hands out rows of stride 0
    for a sum over the tokens, and slices at any column for a concatenation.)"""
    rows, cols = t.shape
    if t.stride(1) == 1 and (rows <= 1 or (t.stride(0) >= cols and t.stride(0) % 8 == 0)) and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _gradients(need, dout, x, w13, w2, gu, act):
    return bi_ffn_backward(dout, x, w13, w2, gu, act, need=need)


class _FfnGradients(torch.autograd.Function):
    """The backward pass as a node of its own: where a gradient is taken with create_graph=True its results stay
    connected to what they depend on, so that a second derivative, which the library does not have, is refused
    instead of counted as zero."""

    @staticmethod
    def forward(ctx, *args):
        return _gradients(*args)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("gated_ffn has no second derivative (it came up in a gradient of its gradients)")


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w13, w2, addend):
        out, gu, act = bi_ffn_forward_train(x, w13, w2, addend=addend)
        ctx.save_for_backward(x, w13, w2, gu, act)
        return out

    @staticmethod
    def backward(ctx, dout):
        x, w13, w2, gu, act = ctx.saved_tensors
        dout = _rows16(dout)
        gradients = _FfnGradients.apply if torch.is_grad_enabled() else _gradients
        dx, dw13, dw2 = gradients(ctx.needs_input_grad[:3], dout, x, w13, w2, gu, act)
        return dx, dw13, dw2, dout if ctx.needs_input_grad[3] else None


def gated_ffn(x, w13, w2, addend=None):
    """(silu(x Wg^T) * (x Wu^T)) W2^T (+ addend), differentiable once, in reverse mode, in every argument;
    x [M,H], w13 [2I,H], w2 [H,I] and addend [M,H] bf16."""
    # (copies that the layout needs are made here, where autograd sees them)
    x, addend = _rows16(x), None if addend is None else _rows16(addend)
    args = [t for t in (x, w13, w2, addend) if t is not None]
    # a tangent of forward-mode differentiation goes to the autograd function too, which refuses it
    if not (torch.is_grad_enabled() and any(t.requires_grad for t in args)) and all(
            unpack_dual(t).tangent is None for t in args):
        return bi_ffn_forward(x, w13, w2, addend=addend)
    return _GatedFfn.apply(x, w13, w2, addend)


def moe_layer_with_shared_expert(x, w_router, w13, w2, top_k, shared_w13, shared_w2, bias=None, stream=None):
    """moe_layer plus a bf16 shared expert on the same tokens, summed in fp32 before the one rounding of the
    sum.  Returns (out, scores, ids, wts); a token's row of out has the same bits in every batch."""
    if stream is not None:
        return _on_stream(stream, moe_layer_with_shared_expert, x, w_router, w13, w2, top_k, shared_w13, shared_w2,
                          bias)
    out, scores, ids, wts = moe_layer(x, w_router, w13, w2, top_k, bias=bias)
    bi_ffn_forward(x, shared_w13, shared_w2, addend=out, out=out)
    return out, scores, ids, wts


class Mx4SharedExpert:
    """A shared expert whose weights are kept in 4 bits: a little over a quarter of their bf16 bytes."""

    def __init__(self, w13, w2):
        if w13.shape[0] % 64 or w13.shape[1] % 32:
            raise ValueError("the 4-bit form needs H and I to be multiples of 32")
        self.w13, self.s13 = bi_mx4_quantize(mx4_interleave_gate_up(w13))
        self.w2, self.s2 = bi_mx4_quantize(w2)

    def __call__(self, x, addend=None, stream=None):
        if stream is not None:
            return _on_stream(stream, self.__call__, x, addend)
        xq, xs = bi_mx4_quantize(x)
        act = bi_mx4_gate_up(xq, xs, self.w13, self.s13)
        aq, as_ = bi_mx4_quantize(act)
        return bi_mx4_gemm(aq, as_, self.w2, self.s2, addend=addend)


def main():
    """Fine-tune a shared expert to a teacher's output, then serve it beside routed experts in bf16 and in 4 bits."""
    torch.manual_seed(0)
    dev, bf = torch.device("cuda:0"), torch.bfloat16
    M, H, I, E, k = 512, 512, 256, 16, 4

    def normal(*shape, std):
        return torch.randn(*shape, device=dev) * std

    teacher = [normal(2 * I, H, std=H ** -0.5).to(bf), normal(H, I, std=I ** -0.5).to(bf)]
    # fp32 weights, begun half a standard deviation from the teacher's
    master = [t.float() + normal(*t.shape, std=0.5 * float(t.float().std())) for t in teacher]
    for step in range(60):
        x = normal(M, H, std=1.0).to(bf)
        target = gated_ffn(x, *teacher)
        w13, w2 = (w.to(bf).requires_grad_() for w in master)
        loss = (gated_ffn(x, w13, w2).float() - target.float()).square().mean()
        loss.backward()
        with torch.no_grad():
            for w, g in zip(master, (w13.grad, w2.grad)):
                w -= 20.0 * g.float()
        if step % 20 == 0 or step == 59:
            print(f"step {step:2d}  loss {float(loss.detach()):.5f}")
    w13, w2 = (w.to(bf) for w in master)

    # serve it beside routed experts, for a prefill and for a single token
    router = normal(E, H, std=0.02)
    routed = normal(E, 2 * I, H, std=H ** -0.5).to(bf), normal(E, H, I, std=I ** -0.5).to(bf)
    out, _, ids, wts = moe_layer_with_shared_expert(x, router, *routed, k, w13, w2)
    one = moe_layer_with_shared_expert(x[:1], router, *routed, k, w13, w2)[0]
    print("one token has its row of the batch bit for bit:", bool(torch.equal(one, out[:1])))
    base = moe_layer(x, router, *routed, k)[0]
    out4 = Mx4SharedExpert(w13, w2)(x, addend=base)
    err = float((out4.float() - out.float()).norm() / (out.float() - base.float()).norm())
    print(f"4-bit shared expert: {err:.3f} of the expert's output off the bf16 one's")


if __name__ == "__main__":
    main()
