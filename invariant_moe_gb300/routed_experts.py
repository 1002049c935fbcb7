"""A routed-experts layer trained: the framework's grouped products, norm, experts
and router as differentiable functions.

``grouped_linear`` is the product of grouped rows with their groups' matrices,
``layer_norm`` the norm before a layer, ``routed_experts`` the gated experts under
a given routing, ``moe_layer_train`` the whole layer (router, top-k, experts) and
``moe_block`` the layer behind its norm, added to its input.  Each is
differentiable once, in reverse mode; their products, sums and norms run in the
library's kernels, copies of inputs that lie off its layout, grouped_linear's rows
of no group and moe_block's sum in torch's.

A backward pass is captured into a CUDA graph only while no eager graph of the same
leaves is alive: such a graph keeps the stream on which autograd adds up a leaf's
gradient, and a capture cannot wait for another stream's work."""
from __future__ import annotations

import contextlib

import torch
from torch.autograd.forward_ad import unpack_dual

from . import (_current_device, bi_grouped_gemm, bi_grouped_gemm_dw, bi_grouped_gemm_dx, bi_layer_norm,
               bi_layer_norm_backward, bi_layer_norm_train, bi_moe_backward, bi_moe_forward, bi_moe_forward_train,
               bi_moe_layer, bi_router_backward, bi_router_topk)
from .shared_expert import _rows16


class _Gradients(torch.autograd.Function):
    """A backward pass as a node of its own: where a gradient is taken with create_graph=True its results stay
    connected to what they depend on (the tensors given besides the function), so that a second derivative, which
    the library does not have, is refused instead of counted as zero.  (Those are the saved inputs of the forward
    pass, so a copy that the library's layout needs is made outside of it, where autograd sees the copy.)"""

    @staticmethod
    def forward(ctx, f, *tensors):
        return f()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("this function has no second derivative (it came up in a gradient of its gradients)")


def _gradients(f, *tensors):
    return _Gradients.apply(f, *tensors) if torch.is_grad_enabled() else f()


def _plain(*tensors):
    """Whether nothing is to be differentiated.  (A tangent of forward-mode differentiation goes to the autograd
    function too, which refuses it.)"""
    tensors = [t for t in tensors if t is not None]
    return not (torch.is_grad_enabled() and any(t.requires_grad for t in tensors)) and all(
        unpack_dual(t).tangent is None for t in tensors)


def _device_of(x):
    """A context in which x's device is the current one, where the library's calls launch."""
    at = x.get_device()
    return torch.cuda.device(at) if at >= 0 and at != _current_device() else contextlib.nullcontext()


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return bi_grouped_gemm(x, w, offsets, out=x.new_zeros(x.shape[0], w.shape[1]))

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy, need = _rows16(dy), ctx.needs_input_grad

        def f():
            dx = bi_grouped_gemm_dx(dy, w, offsets, dx=torch.zeros_like(x)) if need[0] else None
            return dx, bi_grouped_gemm_dw(dy, x, offsets) if need[1] else None

        return (*_gradients(f, dy, x, w), None)


def grouped_linear(x, w, offsets):
    """y [P,N] with y[p] = w[e] x[p] for offsets[e] <= p < offsets[e+1], rows of no group 0; x [P,K] and w [E,N,K]
    bf16, offsets int32 [E+1].  Differentiable in x and w."""
    x = _rows16(x)
    if _plain(x, w):
        return bi_grouped_gemm(x, w, offsets, out=x.new_zeros(x.shape[0], w.shape[1]))
    return _GroupedLinear.apply(x, w, offsets)


def _unit_columns(t):
    return t if t.stride(1) == 1 and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1]) else t.contiguous()


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = bi_layer_norm_train(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.param = next((t.dtype for t in (weight, bias) if t is not None), None)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dy, need, param = _unit_columns(dy), ctx.needs_input_grad[:3], ctx.param

        def f():
            dx, dw, db = bi_layer_norm_backward(dy, x, weight, mean, rstd, need=need)
            return dx, None if dw is None else dw.to(param), None if db is None else db.to(param)

        return (*_gradients(f, dy, x, *(t for t in (weight,) if t is not None)), None)


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Layer norm over the last dimension of x [..., H] (bf16 or fp32), weight and bias [H] (bf16 or fp32) or None.
    Differentiable in x, weight and bias, whose gradients are summed in fp32."""
    rows = _unit_columns(x.reshape(-1, x.shape[-1]))
    y = (bi_layer_norm if _plain(x, weight, bias) else _LayerNorm.apply)(rows, weight, bias, eps)
    return y.view(x.shape)


class _Experts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ids, wts, w13, w2):
        out, saved = bi_moe_forward_train(x, ids, wts, w13, w2)
        ctx.save_for_backward(ids, wts, w13, w2, x, *saved)
        ctx.saved_type = type(saved)
        return out

    @staticmethod
    def backward(ctx, dout):
        ids, wts, w13, w2, x, *saved = ctx.saved_tensors
        saved, dout, n = ctx.saved_type(*saved), _rows16(dout).contiguous(), ctx.needs_input_grad

        def f():
            return bi_moe_backward(dout, ids, wts, w13, w2, saved, need=(n[0], n[2], n[3], n[4]))

        dx, dwts, dw13, dw2 = _gradients(f, dout, x, wts, w13, w2)
        return dx, None, dwts, dw13, dw2


def routed_experts(x, ids, wts, w13, w2):
    """bi_moe_forward, differentiable in x [M,H], wts [M,k] (fp32), w13 [E,2I,H] and w2 [E,H,I]."""
    x, wts = _rows16(x).contiguous(), wts.contiguous()
    with _device_of(x):
        return (bi_moe_forward if _plain(x, wts, w13, w2) else _Experts.apply)(x, ids, wts, w13, w2)


class _MoeLayer(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_router, bias, w13, w2, top_k):
        scores, ids, wts, _ = bi_router_topk(x, w_router, top_k, bias=bias)
        out, saved = bi_moe_forward_train(x, ids, wts, w13, w2)
        ctx.save_for_backward(x, w_router, bias, ids, wts, w13, w2, *saved)
        ctx.saved_type = type(saved)
        ctx.mark_non_differentiable(scores, ids, wts)
        return out, scores, ids, wts

    @staticmethod
    def backward(ctx, dout, *unused):
        x, w_router, bias, ids, wts, w13, w2, *saved = ctx.saved_tensors
        saved, dout, n = ctx.saved_type(*saved), _rows16(dout).contiguous(), ctx.needs_input_grad

        def f():
            dx, dwts, dw13, dw2 = bi_moe_backward(dout, ids, wts, w13, w2, saved, w_router=w_router,
                                                  need=(n[0], n[1] or n[2], n[3], n[4]))
            dw, db = None, None
            if n[1] or n[2]:
                _, dw, db = bi_router_backward(dwts, ids, wts, x, w_router, saved.offsets, saved.perm,
                                               need=(False, n[1], n[2]))
            return dx, dw, db, dw13, dw2

        # (everything depends on the bias through the routing weights)
        return (*_gradients(f, dout, x, w_router, w13, w2, *(t for t in (bias,) if t is not None)), None)


def moe_layer_train(x, w_router, w13, w2, top_k, bias=None):
    """moe_layer (the same bits up to H = 2048), differentiable in x, w_router, bias, w13 and w2.  Returns (out, scores, ids, wts);
    the last three carry no gradient."""
    x = _rows16(x).contiguous()
    with _device_of(x):
        if _plain(x, w_router, bias, w13, w2):
            return bi_moe_layer(x, w_router, w13, w2, top_k, bias=bias)
        return _MoeLayer.apply(x, w_router, bias, w13, w2, top_k)


def moe_block(x, norm_weight, norm_bias, w_router, w13, w2, top_k, bias=None):
    """x + moe_layer_train(layer_norm(x)): the layer as it stands in a model."""
    return x + moe_layer_train(layer_norm(x, norm_weight, norm_bias), w_router, w13, w2, top_k, bias=bias)[0]


def main():
    """Fine-tune a block of routed experts to a teacher's output, then serve its layer."""
    torch.manual_seed(0)
    dev, bf = torch.device("cuda:0"), torch.bfloat16
    M, H, I, E, k = 1024, 512, 256, 16, 4

    def normal(*shape, std):
        return torch.randn(*shape, device=dev) * std

    teacher = [1.0 + normal(H, std=0.1), normal(H, std=0.1), normal(E, H, std=H ** -0.5),
               normal(E, 2 * I, H, std=H ** -0.5), normal(E, H, I, std=I ** -0.5)]
    # fp32 weights, begun some way off; the norm and the router stay in fp32, the experts compute in bf16
    master = [t + 0.3 * normal(*t.shape, std=float(t.std())) for t in teacher]

    def params(ws, grad=False):
        return [w.to(bf if w.dim() == 3 else torch.float32, copy=True).requires_grad_(grad) for w in ws]

    for step in range(60):
        x = normal(M, H, std=1.0).to(bf)
        with torch.no_grad():
            target = moe_block(x, *params(teacher), k)
        ws = params(master, grad=True)
        loss = (moe_block(x, *ws, k).float() - target.float()).square().mean()
        loss.backward()
        with torch.no_grad():
            for w, p in zip(master, ws):
                w -= 20.0 * p.grad.float()
        if step % 20 == 0 or step == 59:
            print(f"step {step:2d}  loss {float(loss.detach()):.5f}")

    # serve the layer: a batch, and a single token
    norm_w, norm_b, router, w13, w2 = params(master)
    h = layer_norm(x, norm_w, norm_b)
    out = bi_moe_layer(h, router, w13, w2, k)[0]
    one = bi_moe_layer(h[:1], router, w13, w2, k)[0]
    print("one token has its row of the batch bit for bit:", bool(torch.equal(one, out[:1])))


if __name__ == "__main__":
    main()
