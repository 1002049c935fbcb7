"""The differentiable routed layer's handling of autograd (no GPU): the library's
calls are replaced by their formulas."""
import pytest
import torch

import invariant_moe_gb300 as bm
from invariant_moe_gb300 import routed_experts as rx
from tests import train_reference as ref

BF, F32 = torch.bfloat16, torch.float32
M, H, E, K, I = 6, 16, 4, 2, 8
OFFSETS = torch.tensor([0, 2, 2, 5, 6], dtype=torch.int32)
IDS = torch.tensor([[0, 1], [1, 2], [3, 0], [2, 3], [1, 3], [0, 2]], dtype=torch.int32)


@pytest.fixture
def formulas(monkeypatch):
    def saved_of(wts):
        z = torch.zeros(1)
        return bm.MoeSaved(OFFSETS.clone(), torch.zeros(M * K, dtype=torch.int32), z.int(), z, z, z)

    def grouped_gemm(x, w, offsets, out=None):
        return out.copy_(ref.grouped(x, w, offsets)[0])

    def grouped_gemm_dx(dy, w, offsets, dx=None):
        return dx.copy_(ref.grouped(dy, w.transpose(1, 2), offsets)[0])

    def norm_train(x, weight, bias, eps):
        r, _ = ref.norm(x, weight, bias, eps)
        return r["y"].to(x.dtype), r["mean"].float(), r["rstd"].float()

    def norm_backward(dy, x, weight, mean, rstd, need):
        r, _ = ref.norm(x, weight, None, 1e-5, dy)
        return tuple(r[n].to(t) if f else None
                     for n, t, f in zip(("dx", "dweight", "dbias"), (x.dtype, F32, F32), need))

    def forward(x, ids, wts, w13, w2):
        return ref.experts(x, ids, wts, w13, w2)[0]["out"].to(BF)

    def backward(dout, ids, wts, w13, w2, saved, need, w_router=None):
        r, _ = ref.experts(given["x"], ids, wts, w13, w2, dout)
        if w_router is not None:
            r["dx"] = r["dx"] + ref.router_grads(r["dwts"], ids, wts, given["x"], w_router)[0]["dx"]
        return tuple(r[n].to(t) if f else None
                     for n, t, f in zip(("dx", "dwts", "dw13", "dw2"), (BF, F32, BF, BF), need))

    def forward_train(x, ids, wts, w13, w2):
        given["x"] = x.detach().clone()
        return forward(x, ids, wts, w13, w2), saved_of(wts)

    def router(x, w, k, bias=None):
        s = x.float() @ w.T + (0 if bias is None else bias)
        ids = s.topk(k, dim=1).indices.int()
        return s, ids, torch.sigmoid(s.gather(1, ids.long())), None

    def router_backward(dwts, ids, wts, x, w, offsets, perm, need):
        r, _ = ref.router_grads(dwts, ids, wts, x, w)
        return tuple(r[n].float() if f else None for n, f in zip(("dx", "dw", "dbias"), need))

    def layer(x, w_router, w13, w2, k, bias=None):
        s, ids, wts, _ = router(x, w_router, k, bias)
        return forward(x, ids, wts, w13, w2), s, ids, wts

    given = {}
    for name, f in (("bi_grouped_gemm", grouped_gemm), ("bi_grouped_gemm_dx", grouped_gemm_dx),
                    ("bi_grouped_gemm_dw", lambda dy, x, off: ref.grouped_dw(dy, x, off)[0].to(BF)),
                    ("bi_layer_norm", lambda *a: norm_train(*a)[0]), ("bi_layer_norm_train", norm_train),
                    ("bi_layer_norm_backward", norm_backward), ("bi_moe_forward", forward),
                    ("bi_moe_forward_train", forward_train), ("bi_moe_backward", backward), ("bi_moe_layer", layer),
                    ("bi_router_topk", router), ("bi_router_backward", router_backward)):
        monkeypatch.setattr(rx, name, f)


def values(seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*s, dtype=BF):
        return torch.randn(*s, generator=g).to(dtype)

    return {"x": normal(M, H), "wg": normal(E, I, H), "router": normal(E, H, dtype=F32), "bias": normal(E, dtype=F32),
            "w13": normal(E, 2 * I, H), "w2": normal(E, H, I), "wts": torch.rand(M, K, generator=g),
            "nw": normal(H, dtype=F32)}


FUNCTIONS = {
    "grouped_linear": lambda v: rx.grouped_linear(v["x"], v["wg"], OFFSETS),
    "layer_norm": lambda v: rx.layer_norm(v["x"]),
    "layer_norm_weight": lambda v: rx.layer_norm(v["x"], v["nw"]),
    "routed_experts": lambda v: rx.routed_experts(v["x"], IDS, v["wts"], v["w13"], v["w2"]),
    "moe_layer_train": lambda v: rx.moe_layer_train(v["x"], v["router"], v["w13"], v["w2"], K, bias=v["bias"])[0],
}
# the functions whose gradient with respect to an argument depends on that argument, or may
SECOND = [("layer_norm", "x"), ("layer_norm_weight", "x"), ("routed_experts", "x"), ("routed_experts", "wts"),
          ("routed_experts", "w13"), ("moe_layer_train", "x"), ("moe_layer_train", "router"),
          ("moe_layer_train", "bias"), ("moe_layer_train", "w13")]


def strided(t):
    """t's values, in a view that no kernel takes as it lies."""
    if t.dim() != 2:
        return t.clone()
    return t.t().contiguous().t()


@pytest.mark.parametrize("name,arg", SECOND)
@pytest.mark.parametrize("view", [strided, torch.clone])
def test_second_derivatives_are_refused_in_every_layout(formulas, name, arg, view):
    """The gradient of a sum (a constant dout) with respect to one argument alone still depends on that argument:
    a penalty on it raises, however the argument lies in memory, instead of being dropped."""
    v = values()
    v[arg] = view(v[arg]).requires_grad_()
    (g,) = torch.autograd.grad(FUNCTIONS[name](v).float().sum(), v[arg], create_graph=True)
    assert g.requires_grad
    with pytest.raises(RuntimeError, match="second derivative"):
        (g.float().square().sum() + v[arg].float().sum()).backward()


@pytest.mark.parametrize("name", list(FUNCTIONS))
def test_gradients_of_strided_arguments(formulas, name):
    """Those of the same values in contiguous tensors, in the arguments' own shapes."""
    grads = []
    for view in (torch.clone, strided):
        v = {n: view(t).requires_grad_() for n, t in values(1).items()}
        FUNCTIONS[name](v).float().square().sum().backward()
        grads.append({n: t.grad for n, t in v.items() if t.grad is not None})
    assert grads[0] and grads[0].keys() == grads[1].keys()
    assert all(torch.equal(grads[0][n], grads[1][n]) for n in grads[0])


@pytest.mark.parametrize("name", ["routed_experts", "moe_layer_train"])
@pytest.mark.parametrize("grad", [False, True])
def test_runs_with_the_tensors_device_current(formulas, monkeypatch, name, grad):
    """Tensors of device 1 while device 0 is the current one: the calls underneath launch on the current device's
    stream, so device 1 is made current around all of them."""
    current, seen = [0], []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *a):
            current.pop()

    for f in ("bi_moe_forward", "bi_moe_forward_train", "bi_moe_layer", "bi_router_topk"):
        def call(*a, f=getattr(rx, f), **k):
            seen.append(current[-1])
            return f(*a, **k)
        monkeypatch.setattr(rx, f, call)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(rx, "_current_device", lambda: current[-1], raising=False)
    v = values(2)
    if grad:
        v["w2"].requires_grad_()
    FUNCTIONS[name](v)
    assert seen and set(seen) == {1} and current == [0]


@pytest.mark.parametrize("name", ["routed_experts", "moe_layer_train"])
@pytest.mark.parametrize("grad", [False, True])
def test_rows_off_the_16_byte_grid(formulas, monkeypatch, name, grad):
    """A contiguous x that starts off a 16-byte boundary is copied, not refused; and a copy is all that differs."""
    def checked(f):
        def call(x, *a, **k):
            if x.data_ptr() % 16 or not x.is_contiguous():
                raise RuntimeError("alignment")
            return f(x, *a, **k)
        return call

    for f in ("bi_moe_forward", "bi_moe_forward_train", "bi_moe_layer"):
        monkeypatch.setattr(rx, f, checked(getattr(rx, f)))
    v = values(3)
    want = FUNCTIONS[name](v)
    flat = torch.empty(M * H + 16, dtype=BF)
    at = (-flat.data_ptr() // 2) % 8 + 3
    v["x"] = flat[at:at + M * H].view(M, H).copy_(v["x"]).detach().requires_grad_(grad)
    assert v["x"].data_ptr() % 16 and v["x"].is_contiguous()
    out = FUNCTIONS[name](v)
    assert torch.equal(out, want)
    if grad:
        out.float().square().sum().backward()
        got, v["x"] = v["x"].grad, v["x"].detach().clone().requires_grad_()
        FUNCTIONS[name](v).float().square().sum().backward()
        assert torch.equal(got, v["x"].grad)
