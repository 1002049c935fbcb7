"""Calls given ``stream=``: everything they allocate comes from that stream's
memory pool (no GPU: the allocator, the streams and the library are recorded).

Memory of the current stream's pool may still be read or written by work that is
pending there, and goes back to it when the call returns, while the kernels on
the other stream are still to run: both are races that a result shows only by
chance, so the rule is checked here."""
import contextlib

import pytest
import torch

import invariant_moe_gb300 as bm
from invariant_moe_gb300 import shared_expert as se

BF = torch.bfloat16


class Stream:
    """Stands for torch.cuda.Stream."""
    device = torch.device("cuda", 0)

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def world(monkeypatch):
    """Records the stream that is current at each allocation, the streams that kernels go to, and record_stream."""
    class World:
        here, other = Stream(1), Stream(2)
        current = here
        allocated, launched, recorded = [], [], []

    w = World()
    w.allocated, w.launched, w.recorded = [], [], []

    @contextlib.contextmanager
    def stream_context(s):
        old, w.current = w.current, s
        yield
        w.current = old

    real_empty = torch.empty

    def empty(*shape, dtype=None, device=None):
        w.allocated.append(w.current.cuda_stream)
        return real_empty(*shape, dtype=dtype)

    class Library:
        @staticmethod
        def bi_ffn_workspace_bytes(M, H, I):
            return 256

        def __getattr__(self, name):
            if name == "bi_moe_workspace_bytes" or name == "bi_moe_permute_workspace_bytes":
                return lambda *a: 256

            def call(*a):
                h = a[-1]
                w.launched.append(getattr(h, "value", h))
                return 0
            return call

    lib = Library()
    monkeypatch.setattr(bm, "load_library", lambda *a: lib)
    monkeypatch.setattr(bm, "_fns", {})
    monkeypatch.setattr(bm, "_device_of", lambda t, name: 0)
    monkeypatch.setattr(bm, "_current_device", lambda: 0)
    monkeypatch.setattr(bm, "_raw_stream", lambda dev: w.current.cuda_stream)
    monkeypatch.setattr(bm, "_rows", lambda t, dtype, name, rows, cols, dev: (t.data_ptr(), cols))
    monkeypatch.setattr(bm, "_flat", lambda t, dtype, name, dev: t.data_ptr())
    monkeypatch.setattr(bm, "_ptr", lambda t, dtype, name, dev=None: None)
    monkeypatch.setattr(bm, "_mx4_operand",
                        lambda q, s, name, dev: (q.data_ptr(), s.data_ptr(), q.shape[0], 2 * q.shape[1]))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w.recorded.append((id(t), s.cuda_stream)))
    return w


M, H, I, K = 4, 64, 32, 64


def tensors():
    z = torch.zeros
    return {"x": z(M, H, dtype=BF), "w13": z(2 * I, H, dtype=BF), "w2": z(H, I, dtype=BF),
            "gu": z(M, 2 * I), "act": z(M, I, dtype=BF), "q": z(M, K // 2, dtype=torch.uint8),
            "s": z(1, 1, 512, dtype=torch.uint8), "wq": z(2 * I, K // 2, dtype=torch.uint8),
            **routed()}


def expert():
    e = se.Mx4SharedExpert.__new__(se.Mx4SharedExpert)
    z = torch.zeros
    e.w13, e.s13 = z(2 * I, H // 2, dtype=torch.uint8), z(1, 1, 512, dtype=torch.uint8)
    e.w2, e.s2 = z(H, I // 2, dtype=torch.uint8), z(1, 1, 512, dtype=torch.uint8)
    return e


E, TOPK = 4, 2


def routed():
    """Arguments of the routed experts' calls."""
    z = torch.zeros
    return {"scores": z(M, E), "w_router": z(E, H), "e13": z(E, 2 * I, H, dtype=BF), "e2": z(E, H, I, dtype=BF),
            "ids": z(M, TOPK, dtype=torch.int32), "wts": z(M, TOPK), "off": z(E + 1, dtype=torch.int32),
            "perm": z(M * TOPK, dtype=torch.int32), "xp": z(M * TOPK, H, dtype=BF),
            "actp": z(M * TOPK, I, dtype=BF), "contrib": z(M * TOPK, H)}


def layer(t, s):
    z = torch.zeros
    return se.moe_layer_with_shared_expert(t["x"], z(E, H), z(E, 2 * I, H, dtype=BF), z(E, H, I, dtype=BF), TOPK,
                                           t["w13"], t["w2"], stream=s)


CALLS = {
    "ffn_forward": lambda t, s: bm.bi_ffn_forward(t["x"], t["w13"], t["w2"], stream=s),
    "ffn_forward_out": lambda t, s: bm.bi_ffn_forward(t["x"], t["w13"], t["w2"], out=t["x"], stream=s),
    "ffn_forward_train": lambda t, s: bm.bi_ffn_forward_train(t["x"], t["w13"], t["w2"], stream=s),
    "ffn_backward": lambda t, s: bm.bi_ffn_backward(t["x"], t["x"], t["w13"], t["w2"], t["gu"], t["act"], stream=s),
    "mx4_quantize": lambda t, s: bm.bi_mx4_quantize(t["x"], stream=s),
    "mx4_dequantize": lambda t, s: bm.bi_mx4_dequantize(t["q"], t["s"], stream=s),
    "mx4_gemm": lambda t, s: bm.bi_mx4_gemm(t["q"], t["s"], t["wq"], t["s"], stream=s),
    "mx4_gate_up": lambda t, s: bm.bi_mx4_gate_up(t["q"], t["s"], t["wq"], t["s"], stream=s),
    "Mx4SharedExpert": lambda t, s: expert()(t["x"], stream=s),
    "moe_layer_with_shared_expert": layer,
    # the routed experts' calls
    "cast": lambda t, s: bm.bi_cast_bf16_to_f32(t["x"], stream=s),
    "router_gemm": lambda t, s: bm.bi_router_gemm(t["x"], t["w_router"], stream=s),
    "router_gemm_splitk_negctl": lambda t, s: bm.bi_router_gemm_splitk_negctl(t["x"], t["w_router"], stream=s),
    "topk": lambda t, s: bm.bi_topk(t["scores"], TOPK, want_probs=True, stream=s),
    "router_topk": lambda t, s: bm.bi_router_topk(t["x"], t["w_router"], TOPK, want_probs=True, stream=s),
    "moe_forward": lambda t, s: bm.bi_moe_forward(t["x"], t["ids"], t["wts"], t["e13"], t["e2"], stream=s),
    "moe_layer": lambda t, s: bm.moe_layer(t["x"], t["w_router"], t["e13"], t["e2"], TOPK, stream=s),
    "permute": lambda t, s: bm.bi_moe_permute(t["ids"], E, stream=s),
    "gather": lambda t, s: bm.bi_moe_gather(t["x"], t["off"], t["perm"], TOPK, stream=s),
    "gate_up": lambda t, s: bm.bi_moe_gate_up(t["xp"], t["off"], t["perm"], t["wts"], t["e13"], TOPK, stream=s),
    "gate_up_tokens": lambda t, s: bm.bi_moe_gate_up_tokens(t["x"], t["off"], t["perm"], t["wts"], t["e13"], TOPK,
                                                            stream=s),
    "down": lambda t, s: bm.bi_moe_down(t["actp"], t["off"], t["perm"], t["e2"], M, TOPK, stream=s),
    "gather_routing": lambda t, s: bm.bi_moe_gather_routing(t["ids"], t["wts"], t["off"], t["perm"], E, stream=s),
    "scatter_contrib": lambda t, s: bm.bi_moe_scatter_contrib(t["xp"], t["off"], t["perm"], M, TOPK, stream=s),
    "combine": lambda t, s: bm.bi_moe_combine(t["contrib"], M, TOPK, stream=s),
    "combine_consume": lambda t, s: bm.bi_moe_combine_consume(t["contrib"], M, TOPK, stream=s),
    "fp32_fma_probe": lambda t, s: bm.bi_fp32_fma_probe(1, 1, stream=s),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_allocates_and_launches_on_the_stream_given(world, name):
    t = tensors()
    out = CALLS[name](t, world.other)
    assert world.allocated and set(world.allocated) == {world.other.cuda_stream}
    assert world.launched and set(world.launched) == {world.other.cuda_stream}
    assert world.current is world.here
    # what the call hands out may be used, and dropped, on the stream that was current
    given = {id(v) for v in t.values()}
    for r in out if isinstance(out, tuple) else (out,):
        if r is not None and id(r) not in given:
            assert (id(r), world.here.cuda_stream) in world.recorded


@pytest.mark.parametrize("name", list(CALLS))
def test_without_a_stream_nothing_is_recorded(world, name):
    CALLS[name](tensors(), None)
    assert set(world.allocated) == set(world.launched) == {world.here.cuda_stream}
    assert not world.recorded
    CALLS[name](tensors(), world.here)
    assert set(world.allocated) == set(world.launched) == {world.here.cuda_stream}
    assert not world.recorded
