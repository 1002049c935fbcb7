"""Calls given ``stream=`` beside a busy current stream: the same bits as on the
current stream, whatever happens to memory on the other one meanwhile."""
import pytest
import torch

from tests import synthetic as syn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
BUSY = 100_000_000  # clock cycles: 50 ms or so, far longer than the calls and the host's work between them


def calls(dev):
    """name -> f(stream) for calls that allocate."""
    import invariant_moe_gb300 as bm
    from invariant_moe_gb300 import shared_expert as se
    M, H, I, E, k = 1500, 512, 256, 16, 4
    x = syn.normal((M, H), 1.0, 1, BF).to(dev)
    w13, w2 = syn.normal((2 * I, H), H ** -0.5, 2, BF).to(dev), syn.normal((H, I), I ** -0.5, 3, BF).to(dev)
    add, dout = syn.normal((M, H), 0.5, 4, BF).to(dev), syn.normal((M, H), 1.0, 5, BF).to(dev)
    _, gu, act = bm.bi_ffn_forward_train(x, w13, w2)
    xq, wq = bm.bi_mx4_quantize(x), bm.bi_mx4_quantize(w13)
    four = se.Mx4SharedExpert(w13, w2)
    w = syn.moe_weights(H, E, I, seed=11, unit=True)
    routed = [t.to(dev) for t in (w.w_router, w.w13, w.w2)]
    return {
        "forward": lambda s: bm.bi_ffn_forward(x, w13, w2, addend=add, stream=s),
        "forward_train": lambda s: bm.bi_ffn_forward_train(x, w13, w2, stream=s),
        "backward": lambda s: bm.bi_ffn_backward(dout, x, w13, w2, gu, act, stream=s),
        "quantize": lambda s: bm.bi_mx4_quantize(x, stream=s),
        "gemm": lambda s: bm.bi_mx4_gemm(*xq, *wq, stream=s),
        "four_bits": lambda s: four(x, addend=add, stream=s),
        "layer": lambda s: se.moe_layer_with_shared_expert(x, *routed, k, w13, w2, stream=s),
    }


def as_tuple(r):
    return r if isinstance(r, tuple) else (r,)


@pytest.mark.parametrize("name", ["forward", "forward_train", "backward", "quantize", "gemm", "four_bits", "layer"])
def test_beside_work_on_the_current_stream(cuda, name):
    f = calls(cuda)[name]
    want = [t.clone() for t in as_tuple(f(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for size in (1 << 16, 1 << 20, 3 << 20):  # sizes of the calls' own temporaries and results
        # memory whose last use on the current stream is still to come when the call allocates
        old = [torch.full((size,), i, dtype=torch.uint8, device=cuda) for i in range(8)]
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        kept = [t.clone() for t in old]
        del old
        got = as_tuple(f(side))
        torch.cuda.synchronize()
        assert all(bool((t == i).all()) for i, t in enumerate(kept)), "the call wrote memory that was in use"
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        del got, kept
        # memory that the call has given back, reused on the current stream before its kernels have run
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
        got = as_tuple(f(side))
        junk = [torch.full((size,), 0xff, dtype=torch.uint8, device=cuda) for _ in range(8)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), "the call's memory was reused too early"
        del got, junk


def test_two_streams_at_once(cuda):
    """Overlapping calls on two streams share no temporaries."""
    f = calls(cuda)
    want = {n: [t.clone() for t in as_tuple(f[n](None))] for n in ("forward", "backward", "four_bits")}
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s in sides:
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
    for _ in range(4):
        for s in sides:
            got += [(n, as_tuple(f[n](s))) for n in want]
    torch.cuda.synchronize()
    for n, r in got:
        assert all(torch.equal(a, b) for a, b in zip(want[n], r)), n


def test_results_dropped_on_the_current_stream(cuda):
    """A result that is still read on the current stream when it is dropped is not overwritten by the next call."""
    f = calls(cuda)["forward"]
    want = f(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = f(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    kept = out.clone()
    del out
    with torch.cuda.stream(side):
        junk = [torch.full((want.numel() * 2,), 0xff, dtype=torch.uint8, device=cuda) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(kept, want)
    del junk


@pytest.mark.parametrize("name", ["forward", "backward", "four_bits", "layer"])
def test_captured_on_a_forked_stream(cuda, name):
    """Inside a graph capture, on a stream that is forked from the captured one and joined again."""
    f = calls(cuda)[name]
    want = [t.clone() for t in as_tuple(f(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        first = as_tuple(f(side))
        second = as_tuple(f(side))
        torch.cuda.current_stream().wait_stream(side)
        total = [a.float() + b.float() for a, b in zip(first, second)]
    for _ in range(2):
        for t in (*first, *second, *total):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for w, a, b, t in zip(want, first, second, total):
            assert torch.equal(a, w) and torch.equal(b, w) and torch.equal(t, w.float() + w.float())
