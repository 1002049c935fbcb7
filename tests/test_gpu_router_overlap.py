"""bi_router_backward's dx and dW, which run side by side: a bad grouping leaves dx whole, and the pair is captured,
replayed with other inputs and run on two streams."""
import pytest
import torch

from tests.test_gpu_router_backward import BF, F32, make

pytestmark = pytest.mark.gpu

# tokens, hidden, experts, slots: all read W from shared memory, so that dW runs beside dx
SIZES = [(700, 520, 8, 2), (3000, 1024, 64, 4)]


@pytest.mark.parametrize("M,H,E,k", SIZES)
def test_a_bad_grouping_leaves_dx_whole(cuda, M, H, E, k):
    """dx depends on no offsets.  The next work on the stream reads all of it, whichever expert's offsets are bad."""
    import invariant_moe_gb300 as bm
    a = [t.to(cuda) for t in make(M, H, E, k, 1800, BF)]
    off, perm = bm.bi_moe_permute(a[1], E)
    want = bm.bi_router_backward(*a, off, perm)[0].clone()
    dx, seen = torch.empty_like(want), torch.empty_like(want)
    for e, value in ((0, -1), (1, M * k + 1), (E, M * k + 1), (2, -5)):
        bad = off.clone()
        bad[e] = value
        for _ in range(3):
            dx.fill_(7)
            bm.bi_router_backward(*a, bad, perm, dx=dx)
            seen.copy_(dx)
            assert torch.equal(seen, want)
        assert bm.device_error() == 4


def step(bm, a, off, perm, buf):
    bm.bi_router_backward(*a, off, perm, dx=buf[0], dw=buf[1], dbias=buf[2])
    buf[3].copy_(buf[0])  # the next work on the stream
    return buf


def buffers(M, H, E, dtype, dev):
    return [torch.empty(M, H, dtype=dtype, device=dev), torch.empty(E, H, device=dev), torch.empty(E, device=dev),
            torch.empty(M, H, dtype=dtype, device=dev)]


@pytest.mark.parametrize("M,H,E,k", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_captured_and_replayed(cuda, M, H, E, k, dtype):
    import invariant_moe_gb300 as bm
    sets = []
    for i in range(3):
        a = [t.to(cuda) for t in make(M, H, E, k, 1900 + 10 * i, dtype)]
        g = bm.bi_moe_permute(a[1], E)
        sets.append(([*a, *g], [t.clone() for t in step(bm, a, *g, buffers(M, H, E, dtype, cuda))]))
    given = [t.clone() for t in sets[0][0]]
    buf = buffers(M, H, E, dtype, cuda)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        # the inputs change in the graph too, right before the pair
        dwts = given[0] * 1.0
        step(bm, [dwts, *given[1:5]], given[5], given[6], buf)
    for i in (1, 0, 2, 1):
        for t, v in zip(given, sets[i][0]):
            t.copy_(v)
        for t in buf:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(buf, sets[i][1]))


def test_on_two_streams_at_once(cuda):
    import invariant_moe_gb300 as bm
    work = []
    for i, (M, H, E, k) in enumerate(SIZES):
        a = [t.to(cuda) for t in make(M, H, E, k, 2000 + 10 * i, BF)]
        g = bm.bi_moe_permute(a[1], E)
        want = [t.clone() for t in step(bm, a, *g, buffers(M, H, E, BF, cuda))]
        work.append((a, g, buffers(M, H, E, BF, cuda), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for a, g, buf, _, s in work:
            with torch.cuda.stream(s):
                step(bm, a, *g, buf)
    torch.cuda.synchronize()
    for _, _, buf, want, _ in work:
        assert all(torch.equal(x, y) for x, y in zip(buf, want))
