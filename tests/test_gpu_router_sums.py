"""The router gradient's sums over long groups: few roundings one behind another, and an order that only the
position within the group decides."""
import pytest
import torch

from tests import synthetic as syn

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_long_group(cuda, dtype):
    """66048 products of 1 + 2^-12, which a running sum of thousands rounds the same way again and again (eight sums
    of 8256 of them, added up: 1.2e-4 too small).

    A product is rounded on its way into at most 64 partial sums of a batch of 512 positions (eight warps), into one
    sum for each of 129 batches and into 8 over the warps, each time by at most half a step, 2^-24 of a partial sum
    that is no larger than the result; in dbias into 16 of a batch (32 lanes), 129 and 5.  c is exact: 4 (1 + 2^-12)
    by 0.5 by 0.5."""
    import invariant_moe_gb300 as bm
    n, H, E = 66048, 264, 3
    v = 1 + 2.0 ** -12
    dwts = torch.full((n, 1), 4 * v, device=cuda)
    wts = torch.full((n, 1), 0.5, device=cuda)
    ids = torch.ones(n, 1, dtype=torch.int32, device=cuda)
    x, w = torch.ones(n, H, dtype=dtype, device=cuda), torch.zeros(E, H, device=cuda)
    off, perm = bm.bi_moe_permute(ids, E)
    _, dw, db = bm.bi_router_backward(dwts, ids, wts, x, w, off, perm)
    assert not dw[0].any() and not dw[2].any() and not db[0] and not db[2]
    for name, t, adds in (("dw", dw[1], 64 + 129 + 8), ("dbias", db[1], 16 + 129 + 5)):
        rel = float((t.double() / (n * v) - 1).abs().max())
        assert rel <= adds * 2.0 ** -24, f"{name}: {rel:.2e}"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 31, 512, 513, 1500])
def test_a_group_alone_has_its_bits_among_others(cuda, dtype, n):
    """The order of a group's sum depends on the positions within it, not on what stands before it or behind."""
    import invariant_moe_gb300 as bm
    E, H, before, after = 4, 520, 333, 200
    M = before + n + after
    ids = torch.tensor([0] * before + [2] * n + [3] * after, dtype=torch.int32)[:, None].to(cuda)
    g = torch.Generator().manual_seed(n)
    dwts, wts = torch.randn(M, 1, generator=g).to(cuda), torch.rand(M, 1, generator=g).to(cuda)
    x, w = syn.normal((M, H), 1.0, 5, dtype).to(cuda), syn.normal((E, H), 1.0, 6, F32).to(cuda)
    _, dw, db = bm.bi_router_backward(dwts, ids, wts, x, w, *bm.bi_moe_permute(ids, E))
    s = slice(before, before + n)
    a = [t[s].contiguous() for t in (dwts, ids, wts, x)]
    _, dw1, db1 = bm.bi_router_backward(*a, w, *bm.bi_moe_permute(a[1], E))
    assert torch.equal(dw1[2], dw[2]) and torch.equal(db1[2], db[2])


def test_a_group_past_2_31_elements(cuda):
    """The same where the group's rows lie beyond 2^31 elements of x."""
    import invariant_moe_gb300 as bm
    M, H, E, n = 530000, 4096, 2, 66000
    ids = (torch.arange(M, device=cuda) >= M - n).int()[:, None].contiguous()
    g = torch.Generator(device=cuda)
    g.manual_seed(1)
    dwts, wts = (torch.rand(M, 1, generator=g, device=cuda) for _ in range(2))
    x, w = torch.zeros(M, H, dtype=BF, device=cuda), torch.zeros(E, H, device=cuda)
    x[-n:].copy_(torch.randn(n, H, generator=g, device=cuda))
    _, dw, db = bm.bi_router_backward(dwts, ids, wts, x, w, *bm.bi_moe_permute(ids, E), need=(False, True, True))
    a = [t[-n:] for t in (dwts, ids, wts, x)]
    _, dw1, db1 = bm.bi_router_backward(*a, w, *bm.bi_moe_permute(a[1], E), need=(False, True, True))
    assert not dw[0].any()
    assert torch.equal(dw1[1], dw[1]) and torch.equal(db1[1], db[1])
