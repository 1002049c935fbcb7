"""The routed experts' training step where its reductions are cut into slices (H > 2048: gate/up; H > 4096: dact
too): the fp32 result's error, and wide tiles, several to a CTA pair."""
import pytest
import torch

from tests import train_reference as ref
from tests.test_gpu_moe_train import make

pytestmark = pytest.mark.gpu


def dwts_bound(H):
    """2-norm of dwts' error over dwts', for g, u and dact of random data.

    The tensor cores add 16 products at a time and drop what does not fit 24 bits: at most 2^-23 of the running sum,
    half of that on average, always towards zero.  Over a chain of s additions the running sum grows evenly to the
    final one as far as that goes with it, so a chain takes off s/2 halves: s/4 2^-23; twice that is allowed.  The rest
    of the additions' errors has no direction and averages out over the 128 features summed, as have the roundings of
    s, silu and of the products (APPROX and a few 2^-24): 2e-6 for all of them."""
    gate_up, dact = H if H <= 2048 else 1024, min(H, 4096)
    return (2 * gate_up + dact) / 16 / 2 * 2.0 ** -23 + 2e-6


@pytest.mark.parametrize("H", [256, 1024, 2048, 2176, 4096, 4224, 8192, 32768])
def test_the_error_of_dwts_does_not_grow_with_long_reductions(cuda, H):
    import invariant_moe_gb300 as bm
    M, E, k, I = 48, 2, 2, 128
    x, ids, wts, w13, w2, dout = make(M, H, E, k, I, 3000)
    a = [t.to(cuda) for t in (x, ids, wts, w13, w2)]
    _, saved = bm.bi_moe_forward_train(*a)
    got = bm.bi_moe_backward(dout.to(cuda), *a[1:], saved, need=(False, True, False, False))[1]
    want = ref.experts(x, ids, wts, w13, w2, dout)[0]["dwts"]
    rel = ref.rel_norm(got.cpu(), want)
    assert rel <= dwts_bound(H), f"{rel:.2e} (bound {dwts_bound(H):.2e})"


# groups of several hundred rows and more tiles than CTA pairs
@pytest.mark.parametrize("M,H,E,k,I", [(1500, 2304, 3, 2, 1152), (2100, 4096, 2, 2, 1152), (2100, 4224, 2, 2, 1152),
                                       (5000, 8320, 3, 1, 640)])
def test_wide_tiles(cuda, M, H, E, k, I):
    """The rows of a few tokens among many are those of the tokens alone, bit for bit (a group of few rows has tiles of
    32 columns, a CTA pair one of them), and theirs by the formulas."""
    import invariant_moe_gb300 as bm
    x, ids, wts, w13, w2, dout = make(M, H, E, k, I, 3100)
    a = [t.to(cuda) for t in (x, ids, wts, w13, w2)]
    gd = dout.to(cuda)
    out, saved = bm.bi_moe_forward_train(*a)
    dx, dwts = bm.bi_moe_backward(gd, *a[1:], saved, need=(True, True, False, False))[:2]
    for beg, end in ((0, 1), (M // 2 - 9, M // 2 + 8), (M - 40, M)):
        s = slice(beg, end)
        o, sv = bm.bi_moe_forward_train(*(t[s] for t in a[:3]), *a[3:])
        d = bm.bi_moe_backward(gd[s], *(t[s] for t in a[1:3]), *a[3:], sv, need=(True, True, False, False))
        assert torch.equal(o, out[s]) and torch.equal(d[0], dx[s]) and torch.equal(d[1], dwts[s])
        r, b = ref.experts(x[s], ids[s], wts[s], w13, w2, dout[s])
        ref.check("out", o, r["out"], b["out"], None, 2)
        ref.check("dx", d[0], r["dx"], b["dx"], None, 2)
        ref.check("dwts", d[1], r["dwts"], b["dwts"], 2.0 ** -24)
        if end - beg > 8:
            rel = ref.rel_norm(d[1].cpu(), r["dwts"])
            assert rel <= dwts_bound(H), f"{rel:.2e}"
