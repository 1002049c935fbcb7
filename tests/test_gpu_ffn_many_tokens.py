"""Weight gradients over very many tokens (bi_ffn_backward) on a GPU.

Bound.  A slice of 1024 tokens is one fp32 chain in tensor memory, off by at
most 1024 * 2^-23 of the sum of its products' magnitudes (whether its additions
round or truncate); the slices are added to nearest in fp32, each addition off
by at most 2^-24 of what has been added up, so n slices give n * 2^-24.
The operands of the sums are taken as the call has them, act from
bi_ffn_forward_train and dg, du from the workspace, so that only the reduction
over the tokens is measured."""
import pytest
import torch

from tests import synthetic as syn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
SLICE = 1024


def bound(M):
    return min(SLICE, M) * 2.0 ** -23 + -(-M // SLICE) * 2.0 ** -24


def positive(M, N, seed):
    return syn.normal((M, N), 1.0, seed, device="cuda").abs().add_(0.25).to(BF)


def product64(a, b):
    """a^T b in fp64, a chunk of rows at a time."""
    r = torch.zeros(a.shape[1], b.shape[1], dtype=torch.float64, device=a.device)
    for i in range(0, a.shape[0], 1 << 16):
        r += a[i:i + (1 << 16)].double().T @ b[i:i + (1 << 16)].double()
    return r


@pytest.mark.parametrize("M", [1000, 1025, 5000, 100_003, 1 << 20])
def test_dw2_of_many_tokens(cuda, M):
    """fp32 dW2 = dout^T act of one sign, where every step's error adds up: within the bound of slices."""
    import invariant_moe_gb300 as bm
    H, I = 64, 32
    x, dout = positive(M, H, 1), positive(M, H, 2)
    w13, w2 = positive(2 * I, H, 3) / 64, positive(H, I, 4)
    _, gu, act = bm.bi_ffn_forward_train(x, w13, w2)
    assert bool((act > 0).all())
    d2 = torch.empty(H, I, device=cuda)
    bm.bi_ffn_backward(dout, x, w13, w2, gu, act, dw2=d2, need=(False, False, True))
    ref = product64(dout, act)
    err = float(((d2.double() - ref) / ref).abs().max())
    assert err <= bound(M), err


@pytest.mark.parametrize("M", [5000, 1 << 20])
def test_dw13_of_many_tokens(cuda, M):
    """fp32 dW13 likewise, against dg and du as the call left them in its workspace."""
    import invariant_moe_gb300 as bm
    H, I = 64, 32
    x, dout = positive(M, H, 5), positive(M, H, 6)
    w13, w2 = positive(2 * I, H, 7) / 64, positive(H, I, 8)
    _, gu, act = bm.bi_ffn_forward_train(x, w13, w2)
    d13 = torch.empty(2 * I, H, device=cuda)
    ws = bm.ffn_workspace(M, H, I, cuda)
    bm.bi_ffn_backward(dout, x, w13, w2, gu, act, dw13=d13, need=(False, True, False), workspace=ws)
    dgu = ws[:M * 2 * I * 2].view(BF).view(M, 2 * I)
    assert bool((dgu > 0).all())
    ref = product64(dgu, x)
    err = float(((d13.double() - ref) / ref).abs().max())
    assert err <= bound(M), err


def test_accumulated_over_micro_batches(cuda):
    """The same tokens in one call and added up over calls of whole slices: one fp32 addition apart at each."""
    import invariant_moe_gb300 as bm
    M, H, I, n = 8192, 80, 48, 4
    x, dout = positive(M, H, 9), positive(M, H, 10)
    w13, w2 = positive(2 * I, H, 11) / 64, positive(H, I, 12)
    _, gu, act = bm.bi_ffn_forward_train(x, w13, w2)
    one13, one2 = torch.empty(2 * I, H, device=cuda), torch.empty(H, I, device=cuda)
    bm.bi_ffn_backward(dout, x, w13, w2, gu, act, dw13=one13, dw2=one2, need=(False, True, True))
    d13, d2 = torch.zeros_like(one13), torch.zeros_like(one2)
    for i in range(n):
        s = slice(i * M // n, (i + 1) * M // n)
        bm.bi_ffn_backward(dout[s], x[s], w13, w2, gu[s], act[s], dw13=d13, dw2=d2, need=(False, True, True),
                           accumulate=True)
    for a, b in ((d13, one13), (d2, one2)):
        assert float(((a.double() - b.double()) / b.double()).abs().max()) <= (M // SLICE + n) * 2.0 ** -24
