"""dx of bi_ffn_backward over memory that the same launch still reads: refused
(host checks, no GPU), and where it reads nothing there any more: the same bits."""
import ctypes

import pytest
import torch

from tests import synthetic as syn

NUL = ctypes.c_void_p(None)
BF = torch.bfloat16
M, H, I = 4, 64, 32


@pytest.fixture(scope="module")
def lib():
    from invariant_moe_gb300 import _build
    _build.build()
    import invariant_moe_gb300 as bm
    return bm.load_library()


def backward(lib, dx, lddx, dout=0x10000, lddo=H, x=0x20000, ldx=H):
    """Status for made-up addresses, all of which the host refuses."""
    p = ctypes.c_void_p
    return lib.bi_ffn_backward(p(dout), lddo, p(x), ldx, p(0x30000), p(0x40000), p(0x50000), p(0x60000), p(dx), lddx,
                               p(0x80000), p(0x90000), 0, M, H, I, p(0x100000), 1 << 20, NUL)


def test_overlap_is_refused(lib):
    for base in (0x10000, 0x20000):
        assert backward(lib, base, H) == 1
        assert b"overlap" in lib.bi_last_error_message()
        assert backward(lib, base + 16, H) == 1 and backward(lib, base - 16, H) == 1
        assert backward(lib, base + (M - 1) * H * 2, H) == 1 and backward(lib, base - (M * H - 8) * 2, H) == 1
        assert backward(lib, base + 2 * H, 3 * H) == 1        # another row stride inside the same range
    # columns of one wider matrix that run into another's
    for off in (2 * H - 8, 4 * H + 8, -8, 2 * 3 * H + 3 * H - 8):
        assert backward(lib, 0x10000 + 2 * off, 3 * H, lddo=3 * H, x=0x10000 + 2 * H, ldx=3 * H) == 1, off


@pytest.mark.gpu
@pytest.mark.parametrize("m,h,i", [(1, 1040, 720), (40, 4096, 2048), (300, 272, 144)])
def test_dx_over_what_is_read_no_more(cuda, m, h, i):
    import invariant_moe_gb300 as bm
    x, dout = syn.normal((m, h), 1.0, 1, BF).to(cuda), syn.normal((m, h), 1.0, 2, BF).to(cuda)
    w13, w2 = syn.normal((2 * i, h), h ** -0.5, 3, BF).to(cuda), syn.normal((h, i), i ** -0.5, 4, BF).to(cuda)
    _, gu, act = bm.bi_ffn_forward_train(x, w13, w2)
    want = bm.bi_ffn_backward(dout, x, w13, w2, gu, act)
    for over, need in ((dout, (True, True, False)), (x, (True, False, True)), (x, (True, False, False))):
        for t, n in ((dout, 2), (x, 1)):
            if need[n]:
                with pytest.raises(bm.BimoeError, match="overlap"):
                    bm.bi_ffn_backward(dout, x, w13, w2, gu, act, dx=t, need=need)
        buf = over.clone()
        args = (buf, x) if over is dout else (dout, buf)
        got = bm.bi_ffn_backward(*args, w13, w2, gu, act, dx=buf, need=need)
        for a, b, n in zip(got, want, need):
            assert a is None if not n else torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 2, 70])
def test_dx_beside_what_is_read(cuda, m):
    """dx, dout and x as columns, or as rows, of one matrix do not overlap and are taken."""
    import invariant_moe_gb300 as bm
    h, i = 144, 80
    x, dout = syn.normal((m, h), 1.0, 1, BF).to(cuda), syn.normal((m, h), 1.0, 2, BF).to(cuda)
    w13, w2 = syn.normal((2 * i, h), h ** -0.5, 3, BF).to(cuda), syn.normal((h, i), i ** -0.5, 4, BF).to(cuda)
    _, gu, act = bm.bi_ffn_forward_train(x, w13, w2)
    want = bm.bi_ffn_backward(dout, x, w13, w2, gu, act)
    for order in ((0, 1, 2), (1, 2, 0), (2, 0, 1)):
        columns, rows = torch.zeros(m, 3 * h, dtype=BF, device=cuda), torch.zeros(3 * m, h, dtype=BF, device=cuda)
        for parts in ([columns[:, k * h:(k + 1) * h] for k in order], [rows[k * m:(k + 1) * m] for k in order]):
            d, a, g = parts
            d.copy_(dout), a.copy_(x)
            got = bm.bi_ffn_backward(d, a, w13, w2, gu, act, dx=g)
            assert all(torch.equal(p, q) for p, q in zip(got, want))
            assert torch.equal(d, dout) and torch.equal(a, x)
