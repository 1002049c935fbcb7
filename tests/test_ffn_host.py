"""Gated feed-forward block and 4-bit operators: host argument checks, layout
helpers and the 64-bit reference itself (no GPU)."""
import ctypes

import pytest
import torch

from tests import ffn_reference as ref

NUL = ctypes.c_void_p(None)
FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    from invariant_moe_gb300 import _build
    _build.build()
    import invariant_moe_gb300 as bm
    return bm.load_library()


def test_workspace_and_scale_bytes(lib):
    assert lib.bi_ffn_workspace_bytes(100, 64, 32) >= 100 * 64 * 2
    assert lib.bi_ffn_workspace_bytes(100, 64, 32) % 256 == 0
    assert lib.bi_ffn_workspace_bytes(0, 64, 32) == 256
    for bad in ((-1, 64, 32), (1, 0, 32), (1, 64, 24), (1, 72, 32), (1, 64, 1 << 21)):
        assert lib.bi_ffn_workspace_bytes(*bad) == 0
    assert lib.bi_mx4_scale_bytes(1, 32) == 512
    assert lib.bi_mx4_scale_bytes(129, 160) == 4 * 512
    assert lib.bi_mx4_scale_bytes(0, 32) == 0 and lib.bi_mx4_scale_bytes(4, 40) == 0


def fwd(lib, x=FAKE, ldx=64, w13=FAKE, w2=FAKE, add=NUL, lda=0, out=FAKE, ldo=64, M=4, H=64, I=32, ws=FAKE, n=1 << 20):
    return lib.bi_ffn_forward(x, ldx, w13, w2, add, lda, out, ldo, M, H, I, ws, n, NUL)


def test_forward_checks(lib):
    assert fwd(lib, M=0, x=NUL, out=NUL, ws=NUL) == 0
    assert fwd(lib, M=-1) == 1 and fwd(lib, H=0) == 1
    assert fwd(lib, H=72, ldx=72, ldo=72) == 2 and fwd(lib, I=40) == 2 and fwd(lib, M=1 << 31) == 2
    for bad in ({"x": NUL}, {"out": NUL}, {"w13": NUL}, {"w2": NUL}, {"x": ODD}, {"w13": ODD}, {"w2": ODD},
                {"out": ODD}, {"ldx": 56}, {"ldx": 68}, {"ldo": 68}, {"add": FAKE, "lda": 32}, {"add": ODD, "lda": 64},
                {"ws": NUL}, {"ws": ODD}):
        assert fwd(lib, **bad) == 1, bad
    assert fwd(lib, n=255) == 3


def test_train_and_backward_checks(lib):
    t = lambda gu, act: lib.bi_ffn_forward_train(FAKE, 64, FAKE, FAKE, NUL, 0, FAKE, 64, gu, act, 4, 64, 32, NUL)
    assert t(NUL, FAKE) == 1 and t(FAKE, NUL) == 1 and t(ODD, FAKE) == 1

    def bwd(dout=FAKE, lddo=64, x=FAKE, w13=FAKE, w2=FAKE, gu=FAKE, act=FAKE, dx=FAKE, lddx=64, d13=FAKE, d2=FAKE,
            mode=0, M=4, ws=FAKE, n=1 << 20):
        return lib.bi_ffn_backward(dout, lddo, x, 64, w13, w2, gu, act, dx, lddx, d13, d2, mode, M, 64, 32, ws, n, NUL)

    assert bwd(dx=NUL, d13=NUL, d2=NUL) == 0
    assert bwd(M=0, d13=NUL, d2=NUL) == 0
    for bad in ({"mode": 3}, {"mode": -1}, {"dout": NUL}, {"dout": ODD}, {"lddo": 60}, {"x": NUL}, {"w2": NUL},
                {"gu": NUL}, {"w13": NUL}, {"act": NUL}, {"lddx": 8}, {"d13": ODD}, {"d2": ODD}, {"ws": NUL}):
        assert bwd(**bad) == 1, bad
    assert bwd(n=511) == 3


def test_mx4_checks(lib):
    q = lambda x=FAKE, ldx=64, c=FAKE, s=FAKE, R=4, K=64: lib.bi_mx4_quantize(x, 0, ldx, c, s, R, K, NUL)
    assert q(R=0, x=NUL) == 0 and q(K=48) == 2 and q(K=0) == 1 and q(R=-1) == 1
    assert q(x=ODD) == 1 and q(ldx=60) == 1 and q(c=NUL) == 1 and q(s=ODD) == 1
    d = lambda y=FAKE, ldy=64, R=4: lib.bi_mx4_dequantize(FAKE, FAKE, y, 1, ldy, R, 64, NUL)
    assert d(R=0, y=NUL) == 0 and d(y=NUL) == 1 and d(ldy=32) == 1

    def g(xq=FAKE, ws=FAKE, add=NUL, lda=0, y=FAKE, ldy=9, M=4, N=9, K=64):
        return lib.bi_mx4_gemm(xq, FAKE, FAKE, ws, add, lda, y, ldy, M, N, K, NUL)

    assert g(M=0, xq=NUL) == 0 and g(K=40) == 2 and g(N=0) == 1 and g(ldy=8) == 1 and g(y=NUL) == 1
    assert g(xq=ODD) == 1 and g(ws=ODD) == 1 and g(add=FAKE, lda=8) == 1 and g(N=1 << 23, ldy=1 << 23) == 2
    u = lambda I: lib.bi_mx4_gate_up(FAKE, FAKE, FAKE, FAKE, FAKE, I, 4, I, 64, NUL)
    assert u(0) == 1 and u(24) == 2


def test_layout_helpers():
    import invariant_moe_gb300 as bm
    g = torch.Generator().manual_seed(1)
    for R, K in ((1, 32), (130, 160), (256, 512)):
        s = torch.randint(0, 255, (R, K // 32), generator=g, dtype=torch.uint8)
        t = bm.mx4_tile_scales(s)
        assert tuple(t.shape) == bm.mx4_scale_shape(R, K)
        assert torch.equal(t, ref.tile_scales(s)) and torch.equal(bm.mx4_untile_scales(t, R, K), s)
    I = 48
    w = torch.arange(2 * I)[:, None].expand(2 * I, 3)
    o = bm.mx4_interleave_gate_up(w)[:, 0]
    for r in range(2 * I):
        j, i = divmod(r, 32)
        assert int(o[r]) == (16 * j + i if i < 16 else I + 16 * j + i - 16)
    with pytest.raises(ValueError):
        bm.mx4_interleave_gate_up(torch.zeros(24, 2))


def test_reference_gradient_is_autograds():
    """The 64-bit backward formulas against automatic differentiation and against differences."""
    g = torch.Generator().manual_seed(2)
    M, H, I = 5, 16, 16
    x, w13, w2, dout = (torch.randn(s, generator=g, dtype=torch.float64)
                        for s in ((M, H), (2 * I, H), (H, I), (M, H)))
    r = ref.ffn(x, w13, w2, dout=dout)
    leaves = [t.clone().requires_grad_() for t in (x, w13, w2)]
    a, b, c = leaves
    out = (torch.nn.functional.silu(a @ b[:I].T) * (a @ b[I:].T)) @ c.T
    out.backward(dout)
    for name, t in zip(("dx", "dw13", "dw2"), leaves):
        assert torch.allclose(r[name], t.grad, rtol=1e-10, atol=1e-10)
    h = 1e-6
    e = torch.zeros_like(x)
    e[2, 3] = h
    slope = ((ref.ffn(x + e, w13, w2)["out"] - ref.ffn(x - e, w13, w2)["out"]) * dout).sum() / (2 * h)
    assert abs(float(slope - r["dx"][2, 3])) < 1e-6


def test_reference_quantisation():
    """Codes and scales of hand-worked blocks."""
    x = torch.zeros(1, 32)
    x[0, :8] = torch.tensor([6.0, -3.5, 2.5, 1.25, 0.75, 0.25, 5.0, -0.25])
    c, s = ref.mx4_quantize(x)
    assert int(s) == 127                       # 6 = 1.5 * 2^2: scale 2^0
    assert c[0, :8].tolist() == [7, 14, 4, 2, 2, 0, 6, 8]
    x[0, 0] = 7.5                              # above 6 times the scale: saturates
    c, s = ref.mx4_quantize(x)
    assert int(s) == 127 and int(c[0, 0]) == 7
    x[0, 0] = 8.0
    c, s = ref.mx4_quantize(x)
    assert int(s) == 128 and int(c[0, 0]) == 6
    c, s = ref.mx4_quantize(torch.zeros(1, 32))
    assert int(s) == 0 and not c.any()
    assert torch.isnan(ref.mx4_values(*ref.mx4_quantize(torch.full((1, 32), float("nan"))))).all()
