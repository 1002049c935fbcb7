"""The three forms of the 4-bit product (single CTAs, CTA pairs of 192 and of 256
tokens a tile) on a GPU: each within the 64-bit bound, all of the same bits."""
import ctypes

import pytest
import torch

from tests import ffn_reference as ref
from tests import synthetic as syn

BF = torch.bfloat16
FORMS = (1, 2, 3)


@pytest.fixture
def form():
    """Sets the form; the test leaves it automatic."""
    import invariant_moe_gb300 as bm
    yield bm.bi_mx4_form
    bm.bi_mx4_form(0)


def test_form_argument():
    from invariant_moe_gb300 import _build
    _build.build()
    import invariant_moe_gb300 as bm
    lib = bm.load_library()
    prev = ctypes.c_int32(9)
    assert lib.bi_mx4_form(-1, ctypes.byref(prev)) == 1 and lib.bi_mx4_form(4, None) == 1 and prev.value == 9
    assert bm.bi_mx4_form(3) == 0 and bm.bi_mx4_form(0) == 3 and lib.bi_mx4_form(0, None) == 0


def quantized(R, K, std, seed, cuda):
    x = syn.normal((R, K), std, seed)
    x[:, ::61] *= 16.0
    c, s = ref.mx4_quantize(x)
    return ref.mx4_values(c, s).to(cuda), ref.mx4_pack(c).to(cuda), ref.tile_scales(s).to(cuda)


def check(got, want, bound, name):
    d = (got.double() - want).abs()
    assert bool((d <= bound).all()), f"{name}: {float((d - bound).max()):.3e} over its bound"
    assert ref.rel_norm(got, want) <= ref.norm_bound(1), name


# tokens, features, K: fewer than a tile of either side, a token past each tile
# width (and its half, a CTA's share), odd features, K that ends inside a step,
# several tiles a CTA pair, and reductions longer than the ring of stages
SHAPES = [(1, 1, 32), (1, 300, 2080), (17, 129, 96), (95, 255, 160), (97, 257, 224), (128, 256, 256),
          (129, 513, 1120), (191, 128, 288), (193, 300, 64), (256, 640, 4128), (257, 1001, 2080), (385, 127, 352),
          (449, 200, 96), (600, 700, 3104), (5000, 1300, 96), (2500, 2100, 4128)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(cuda, form, M, N, K):
    import invariant_moe_gb300 as bm
    xv, xq, xs = quantized(M, K, 1.0, 1, cuda)
    wv, wq, ws = quantized(N, K, K ** -0.5, 2, cuda)
    add = syn.normal((M, N), 0.5, 3, BF).to(cuda)
    plain, b = ref.mx4_product(xv, wv)
    added, ba = ref.mx4_product(xv, wv, add)
    first = None
    for f in FORMS:
        form(f)
        y, z = bm.bi_mx4_gemm(xq, xs, wq, ws), bm.bi_mx4_gemm(xq, xs, wq, ws, addend=add)
        check(y, plain, b, f"form {f}")
        check(z, added, ba, f"form {f}, addend")
        # in place, and rows of odd strides and addresses with guards on every side
        p = add.clone()
        bm.bi_mx4_gemm(xq, xs, wq, ws, addend=p, out=p)
        assert torch.equal(p, z)
        w = torch.full((M + 2, N + 5), float("nan"), dtype=BF, device=cuda)
        a = torch.full((M, N + 3), float("nan"), dtype=BF, device=cuda)[:, 1:1 + N].copy_(add)
        bm.bi_mx4_gemm(xq, xs, wq, ws, addend=a, out=w[1:1 + M, 3:3 + N])
        assert torch.equal(w[1:1 + M, 3:3 + N], z) and int(torch.isnan(w).sum()) == w.numel() - M * N
        first = first or (y, z)
        assert torch.equal(y, first[0]) and torch.equal(z, first[1])


@pytest.mark.gpu
@pytest.mark.parametrize("M,I,K", [(1, 16, 32), (95, 128, 160), (193, 48, 288), (257, 528, 2080), (385, 272, 96),
                                   (700, 336, 4128), (5000, 656, 96), (2500, 1056, 3104)])
def test_gate_up(cuda, form, M, I, K):
    import invariant_moe_gb300 as bm
    xv, xq, xs = quantized(M, K, 1.0, 11, cuda)
    wv, wq, ws = quantized(2 * I, K, K ** -0.5, 12, cuda)
    f = torch.arange(I, device=cuda)
    rows = f // 16 * 32 + f % 16
    h, e = xv @ wv.T, K * ref.EPS32 * (xv.abs() @ wv.abs().T)
    g, u, eg, eu = h[:, rows], h[:, rows + 16], e[:, rows], e[:, rows + 16]
    want = ref.silu(g) * u
    pre = 1.1 * u.abs() * eg + ref.silu(g).abs() * eu + 1.1 * eg * eu + 16 * ref.EPS32 * want.abs()
    first = None
    for mode in FORMS:
        form(mode)
        y = bm.bi_mx4_gate_up(xq, xs, wq, ws)
        check(y, want, ref.U * want.abs() + (1 + ref.U) * pre, f"form {mode}")
        w = torch.full((M + 2, I + 5), float("nan"), dtype=BF, device=cuda)
        bm.bi_mx4_gate_up(xq, xs, wq, ws, out=w[1:1 + M, 3:3 + I])
        assert torch.equal(w[1:1 + M, 3:3 + I], y) and int(torch.isnan(w).sum()) == w.numel() - M * I
        first = y if first is None else first
        assert torch.equal(y, first)


@pytest.mark.gpu
def test_automatic_choice_has_the_same_bits(cuda, form):
    """Sizes on both sides of the rule, a NaN block among them."""
    import invariant_moe_gb300 as bm
    for M, N, K in ((40, 500, 160), (700, 8192, 544), (3001, 5001, 288), (8192, 2048, 96)):
        x, w = syn.normal((M, K), 1.0, 21, BF).to(cuda), syn.normal((N, K), K ** -0.5, 22, BF).to(cuda)
        x[M // 2, K - 1], w[N - 1, 0] = float("nan"), float("inf")
        x, w = bm.bi_mx4_quantize(x), bm.bi_mx4_quantize(w)
        form(0)
        want = bm.bi_mx4_gemm(*x, *w)
        assert bool(torch.isnan(want[M // 2]).all()) and bool(torch.isnan(want[:, N - 1]).all())
        assert int(torch.isnan(want).sum()) == M + N - 1
        for f in FORMS:
            form(f)
            assert torch.equal(torch.nan_to_num(bm.bi_mx4_gemm(*x, *w), nan=7e30), torch.nan_to_num(want, nan=7e30))
