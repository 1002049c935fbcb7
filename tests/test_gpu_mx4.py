"""Microscaled 4-bit operators (bi_mx4_quantize / _dequantize / _gemm /
_gate_up) on a GPU against the 64-bit definition."""
import math

import pytest
import torch

from tests import ffn_reference as ref
from tests import synthetic as syn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def special_rows(K):
    """Blocks of every kind: zeros, signed zeros, ties, one large value, subnormals, the largest values."""
    x = torch.zeros(12, K)
    x[1] = -0.0
    x[2] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9, -0.25, -0.75, -2.5, -5.0, -7.0, 4.0]
                        ).repeat(K // 16)
    x[3, 5::32] = 3.0e38
    x[4] = 2.0 ** -126
    x[5] = 2.0 ** -133 * torch.arange(K).remainder(8)
    x[6] = syn.normal((K,), 1.0, 5) * 2.0 ** -120
    x[7] = syn.normal((K,), 1.0, 6) * 2.0 ** 120
    x[8] = syn.normal((K,), 1.0, 7)
    x[8, 3::32] = 1000.0
    x[9] = 1.0
    x[10] = 2.0 ** -124 * 1.5
    x[11] = -2.0 ** 127
    return x


def check_quant(bm, x, cuda):
    codes, s = ref.mx4_quantize(x)
    q, t = bm.bi_mx4_quantize(x.to(cuda))
    assert torch.equal(t.cpu(), ref.tile_scales(s)), "scales"
    assert torch.equal(q.cpu(), ref.mx4_pack(codes)), "codes"
    assert torch.equal(bm.mx4_untile_scales(t, *x.shape).cpu(), s)
    v = ref.mx4_values(codes, s)
    for dt in (torch.float32, BF):
        y = bm.bi_mx4_dequantize(q, t, dtype=dt).double().cpu()
        assert torch.equal(torch.isnan(y), torch.isnan(v))
        fine = ~torch.isnan(v)
        assert torch.equal(y[fine], v[fine])
        assert torch.equal(torch.signbit(y[fine]), torch.signbit(v[fine]))


@pytest.mark.parametrize("R,K", [(1, 32), (1, 4096), (3, 96), (31, 160), (127, 128), (128, 2080), (129, 512),
                                 (300, 1024), (257, 32)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_quantize(cuda, R, K, dtype):
    import invariant_moe_gb300 as bm
    x = syn.normal((R, K), 1.0, R + K)
    x[:, ::37] *= 40.0
    check_quant(bm, x.to(dtype), cuda)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_quantize_special_values(cuda, dtype):
    import invariant_moe_gb300 as bm
    x = special_rows(192).to(dtype)
    check_quant(bm, x, cuda)
    for bad in (math.nan, math.inf, -math.inf):
        y = x.clone()
        y[8, 40] = bad
        y[0, 191] = bad
        check_quant(bm, y, cuda)


def test_quantize_strides_and_guards(cuda):
    import invariant_moe_gb300 as bm
    R, K = 37, 96
    for dt in (BF, torch.float32):
        w = syn.normal((R, K + 40), 1.0, 3, dt).to(cuda)
        v = w[:, 8:8 + K]
        q, t = bm.bi_mx4_quantize(v)
        q2, t2 = bm.bi_mx4_quantize(v.contiguous())
        assert torch.equal(q, q2) and torch.equal(t, t2)
        fq = torch.full((R * K // 2 + 64,), 99, dtype=torch.uint8, device=cuda)
        ft = torch.full((t.numel() + 64,), 99, dtype=torch.uint8, device=cuda)
        bm.bi_mx4_quantize(v, q=fq[:R * K // 2].view(R, K // 2), scales=ft[:t.numel()].view(t.shape))
        assert torch.equal(fq[:R * K // 2].view(R, K // 2), q) and torch.equal(ft[:t.numel()].view(t.shape), t)
        assert bool((fq[-64:] == 99).all()) and bool((ft[-64:] == 99).all())
        out = torch.full((R + 2, K + 16), float("nan"), dtype=dt, device=cuda)
        bm.bi_mx4_dequantize(q, t, out=out[1:1 + R, 8:8 + K])
        assert torch.equal(out[1:1 + R, 8:8 + K], bm.bi_mx4_dequantize(q, t, dtype=dt))
        assert int(torch.isnan(out).sum()) == out.numel() - R * K


def quantized(R, K, std, seed, cuda):
    import invariant_moe_gb300 as bm
    x = syn.normal((R, K), std, seed)
    x[:, ::61] *= 16.0
    c, s = ref.mx4_quantize(x)
    return ref.mx4_values(c, s), ref.mx4_pack(c).to(cuda), ref.tile_scales(s).to(cuda)


def check(got, want, bound, name):
    got = got.double().cpu()
    d = (got - want).abs()
    assert bool((d <= bound).all()), f"{name}: {float((d - bound).max()):.3e} over its bound"
    assert ref.rel_norm(got, want) <= ref.norm_bound(1), name


# tokens, features, K: one token, tile edges on every side, odd features, K
# that ends inside a 256-, 128- and 64-value step
GEMM = [(1, 1, 32), (1, 4096, 2048), (2, 17, 64), (5, 1001, 2080), (31, 128, 96), (33, 129, 224), (64, 255, 256),
        (127, 384, 288), (129, 127, 512), (200, 513, 1120), (257, 300, 160), (300, 1000, 4096),
        # enough tiles for CTA pairs, each token tile width, ragged on both sides
        (1100, 2100, 288), (641, 3001, 1056), (2000, 1290, 640), (4100, 600, 96), (385, 4700, 32)]


@pytest.mark.parametrize("M,N,K", GEMM)
@pytest.mark.parametrize("with_addend", [False, True])
def test_gemm(cuda, M, N, K, with_addend):
    import invariant_moe_gb300 as bm
    xv, xq, xs = quantized(M, K, 1.0, 1, cuda)
    wv, wq, ws = quantized(N, K, K ** -0.5, 2, cuda)
    add = syn.normal((M, N), 0.5, 3, BF) if with_addend else None
    y, b = ref.mx4_product(xv, wv, add)
    got = bm.bi_mx4_gemm(xq, xs, wq, ws, addend=None if add is None else add.to(cuda))
    check(got, y, b, "y")


@pytest.mark.parametrize("M,I,K", [(1, 16, 32), (1, 2048, 4096), (3, 48, 160), (33, 768, 2048), (64, 64, 256),
                                   (130, 336, 416), (257, 128, 1024), (300, 272, 2080), (1030, 1120, 544),
                                   (700, 1520, 288)])
def test_gate_up(cuda, M, I, K):
    import invariant_moe_gb300 as bm
    xv, xq, xs = quantized(M, K, 1.0, 11, cuda)
    wv, wq, ws = quantized(2 * I, K, K ** -0.5, 12, cuda)
    y, b = ref.mx4_gated(xv, wv)
    check(bm.bi_mx4_gate_up(xq, xs, wq, ws), y, b, "act")


def test_interleaved_gate_up_is_the_block(cuda):
    """Quantising the interleaved rows gives the gate and up projections of the plain layout."""
    import invariant_moe_gb300 as bm
    M, I, K = 20, 48, 128
    w13 = syn.normal((2 * I, K), K ** -0.5, 21, BF).to(cuda)
    x = syn.normal((M, K), 1.0, 22, BF).to(cuda)
    xq, xs = bm.bi_mx4_quantize(x)
    act = bm.bi_mx4_gate_up(xq, xs, *bm.bi_mx4_quantize(bm.mx4_interleave_gate_up(w13)))
    xv, wv = (bm.bi_mx4_dequantize(*bm.bi_mx4_quantize(t), dtype=torch.float32).double().cpu() for t in (x, w13))
    g, u = xv @ wv[:I].T, xv @ wv[I:].T
    want = ref.silu(g) * u
    assert ref.rel_norm(act.cpu(), want) <= ref.norm_bound(1)


def test_rows_do_not_depend_on_the_batch(cuda):
    import invariant_moe_gb300 as bm
    M, N, K = 1100, 1001, 2080
    x = syn.normal((M, K), 1.0, 31, BF).to(cuda)
    wq, ws = bm.bi_mx4_quantize(syn.normal((N, K), K ** -0.5, 32, BF).to(cuda))
    gq, gs = bm.bi_mx4_quantize(syn.normal((2 * 336, K), K ** -0.5, 33, BF).to(cuda))
    xq, xs = bm.bi_mx4_quantize(x)
    y, act = bm.bi_mx4_gemm(xq, xs, wq, ws), bm.bi_mx4_gate_up(xq, xs, gq, gs)
    # (a matrix of 9000 more rows takes other tiles: CTA pairs)
    big = torch.cat((x, syn.normal((9000, K), 1.0, 34, BF).to(cuda)))
    bq, bs = bm.bi_mx4_quantize(big)
    assert torch.equal(bm.bi_mx4_gemm(bq, bs, wq, ws)[:M], y)
    assert torch.equal(bm.bi_mx4_gate_up(bq, bs, gq, gs)[:M], act)
    for a, n in ((0, 1), (3, 2), (9, 7), (100, 8), (1, 9), (31, 32), (64, 33), (200, 64), (77, 65), (5, 128),
                 (300, 129), (2, 257), (500, 600)):
        sq, ss = bm.bi_mx4_quantize(x[a:a + n])
        assert torch.equal(sq, xq[a:a + n])
        assert torch.equal(bm.bi_mx4_gemm(sq, ss, wq, ws), y[a:a + n]), (a, n)
        assert torch.equal(bm.bi_mx4_gate_up(sq, ss, gq, gs), act[a:a + n]), (a, n)


def test_gemm_strides_guards_and_in_place(cuda):
    import invariant_moe_gb300 as bm
    for M, N in ((1, 33), (70, 129), (300, 161)):
        _, xq, xs = quantized(M, 256, 1.0, 41, cuda)
        _, wq, ws = quantized(N, 256, 0.1, 42, cuda)
        add = syn.normal((M, N), 0.5, 43, BF).to(cuda)
        y = bm.bi_mx4_gemm(xq, xs, wq, ws, addend=add)
        w = torch.full((M + 2, N + 5), float("nan"), dtype=BF, device=cuda)
        bm.bi_mx4_gemm(xq, xs, wq, ws, addend=add, out=w[1:1 + M, 3:3 + N])
        assert torch.equal(w[1:1 + M, 3:3 + N], y) and int(torch.isnan(w).sum()) == w.numel() - M * N
        z = add.clone()
        bm.bi_mx4_gemm(xq, xs, wq, ws, addend=z, out=z)
        assert torch.equal(z, y)


def test_nan_scales_and_extremes(cuda):
    """A NaN block spoils its own row (column) and nothing else; the largest and smallest scales multiply exactly."""
    import invariant_moe_gb300 as bm
    M, N, K = 40, 150, 192
    x, w = syn.normal((M, K), 1.0, 51), syn.normal((N, K), 0.1, 52)
    y = bm.bi_mx4_gemm(*bm.bi_mx4_quantize(x.to(cuda)), *bm.bi_mx4_quantize(w.to(cuda)))
    x2, w2 = x.clone(), w.clone()
    x2[7, 100], w2[131, 3] = math.nan, math.inf
    z = bm.bi_mx4_gemm(*bm.bi_mx4_quantize(x2.to(cuda)), *bm.bi_mx4_quantize(w2.to(cuda)))
    nan = torch.zeros(M, N, dtype=torch.bool)
    nan[7], nan[:, 131] = True, True
    assert torch.equal(torch.isnan(z).cpu(), nan)
    assert torch.equal(z.cpu()[~nan], y.cpu()[~nan])
    for ex, ew in ((100, -100), (-120, 110), (60, 60), (-60, -50)):
        z = bm.bi_mx4_gemm(*bm.bi_mx4_quantize((x * 2.0 ** ex).to(cuda)), *bm.bi_mx4_quantize((w * 2.0 ** ew).to(cuda)))
        assert torch.equal(z.double().cpu() * 2.0 ** -(ex + ew), y.double().cpu()), (ex, ew)


def test_empty_streams_and_graph(cuda):
    import invariant_moe_gb300 as bm
    N, K = 130, 160
    wq, ws = bm.bi_mx4_quantize(syn.normal((N, K), 0.1, 61, BF).to(cuda))
    q, s = bm.bi_mx4_quantize(torch.empty(0, K, dtype=BF, device=cuda))
    assert bm.bi_mx4_gemm(q, s, wq, ws).shape == (0, N) and bm.bi_mx4_dequantize(q, s).shape == (0, K)
    x = syn.normal((50, K), 1.0, 62, BF).to(cuda)
    want = bm.bi_mx4_gemm(*bm.bi_mx4_quantize(x), wq, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = bm.bi_mx4_gemm(*bm.bi_mx4_quantize(x), wq, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    q, s = bm.mx4_empty(50, K, cuda)
    y = torch.empty(50, N, dtype=BF, device=cuda)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bm.bi_mx4_gemm(*bm.bi_mx4_quantize(x, q=q, scales=s), wq, ws, out=y)
    y.zero_()
    g.replay()
    assert torch.equal(y, want)


def test_refusals(cuda):
    import invariant_moe_gb300 as bm
    x = torch.zeros(4, 64, dtype=BF, device=cuda)
    q, s = bm.bi_mx4_quantize(x)
    with pytest.raises(ValueError):
        bm.bi_mx4_quantize(torch.zeros(4, 40, dtype=BF, device=cuda))
    with pytest.raises(TypeError):
        bm.bi_mx4_quantize(x.half())
    with pytest.raises(ValueError):
        bm.bi_mx4_quantize(x.cpu())
    with pytest.raises(ValueError):
        bm.bi_mx4_gemm(q, s, q, s[:, :, :256])
    with pytest.raises(ValueError):
        bm.bi_mx4_gemm(q, s, *bm.bi_mx4_quantize(torch.zeros(4, 96, dtype=BF, device=cuda)))
    with pytest.raises(ValueError):
        bm.bi_mx4_gate_up(q, s, *bm.bi_mx4_quantize(torch.zeros(24, 64, dtype=BF, device=cuda)))
    with pytest.raises(TypeError):
        bm.bi_mx4_gemm(q, s, q, s, out=torch.zeros(4, 4, device=cuda))
    big = torch.zeros(4, 72, dtype=BF, device=cuda)
    with pytest.raises(bm.BimoeError) as e:
        bm.bi_mx4_quantize(big[:, 4:68])
    assert e.value.status == 1


def test_offsets_past_32_bits(cuda):
    """More than 2^32 values: the last rows are those of a small call."""
    import invariant_moe_gb300 as bm
    R, K, N, n = (1 << 20) + 200, 4128, 2064, 130
    x = syn.normal((R // 8, K), 1.0, 71, BF, device="cuda").repeat(8, 1)
    x = torch.cat((x, syn.normal((R - x.shape[0], K), 1.0, 72, BF, device="cuda"))) if x.shape[0] < R else x
    x[-n:] = syn.normal((n, K), 1.0, 73, BF).to(cuda)
    assert x.numel() > 1 << 32
    q, s = bm.bi_mx4_quantize(x)
    q2, s2 = bm.bi_mx4_quantize(x[-n:])
    assert torch.equal(q[-n:], q2)
    y = bm.bi_mx4_dequantize(q, s, out=x)
    assert torch.equal(y[-n:], bm.bi_mx4_dequantize(q2, s2))
    del x, y
    wq, ws = bm.bi_mx4_quantize(syn.normal((N, K), K ** -0.5, 74, BF).to(cuda))
    z = bm.bi_mx4_gemm(q, s, wq, ws)
    assert z.numel() > 1 << 31
    assert torch.equal(z[-n:], bm.bi_mx4_gemm(q2, s2, wq, ws))
