"""Gated feed-forward block (bi_ffn_forward / _forward_train / _backward) on a
GPU against the 64-bit formulas, against differences, and against itself for
other batches, strides and streams."""
import pytest
import torch

from tests import ffn_reference as ref
from tests import synthetic as syn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16

# tokens, hidden, intermediate: one token, tile edges on each side of every
# tile size, sizes that are odd multiples of 16, both layer shapes' widths
SHAPES = [(1, 64, 16), (1, 4096, 2048), (2, 16, 48), (7, 2048, 768), (31, 272, 144), (33, 1040, 720),
          (64, 128, 128), (127, 1152, 80), (129, 512, 336), (255, 1024, 256), (300, 2064, 528)]


def make(M, H, I, seed, device="cuda"):
    x = syn.normal((M, H), 1.0, seed, BF)
    w13 = syn.normal((2 * I, H), H ** -0.5, seed + 1, BF)
    w2 = syn.normal((H, I), I ** -0.5, seed + 2, BF)
    add = syn.normal((M, H), 0.5, seed + 3, BF)
    dout = syn.normal((M, H), 1.0, seed + 4, BF)
    return x, w13, w2, add, dout


def check(name, got, r, b, roundings):
    got = got.detach().double().cpu()
    assert got.shape == r[name].shape
    d = (got - r[name]).abs()
    assert bool((d <= b[name]).all()), f"{name}: {float((d - b[name]).max()):.3e} over its bound"
    rel = ref.rel_norm(got, r[name])
    assert rel <= ref.norm_bound(roundings), f"{name}: 2-norm {rel:.3e}"


@pytest.mark.parametrize("M,H,I", SHAPES)
@pytest.mark.parametrize("with_addend", [False, True])
def test_forward(cuda, M, H, I, with_addend):
    import invariant_moe_gb300 as bm
    x, w13, w2, add, _ = make(M, H, I, 10)
    add = add if with_addend else None
    r = ref.ffn(x, w13, w2, add)
    b = ref.ffn_bounds(r, x, w13, w2, add)
    dx, d13, d2 = x.to(cuda), w13.to(cuda), w2.to(cuda)
    da = None if add is None else add.to(cuda)
    out = bm.bi_ffn_forward(dx, d13, d2, addend=da)
    check("out", out, r, b, 2)
    out_t, gu, act = bm.bi_ffn_forward_train(dx, d13, d2, addend=da)
    assert torch.equal(out_t, out), "training and inference differ"
    check("act", act, r, b, 1)
    g = gu.double().cpu()
    eg = H * ref.EPS32 * (x.double().abs() @ w13.double().abs().T)
    assert bool(((g - torch.cat((r["g"], r["u"]), 1)).abs() <= eg).all())


# few weight tiles and many tokens: a tile's tokens are shared by 2 or 4 CTA pairs
@pytest.mark.parametrize("M,H,I", SHAPES + [(1023, 272, 144), (2500, 144, 528), (4133, 512, 48)])
def test_backward(cuda, M, H, I):
    import invariant_moe_gb300 as bm
    x, w13, w2, _, dout = make(M, H, I, 30)
    r = ref.ffn(x, w13, w2, dout=dout)
    b = ref.ffn_bounds(r, x, w13, w2, dout=dout)
    dx_, d13, d2, dd = x.to(cuda), w13.to(cuda), w2.to(cuda), dout.to(cuda)
    _, gu, act = bm.bi_ffn_forward_train(dx_, d13, d2)
    dx, dw13, dw2 = bm.bi_ffn_backward(dd, dx_, d13, d2, gu, act)
    for name, t in (("dx", dx), ("dw13", dw13), ("dw2", dw2)):
        assert t.dtype == BF
        check(name, t, r, b, 2)
    # fp32 gradients: the same sums before their rounding, and added to what is there
    f13, f2 = torch.full_like(dw13, 3.0, dtype=torch.float32), torch.full_like(dw2, -2.0, dtype=torch.float32)
    bm.bi_ffn_backward(dd, dx_, d13, d2, gu, act, dx=dx, dw13=f13, dw2=f2)
    assert torch.equal(f13.to(BF), dw13) and torch.equal(f2.to(BF), dw2)
    a13, a2 = f13.clone(), f2.clone()
    bm.bi_ffn_backward(dd, dx_, d13, d2, gu, act, dx=dx, dw13=a13, dw2=a2, accumulate=True)
    assert torch.equal(a13, f13 + f13) and torch.equal(a2, f2 + f2)


@pytest.mark.parametrize("M,H,I", [(20, 160, 96), (70, 160, 96), (700, 1040, 720), (3000, 272, 144)])
def test_backward_parts(cuda, M, H, I):
    """Each gradient alone has the bits it has beside the others."""
    import invariant_moe_gb300 as bm
    x, w13, w2, _, dout = (t.to(cuda) for t in make(M, H, I, 50))
    _, gu, act = bm.bi_ffn_forward_train(x, w13, w2)
    full = bm.bi_ffn_backward(dout, x, w13, w2, gu, act)
    for i in range(3):
        need = tuple(j == i for j in range(3))
        part = bm.bi_ffn_backward(dout, x, w13, w2, gu, act, need=need)
        assert [p is not None for p in part] == list(need)
        assert torch.equal(part[i], full[i])
    assert bm.bi_ffn_backward(dout, x, w13, w2, gu, act, need=(False, False, False)) == (None, None, None)


def test_gradient_against_differences(cuda):
    """Along each gradient's own direction the 64-bit loss changes by its length."""
    import invariant_moe_gb300 as bm
    M, H, I = 37, 144, 112
    x, w13, w2, _, dout = make(M, H, I, 60)
    dev = [t.to(cuda) for t in (x, w13, w2)]
    _, gu, act = bm.bi_ffn_forward_train(*dev)
    grads = bm.bi_ffn_backward(dout.to(cuda), *dev, gu, act)
    args = [t.double() for t in (x, w13, w2)]
    h = 1e-4
    for i, gr in enumerate(grads):
        v = gr.double().cpu()
        v = v / v.norm()
        side = []
        for sgn in (1.0, -1.0):
            a = list(args)
            a[i] = a[i] + sgn * h * v
            side.append(float((ref.ffn(*a)["out"] * dout.double()).sum()))
        slope = (side[0] - side[1]) / (2 * h)
        length = float((gr.double().cpu() * v).sum())
        assert abs(slope - length) <= ref.norm_bound(2) * abs(length), (i, slope, length)


@pytest.mark.parametrize("H,I", [(1040, 336), (2048, 768), (4096, 128)])
def test_rows_do_not_depend_on_the_batch(cuda, H, I):
    """Bits of out and dx for a token alone, in ragged batches and in a large one."""
    import invariant_moe_gb300 as bm
    M = 1100
    x, w13, w2, add, dout = (t.to(cuda) for t in make(M, H, I, 70))
    out, gu, act = bm.bi_ffn_forward_train(x, w13, w2, addend=add)
    dx = bm.bi_ffn_backward(dout, x, w13, w2, gu, act, need=(True, False, False))[0]
    for a, n in ((0, 1), (5, 2), (17, 8), (3, 9), (100, 16), (64, 17), (7, 33), (1, 64), (130, 65), (0, 129),
                 (9, 256), (40, 257), (2, 513), (500, 600)):
        s = slice(a, a + n)
        o = bm.bi_ffn_forward(x[s], w13, w2, addend=add[s])
        assert torch.equal(o, out[s]), f"out rows {a}..{a + n}"
        o, g, ac = bm.bi_ffn_forward_train(x[s], w13, w2, addend=add[s])
        assert torch.equal(o, out[s]) and torch.equal(g, gu[s]) and torch.equal(ac, act[s])
        d = bm.bi_ffn_backward(dout[s], x[s], w13, w2, g, ac, need=(True, False, False))[0]
        assert torch.equal(d, dx[s]), f"dx rows {a}..{a + n}"


@pytest.mark.parametrize("M", [1, 45, 200])
def test_strides_and_guards(cuda, M):
    """Rows of wider tensors give the contiguous call's bits; nothing beside the results is written."""
    import invariant_moe_gb300 as bm
    H, I = 144, 80
    x, w13, w2, add, dout = (t.to(cuda) for t in make(M, H, I, 80))
    out, gu, act = bm.bi_ffn_forward_train(x, w13, w2, addend=add)
    grads = bm.bi_ffn_backward(dout, x, w13, w2, gu, act)

    def wide(t=None, rows=M, cols=H, dtype=BF):
        w = torch.full((rows + 4, cols + 24), float("nan"), dtype=dtype, device=cuda)
        v = w[2:2 + rows, 8:8 + cols]
        if t is not None:
            v.copy_(t)
        return w, v

    def untouched(w, v):
        keep = v.clone()
        v.fill_(float("nan"))
        ok = bool(torch.isnan(w).all())
        v.copy_(keep)
        return ok

    (_, xv), (_, av), (_, dv), (ow, ov), (gw, gv) = wide(x), wide(add), wide(dout), wide(), wide()
    bm.bi_ffn_forward(xv, w13, w2, addend=av, out=ov)
    assert torch.equal(ov, out) and untouched(ow, ov)
    # flat buffers with a guard behind each
    def flat(n, dtype):
        return torch.full((n + 64,), 77.0, dtype=dtype, device=cuda)
    fg, fa, f13, f2 = flat(M * 2 * I, torch.float32), flat(M * I, BF), flat(2 * I * H, BF), flat(H * I, BF)
    vg, va = fg[:M * 2 * I].view(M, 2 * I), fa[:M * I].view(M, I)
    v13, v2 = f13[:2 * I * H].view(2 * I, H), f2[:H * I].view(H, I)
    bm.bi_ffn_forward_train(xv, w13, w2, addend=av, out=ov, gu=vg, act=va)
    assert torch.equal(vg, gu) and torch.equal(va, act)
    bm.bi_ffn_backward(dv, xv, w13, w2, vg, va, dx=gv, dw13=v13, dw2=v2)
    assert torch.equal(gv, grads[0]) and torch.equal(v13, grads[1]) and torch.equal(v2, grads[2])
    assert untouched(gw, gv)
    for f in (fg, fa, f13, f2):
        assert bool((f[-64:] == 77.0).all())
    # out written over addend
    o2 = add.clone()
    bm.bi_ffn_forward(x, w13, w2, addend=o2, out=o2)
    assert torch.equal(o2, out)


def test_no_tokens(cuda):
    import invariant_moe_gb300 as bm
    H, I = 64, 32
    x, w13, w2, _, _ = (t.to(cuda) for t in make(4, H, I, 90))
    e = x[:0]
    out, gu, act = bm.bi_ffn_forward_train(e, w13, w2)
    assert bm.bi_ffn_forward(e, w13, w2).shape == (0, H) and out.shape == (0, H)
    for dt in (BF, torch.float32):
        d13, d2 = torch.full((2 * I, H), 5.0, dtype=dt, device=cuda), torch.full((H, I), 5.0, dtype=dt, device=cuda)
        dx, _, _ = bm.bi_ffn_backward(e, e, w13, w2, gu, act, dw13=d13, dw2=d2)
        assert dx.shape == (0, H) and not d13.any() and not d2.any()
    d13.fill_(5.0)
    bm.bi_ffn_backward(e, e, w13, w2, gu, act, dw13=d13, dw2=d2, accumulate=True)
    assert bool((d13 == 5.0).all())


def test_repeats_poisoned_workspace_and_stream(cuda):
    """Same bits on every call, whatever the workspace held, on another stream too."""
    import invariant_moe_gb300 as bm
    for M in (1, 19, 400):
        x, w13, w2, add, dout = (t.to(cuda) for t in make(M, 528, 304, 95))
        ws = bm.ffn_workspace(M, 528, 304, cuda)
        first = None
        side = torch.cuda.Stream()
        for i in range(6):
            ws.fill_(0xff)
            st = side if i % 2 else torch.cuda.current_stream()
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                out = bm.bi_ffn_forward(x, w13, w2, addend=add, workspace=ws)
                o, gu, act = bm.bi_ffn_forward_train(x, w13, w2, addend=add)
                g = bm.bi_ffn_backward(dout, x, w13, w2, gu, act, workspace=ws)
            torch.cuda.current_stream().wait_stream(st)
            got = (out, o, gu, act, *g)
            if first is None:
                first = [t.clone() for t in got]
            assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_extreme_gates(cuda):
    """Gates far on both sides: silu and its slope go to 0 and to g, with no NaN on the way."""
    import invariant_moe_gb300 as bm
    H, I, M = 16, 16, 8
    x = torch.zeros(M, H, dtype=BF)
    x[:, 0] = torch.tensor([0.0, 1.0, -1.0, 60.0, -60.0, 100.0, -100.0, -3000.0])
    w13 = torch.zeros(2 * I, H, dtype=BF)
    w13[:, 0] = 1.0
    w2 = torch.eye(H, I, dtype=BF)
    dout = torch.ones(M, H, dtype=BF)
    r = ref.ffn(x, w13, w2, dout=dout)
    b = ref.ffn_bounds(r, x, w13, w2, dout=dout)
    for k in r:  # exp(-g) overflows fp64's plain form at no value used here
        assert bool(torch.isfinite(r[k]).all()), k
    dev = [t.to(cuda) for t in (x, w13, w2)]
    out, gu, act = bm.bi_ffn_forward_train(*dev)
    dx, dw13, dw2 = bm.bi_ffn_backward(dout.to(cuda), *dev, gu, act)
    tiny = 1e-30  # fp32's exp may flush what is far below every other term
    for n, t in (("out", out), ("dx", dx), ("dw13", dw13), ("dw2", dw2)):
        d = (t.double().cpu() - r[n]).abs()
        assert bool((d <= b[n] + tiny).all()), (n, float((d - b[n]).max()))


def test_graph_capture(cuda):
    """Forward and backward replay from a CUDA graph with new inputs in the same buffers."""
    import invariant_moe_gb300 as bm
    M, H, I = 21, 272, 208
    x, w13, w2, add, dout = (t.to(cuda) for t in make(M, H, I, 97))
    ws = bm.ffn_workspace(M, H, I, cuda)
    gu, act = bm.ffn_saved(M, I, cuda)
    out, dx, d13, d2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w13), torch.empty_like(w2)

    def step():
        bm.bi_ffn_forward_train(x, w13, w2, addend=add, out=out, gu=gu, act=act)
        bm.bi_ffn_backward(dout, x, w13, w2, gu, act, dx=dx, dw13=d13, dw2=d2, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.copy_(make(M, H, I, 197)[0])
    g.replay()
    got = [t.clone() for t in (out, dx, d13, d2)]
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, (out, dx, d13, d2)))


def test_refusals(cuda):
    import invariant_moe_gb300 as bm
    x, w13, w2, add, dout = (t.to(cuda) for t in make(8, 64, 32, 99))
    with pytest.raises(TypeError):
        bm.bi_ffn_forward(x.float(), w13, w2)
    with pytest.raises(ValueError):
        bm.bi_ffn_forward(x.cpu(), w13, w2)
    with pytest.raises(ValueError):
        bm.bi_ffn_forward(x, w13[:60], w2)
    with pytest.raises(ValueError):
        bm.bi_ffn_forward(x.t().contiguous().t(), w13, w2)
    with pytest.raises(ValueError):
        bm.bi_ffn_forward(x, w13, w2, addend=add[:4])
    with pytest.raises(bm.BimoeError) as e:  # row stride not a multiple of 8
        bm.bi_ffn_forward(torch.zeros(8, 68, dtype=BF, device=cuda)[:, :64], w13, w2)
    assert e.value.status == 1
    with pytest.raises(bm.BimoeError) as e:  # base not 16-byte aligned
        bm.bi_ffn_forward(torch.zeros(8, 72, dtype=BF, device=cuda)[:, 4:68], w13, w2)
    assert e.value.status == 1
    with pytest.raises(bm.BimoeError) as e:
        bm.bi_ffn_forward(x, w13, w2, workspace=torch.empty(256, dtype=torch.uint8, device=cuda))
    assert e.value.status == 3
    w13b, w2b = torch.zeros(2 * 24, 64, dtype=BF, device=cuda), torch.zeros(64, 24, dtype=BF, device=cuda)
    with pytest.raises((bm.BimoeError, ValueError)):  # I % 16
        bm.bi_ffn_forward(x, w13b, w2b)
    _, gu, act = bm.bi_ffn_forward_train(x, w13, w2)
    with pytest.raises(ValueError):
        bm.bi_ffn_backward(dout, x, w13, w2, gu[:4], act)
    with pytest.raises(ValueError):
        bm.bi_ffn_backward(dout, x, w13, w2, gu, act, accumulate=True)
    with pytest.raises(TypeError):
        bm.bi_ffn_backward(dout, x, w13, w2, gu, act, dw13=w13.half(), dw2=w2.half())
    with pytest.raises(TypeError):  # one gradient bf16, the other fp32
        bm.bi_ffn_backward(dout, x, w13, w2, gu, act, dw13=w13.clone(), dw2=w2.float())


@pytest.mark.parametrize("M,H,I", [(1, 4096, 2048), (5, 1040, 336), (64, 2048, 768), (200, 3088, 1056),
                                   (256, 8192, 64), (300, 512, 528), (700, 2048, 16)])
def test_schedules_agree(cuda, M, H, I):
    """The CTA-pair kernel and the split kernel give the same bits, forward and backward."""
    import invariant_moe_gb300 as bm
    x, w13, w2, add, dout = (t.to(cuda) for t in make(M, H, I, 120))
    got = []
    old = bm.bi_ffn_schedule(0)
    try:
        for mode in (1, 2):
            bm.bi_ffn_schedule(mode)
            out, gu, act = bm.bi_ffn_forward_train(x, w13, w2, addend=add)
            got.append((bm.bi_ffn_forward(x, w13, w2, addend=add), out, gu, act,
                        bm.bi_ffn_backward(dout, x, w13, w2, gu, act, need=(True, False, False))[0]))
    finally:
        bm.bi_ffn_schedule(old)
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(cuda):
    """More than 2^31 saved projections: the last tokens' rows are those of a small call."""
    import invariant_moe_gb300 as bm
    M, H, I, n = (1 << 20) + 77, 16, 1040, 150
    _, w13, w2, _, _ = (t.to(cuda) for t in make(1, H, I, 130))
    x = syn.normal((M, H), 1.0, 131, BF, device="cuda")
    dout = syn.normal((M, H), 1.0, 132, BF, device="cuda")
    out, gu, act = bm.bi_ffn_forward_train(x, w13, w2)
    assert gu.numel() > 1 << 31
    dx = bm.bi_ffn_backward(dout, x, w13, w2, gu, act, need=(True, False, False))[0]
    for s in (slice(M - n, M), slice((1 << 31) // (2 * I) - 5, (1 << 31) // (2 * I) + n)):
        o, g, a = bm.bi_ffn_forward_train(x[s], w13, w2)
        assert torch.equal(o, out[s]) and torch.equal(g, gu[s]) and torch.equal(a, act[s])
        d = bm.bi_ffn_backward(dout[s], x[s], w13, w2, g, a, need=(True, False, False))[0]
        assert torch.equal(d, dx[s])


PLANS = [
    (129, 80, 48), (33, 80, 144),        # weight-gradient tiles of 128 columns, dx's tiles behind and before them
    (129, 2064, 144), (70, 4112, 144),   # of 256 columns
    (33, 80, 2064), (33, 272, 2064),     # dx by the split kernel, tiles of 128 and 256
    (1025, 80, 48), (2100, 2064, 336)]   # more than one slice of tokens, 128 and 256


@pytest.mark.parametrize("M,H,I", PLANS)
def test_backward_by_every_plan(cuda, M, H, I):
    """Every order and width that the backward's last launch chooses, bf16 and fp32 gradients."""
    import invariant_moe_gb300 as bm
    x, w13, w2, _, dout = make(M, H, I, 140)
    r = ref.ffn(x, w13, w2, dout=dout)
    b = ref.ffn_bounds(r, x, w13, w2, dout=dout)
    args = [t.to(cuda) for t in (dout, x, w13, w2)]
    _, gu, act = bm.bi_ffn_forward_train(*args[1:])
    for name, t in zip(("dx", "dw13", "dw2"), bm.bi_ffn_backward(*args, gu, act)):
        check(name, t, r, b, 2)
    f13, f2 = torch.empty(2 * I, H, device=cuda), torch.empty(H, I, device=cuda)
    _, f13, f2 = bm.bi_ffn_backward(*args, gu, act, dw13=f13, dw2=f2, need=(False, True, True))
    check("dw13", f13, r, b, 1)
    check("dw2", f2, r, b, 1)
