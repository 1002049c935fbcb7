"""What the dense gated feed-forward block and the microscaled 4-bit operators
are timed and compared on.

Four operators, the ones a shared (always active) expert beside the routed
experts needs, from training to 4-bit serving:

* ``ffn``    out = (silu(x Wg^T) * (x Wu^T)) W2^T (+ addend), W13 = [Wg; Wu];
* ``train``  the same with its backward pass: dx, dW13, dW2 from dout;
* ``mx4_quant``  bf16 rows to 4-bit floats (E2M1) with one power-of-two scale
  (E8M0) for each 32 consecutive values, and back to the values they stand for;
* ``mx4_gemm``   the product of two such matrices, plain or gated (the rows of
  the weights are then 16 gate rows, the 16 up rows of the same features, and
  so on, and the result is silu(gate) * up).

Hidden and intermediate sizes are those of the repository's two layer shapes
(H=4096, I=2048 and H=2048, I=768) and generic ones between them.
"""
from __future__ import annotations

import math

import torch

own = False  # False: the plain forms below; True: the framework's calls

_DEV = "cuda"


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one token through the shared expert while serving: the weight stream, latency counts
        {"name": "ffn 1 token", "op": "ffn", "M": 1, "H": 4096, "I": 2048, "addend": True},
        # an odd decode batch through the smaller shape
        {"name": "ffn 33 tokens", "op": "ffn", "M": 33, "H": 2048, "I": 768, "addend": False},
        # a prefill chunk, added to the routed experts' output
        {"name": "ffn 4096 tokens", "op": "ffn", "M": 4096, "H": 4096, "I": 2048, "addend": True},
        # a short ragged training batch, sizes that fill no tile
        {"name": "train 257 tokens", "op": "train", "M": 257, "H": 1040, "I": 720},
        # an ordinary training step of the smaller shape
        {"name": "train 4096 tokens", "op": "train", "M": 4096, "H": 2048, "I": 768},
        # the largest training step, with an odd number of tokens
        {"name": "train 8191 tokens", "op": "train", "M": 8191, "H": 4096, "I": 2048},
        # activations of a decode batch, just before a 4-bit product
        {"name": "mx4 quant 9 rows", "op": "mx4_quant", "R": 9, "K": 4096},
        # a large weight, quantised once when it is loaded (or activations of a long prefill)
        {"name": "mx4 quant 32768 rows", "op": "mx4_quant", "R": 32768, "K": 4096},
        # one token against a 4-bit down projection
        {"name": "mx4 gemm 1 token", "op": "mx4_gemm", "M": 1, "N": 4096, "K": 2048, "gated": False},
        # ragged tokens, an odd number of output features, a K that ends inside a tile
        {"name": "mx4 gemm 100 tokens", "op": "mx4_gemm", "M": 100, "N": 1001, "K": 2080, "gated": False},
        # the 4-bit gate/up projection of a prefill chunk
        {"name": "mx4 gate/up 4096 tokens", "op": "mx4_gemm", "M": 4096, "N": 4096, "K": 4096, "gated": True},
        # a large square product
        {"name": "mx4 gemm 8192 tokens", "op": "mx4_gemm", "M": 8192, "N": 8192, "K": 4096, "gated": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "train", "mx4_quant", "mx4_gemm"])
    if op in ("ffn", "train"):
        H, I = 16 * _log(rng, 16, 256), 16 * _log(rng, 24, 128)
        M = min(_log(rng, 1, 4096) if op == "ffn" else _log(rng, 48, 8191), (1 << 35) // (H * I))
        c = {"op": op, "M": M, "H": H, "I": I}
        if op == "ffn":
            c["addend"] = rng.random() < 0.5
        return c
    if op == "mx4_quant":
        K = 32 * _log(rng, 8, 256)
        return {"op": op, "R": min(_log(rng, 4, 32768), (1 << 27) // K), "K": K}
    gated = rng.random() < 0.4
    N = 32 * _log(rng, 4, 256) if gated else _log(rng, 100, 8192)
    return {"op": op, "M": _log(rng, 1, 8192), "N": N, "K": 32 * _log(rng, 8, 128), "gated": gated}


def work(case):
    op = case["op"]
    if op in ("ffn", "train"):
        M, H, I = case["M"], case["H"], case["I"]
        if op == "ffn":
            # x, W13, W2 (and the addend) read, out written
            return {"bytes": 2 * (2 * M * H + 3 * I * H + (M * H if case["addend"] else 0)), "flops": 6 * M * H * I}
        # x, dout, W13, W2 read; out, dx, dW13, dW2 written; backward is twice the forward's products
        return {"bytes": 2 * (4 * M * H + 6 * I * H), "flops": 18 * M * H * I}
    if op == "mx4_quant":
        n = case["R"] * case["K"]
        # values read, codes and scales written, codes and scales read, values written
        return {"bytes": 4 * n + 2 * (n // 2 + n // 32), "flops": 0}
    M, N, K = case["M"], case["N"], case["K"]
    n_out = N // 2 if case["gated"] else N
    return {"bytes": (M + N) * (K // 2 + K // 32) + 2 * M * n_out, "flops": 2 * M * N * K}


# ----------------------------------------------- 4-bit layout, plain torch --
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pow2(s):
    """2^(s - 127) in 32 bits for the biased exponents s of E8M0 scales (0..254; 255 stands for NaN)."""
    bits = torch.where(s == 0, torch.full_like(s, 0x400000), s << 23)
    return torch.where(s == 255, torch.full_like(s, 0x7FC00000), bits).view(torch.float32)


def _mx4_parts(x):
    """(codes int32 [R, K], biased scale exponents int32 [R, K/32]) of x [R, K]."""
    R, K = x.shape
    b = x.float().view(R, K // 32, 32)
    e = b.abs().amax(dim=2).view(torch.int32) >> 23  # a NaN's or an infinity's is 255
    s = torch.where(e == 255, e, (e - 2).clamp_min(0))
    inv = ((254 - s).clamp_min(1) << 23).view(torch.float32)
    a = (b * inv[:, :, None]).abs()
    # to the nearest of E2M1's values, ties to the even code, above 6 to 6
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
         + (a >= 3.5).int() + (a > 5.0).int())
    c = c + 8 * torch.signbit(b).int()
    return c.view(R, K), s


def _mx4_values(c, s):
    """fp32 values of codes int32 [R, K] and scales int32 [R, K/32]."""
    R, K = c.shape
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=c.device)
    return (table[c.long()].view(R, K // 32, 32) * _pow2(s)[:, :, None]).view(R, K)


def _pack(c):
    return (c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8)


def _unpack(q):
    q = q.int()
    return torch.stack((q & 15, q >> 4), dim=2).view(q.shape[0], -1)


def _tile_scales(s):
    """[R, K/32] to tiles of 128 rows x 4 scales: byte (r % 32) * 16 + (r // 32 % 4) * 4 + k % 4 of a tile; padding is 0."""
    R, n = s.shape
    rt, kt = (R + 127) // 128, (n + 3) // 4
    p = torch.zeros(rt * 128, kt * 4, dtype=torch.uint8, device=s.device)
    p[:R, :n] = s.to(torch.uint8)
    return p.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(rt, kt, 512).contiguous()


def _untile_scales(t, R, n):
    rt, kt, _ = t.shape
    return t.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:R, :n].int()


# ------------------------------------------------------------------ state --
def _normal(g, shape, std):
    return (torch.randn(*shape, generator=g, device=_DEV) * std).to(torch.bfloat16)


def _hidden(g, M, H):
    """Normalised hidden states with a few strong channels, as a layer's input has them."""
    t = torch.randn(M, H, generator=g, device=_DEV)
    strong = torch.randint(0, H, (max(1, H // 256),), generator=g, device=_DEV)
    t[:, strong] *= 6.0
    return t.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    if op in ("ffn", "train"):
        M, H, I = case["M"], case["H"], case["I"]
        st = {"op": op, "x": _hidden(g, M, H), "w13": _normal(g, (2 * I, H), H ** -0.5),
              "w2": _normal(g, (H, I), I ** -0.5), "addend": None}
        if op == "train":
            st["dout"] = _normal(g, (M, H), 1.0)
        elif case["addend"]:
            st["addend"] = _normal(g, (M, H), 0.5)
        return st
    if op == "mx4_quant":
        return {"op": op, "x": _hidden(g, case["R"], case["K"])}
    M, N, K = case["M"], case["N"], case["K"]
    st = {"op": op, "gated": case["gated"]}
    for name, t in (("x", _hidden(g, M, K)), ("w", _normal(g, (N, K), K ** -0.5))):
        c, s = _mx4_parts(t)
        st[name + "q"], st[name + "s"] = _pack(c), _tile_scales(s)
        del c, s, t
    return st


# ------------------------------------------------------------------- runs --
def _plain_ffn(x, w13, w2, addend):
    """(out, g, u, act) in 32 bits."""
    I = w2.shape[1]
    h = x @ w13.t()
    g, u = h[:, :I], h[:, I:]
    act = g / (1.0 + torch.exp(-g)) * u
    out = act @ w2.t()
    return (out if addend is None else out + addend), g, u, act


def _plain(st):
    op = st["op"]
    if op == "ffn":
        out, _, _, _ = _plain_ffn(st["x"].float(), st["w13"].float(), st["w2"].float(),
                                  None if st["addend"] is None else st["addend"].float())
        return {"out": out.to(torch.bfloat16)}
    if op == "train":
        x, w13, w2, dout = (st[n].float() for n in ("x", "w13", "w2", "dout"))
        out, g, u, act = _plain_ffn(x, w13, w2, None)
        dact = dout @ w2
        sig = 1.0 / (1.0 + torch.exp(-g))
        dgu = torch.cat((dact * u * sig * (1.0 + g * (1.0 - sig)), dact * g * sig), dim=1)
        r = {"out": out, "dx": dgu @ w13, "dw13": dgu.t() @ x, "dw2": dout.t() @ act}
        return {k: v.to(torch.bfloat16) for k, v in r.items()}
    if op == "mx4_quant":
        return {"values": _mx4_values(*_mx4_parts(st["x"])).to(torch.bfloat16)}
    n = st["xq"].shape[1] // 16
    x = _mx4_values(_unpack(st["xq"]), _untile_scales(st["xs"], st["xq"].shape[0], n))
    w = _mx4_values(_unpack(st["wq"]), _untile_scales(st["ws"], st["wq"].shape[0], n))
    y = x @ w.t()
    if st["gated"]:
        h = y.view(y.shape[0], -1, 2, 16)
        g, u = h[:, :, 0], h[:, :, 1]
        y = (g / (1.0 + torch.exp(-g)) * u).reshape(y.shape[0], -1)
    return {"y": y.to(torch.bfloat16)}


def _own(st):
    import invariant_moe_gb300 as bm

    op = st["op"]
    if op in ("ffn", "train"):
        x, w13, w2 = st["x"], st["w13"], st["w2"]
        if "out" not in st:  # buffers that a program keeps from step to step
            (M, H), I = x.shape, w2.shape[1]
            st["out"] = torch.empty_like(x)
            st["workspace"] = bm.ffn_workspace(M, H, I, x.device)
            if op == "train":
                st["saved"] = bm.ffn_saved(M, I, x.device)
                st["grads"] = (torch.empty_like(x), torch.empty_like(w13), torch.empty_like(w2))
        if op == "ffn":
            return {"out": bm.bi_ffn_forward(x, w13, w2, addend=st["addend"], out=st["out"], workspace=st["workspace"])}
        gu, act = st["saved"]
        dx, dw13, dw2 = st["grads"]
        bm.bi_ffn_forward_train(x, w13, w2, out=st["out"], gu=gu, act=act)
        bm.bi_ffn_backward(st["dout"], x, w13, w2, gu, act, dx=dx, dw13=dw13, dw2=dw2, workspace=st["workspace"])
        return {"out": st["out"], "dx": dx, "dw13": dw13, "dw2": dw2}
    if op == "mx4_quant":
        x = st["x"]
        if "out" not in st:
            st["q"], st["s"] = bm.mx4_empty(x.shape[0], x.shape[1], x.device)
            st["out"] = torch.empty_like(x)
        bm.bi_mx4_quantize(x, q=st["q"], scales=st["s"])
        return {"values": bm.bi_mx4_dequantize(st["q"], st["s"], out=st["out"])}
    if "out" not in st:
        N = st["wq"].shape[0]
        st["out"] = torch.empty(st["xq"].shape[0], N // 2 if st["gated"] else N, dtype=torch.bfloat16,
                                device=st["xq"].device)
    f = bm.bi_mx4_gate_up if st["gated"] else bm.bi_mx4_gemm
    return {"y": f(st["xq"], st["xs"], st["wq"], st["ws"], out=st["out"])}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ exact --
def _grid4(x):
    """The definition in 64 bits: x [R, K] to the values that its 4-bit form stands for."""
    R, K = x.shape
    b = x.double().reshape(R, -1, 32)
    top = b.abs().max(dim=2, keepdim=True).values
    _, ex = torch.frexp(top)  # top = m 2^ex, m in [0.5, 1)
    e = torch.where(top == 0, torch.full_like(ex, -127), (ex - 3).clamp(min=-127))
    scale = torch.ldexp(torch.ones_like(top), e)
    a = b / scale
    _, ea = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (ea - 1).clamp(min=0) - 1)
    v = (torch.round(a / step) * step).clamp(-6.0, 6.0)
    return (v * scale).reshape(R, K)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "mx4_quant":
        return {"values": _grid4(st["x"])}
    if op == "mx4_gemm":
        M, N, K = case["M"], case["N"], case["K"]

        def values(q, t, R):
            lo, hi = q.long() % 16, q.long() // 16
            c = torch.stack((lo, hi), dim=-1).reshape(R, K)
            mant, expo, neg = c % 2, c // 2 % 4, c // 8
            v = torch.where(expo == 0, 0.5 * mant, torch.ldexp(1.0 + 0.5 * mant.double(), expo - 1))
            r = torch.arange(R, device=q.device)[:, None]
            k = torch.arange(K // 32, device=q.device)[None, :]
            byte = t[r // 128, k // 4, (r % 32) * 16 + (r // 32 % 4) * 4 + k % 4].long()
            scale = torch.ldexp(torch.ones(R, K // 32, dtype=torch.float64, device=q.device), byte - 127)
            return (v * (1 - 2 * neg)).double() * scale.repeat_interleave(32, dim=1)

        y = values(st["xq"], st["xs"], M) @ values(st["wq"], st["ws"], N).T
        if case["gated"]:
            f = torch.arange(N // 2, device=y.device)
            rows = f // 16 * 32 + f % 16
            g, u = y[:, rows], y[:, rows + 16]
            y = g * torch.sigmoid(g) * u
        return {"y": y}
    x, w13, w2 = st["x"].double(), st["w13"].double(), st["w2"].double()
    I = case["I"]
    g, u = x @ w13[:I].T, x @ w13[I:].T
    sg = torch.sigmoid(g)
    act = g * sg * u
    out = act @ w2.T
    if op == "ffn":
        return {"out": out if st["addend"] is None else out + st["addend"].double()}
    dout = st["dout"].double()
    dact = dout @ w2
    dg, du = dact * u * (sg + g * sg * (1 - sg)), dact * g * sg
    return {"out": out, "dx": dg @ w13[:I] + du @ w13[I:], "dw13": torch.cat((dg.T @ x, du.T @ x)),
            "dw2": dout.T @ act}
