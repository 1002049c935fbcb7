"""Plain 64-bit forms of the gated feed-forward block and of the microscaled
4-bit operators, and the error bounds their tests use.

Bounds.  bf16 keeps 8 significant bits: one rounding to nearest is off by at
most U = 2^-8 of the value.  An fp32 sum of n products is off by at most
n * 2^-23 of the sum of the products' magnitudes, in any order and whether its
additions round or truncate (EPS32 below).  ``ffn_bounds`` carries both through
the formulas element by element.  Over a whole tensor the roundings are
independent with a relative variance of at most U^2 / 3 each, so n of them give
a 2-norm error of at most U * sqrt(n / 3) of the result's 2-norm;
``norm_bound`` allows a quarter more for small samples.  A product that is left
out or taken twice shows in the 2-norm as 1 / sqrt(n)."""
import math

import torch

U = 2.0 ** -8
EPS32 = 2.0 ** -23


def norm_bound(roundings):
    return 1.25 * U * math.sqrt(roundings / 3.0)


def rel_norm(got, ref):
    got, ref = got.double(), ref.double()
    n = float(ref.norm())
    d = float((got - ref).norm())
    return d / n if n else (math.inf if d else 0.0)


def silu(g):
    return g / (1.0 + torch.exp(-g))


def ffn(x, w13, w2, addend=None, dout=None):
    """All of the block's values in fp64 (dict), the gradients too when dout is given."""
    x, w13, w2 = x.double(), w13.double(), w2.double()
    I = w2.shape[1]
    g, u = x @ w13[:I].T, x @ w13[I:].T
    act = silu(g) * u
    r = {"g": g, "u": u, "act": act, "out": act @ w2.T}
    if addend is not None:
        r["out"] = r["out"] + addend.double()
    if dout is not None:
        d = dout.double()
        r["dact"] = d @ w2
        s = 1.0 / (1.0 + torch.exp(-g))
        r["dg"] = r["dact"] * u * s * (1.0 + g * (1.0 - s))
        r["du"] = r["dact"] * g * s
        r["dgu"] = torch.cat((r["dg"], r["du"]), dim=1)
        r["dx"] = r["dgu"] @ w13
        r["dw13"] = r["dgu"].T @ x
        r["dw2"] = d.T @ act
    return r


def ffn_bounds(r, x, w13, w2, addend=None, dout=None):
    """Largest absolute error of each result in r, element by element."""
    x, w13, w2 = x.double().abs(), w13.double().abs(), w2.double().abs()
    I, H = w2.shape[1], x.shape[1]
    eg, eu = (H * EPS32 * (x @ w.T) for w in (w13[:I], w13[I:]))
    # silu' lies in (-0.1, 1.1); exp, the reciprocal and the products of the epilogue: 16 fp32 roundings
    pre = 1.1 * r["u"].abs() * eg + silu(r["g"]).abs() * eu + 1.1 * eg * eu + 16 * EPS32 * r["act"].abs()
    b = {"act": U * r["act"].abs() + (1 + U) * pre}
    mag = r["act"].abs() + b["act"]
    raw = b["act"] @ w2.T + I * EPS32 * (mag @ w2.T)
    if addend is not None:
        raw = raw + EPS32 * (r["out"].abs() + addend.double().abs())
    b["out"] = U * r["out"].abs() + (1 + U) * raw
    if dout is not None:
        d = dout.double().abs()
        M = x.shape[0]
        ed = H * EPS32 * (d @ w2)
        s = 1.0 / (1.0 + torch.exp(-r["g"]))
        dgate = s * (1.0 + r["g"] * (1.0 - s))
        # |silu''| <= 0.5
        pg = (ed * (r["u"] * dgate).abs() + r["dact"].abs() * (eu * dgate.abs() + 0.5 * eg * r["u"].abs()) +
              1.1 * ed * (eu + eg * r["u"].abs()) + 32 * EPS32 * (r["dact"] * r["u"]).abs())
        pu = (ed * (r["g"] * s).abs() + 1.1 * r["dact"].abs() * eg + 1.1 * ed * eg +
              32 * EPS32 * (r["dact"] * r["g"] * s).abs())
        b["dgu"] = U * r["dgu"].abs() + (1 + U) * torch.cat((pg, pu), dim=1)
        mag = r["dgu"].abs() + b["dgu"]
        b["dx"] = U * r["dx"].abs() + (1 + U) * (b["dgu"] @ w13 + 2 * I * EPS32 * (mag @ w13))
        b["dw13"] = U * r["dw13"].abs() + (1 + U) * (b["dgu"].T @ x + M * EPS32 * (mag.T @ x))
        b["dw2"] = U * r["dw2"].abs() + (1 + U) * (d.T @ b["act"] + M * EPS32 * (d.T @ (r["act"].abs() + b["act"])))
    return b


# ------------------------------------------------------------ 4-bit form --
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def mx4_quantize(x):
    """(codes uint8 [R, K], scale bytes uint8 [R, K/32]) of x, by search over E2M1's values."""
    R, K = x.shape
    b = x.double().reshape(R, K // 32, 32)
    bad = ~torch.isfinite(b).all(dim=2)
    amax = torch.nan_to_num(b.abs(), nan=0.0, posinf=0.0).amax(dim=2)
    _, e = torch.frexp(amax)                      # amax = m 2^e, m in [0.5, 1)
    e = torch.where(amax == 0, torch.full_like(e, -127), (e - 3).clamp(min=-127))
    scale = torch.pow(torch.tensor(2.0, dtype=torch.float64), e.double())
    a = (b / scale[:, :, None]).abs()
    grid = torch.tensor(E2M1, dtype=torch.float64)
    d = (a[..., None] - grid).abs()
    best = d.amin(dim=-1, keepdim=True)
    # ties: the even code
    rank = torch.where(d == best, torch.tensor([0, 1, 0, 1, 0, 1, 0, 1]), torch.tensor(9))
    codes = rank.argmin(dim=-1) + 8 * torch.signbit(b).long()
    codes = torch.where(bad[:, :, None], torch.zeros_like(codes), codes)
    sb = torch.where(bad, torch.full_like(e, 255), e + 127)
    return codes.reshape(R, K).to(torch.uint8), sb.to(torch.uint8)


def mx4_pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()


def mx4_values(codes, scales):
    """fp64 values of codes [R, K] and scale bytes [R, K/32]."""
    R, K = codes.shape
    v = torch.tensor(E2M1 + [-a for a in E2M1], dtype=torch.float64)[codes.long()]
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64), scales.double() - 127.0)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return (v.view(R, K // 32, 32) * s[:, :, None]).view(R, K)


def tile_scales(s):
    """Row-major scale bytes to the tiled layout, one byte at a time."""
    R, n = s.shape
    rt, kt = (R + 127) // 128, (n + 3) // 4
    t = torch.zeros(rt, kt, 512, dtype=torch.uint8)
    r = torch.arange(R)[:, None].expand(R, n)
    b = torch.arange(n)[None, :].expand(R, n)
    t[r // 128, b // 4, (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4] = s
    return t


def mx4_product(xv, wv, addend=None):
    """(y, its bound) in fp64 of values xv [M, K], wv [N, K]."""
    K = xv.shape[1]
    y = xv @ wv.T
    raw = K * EPS32 * (xv.abs() @ wv.abs().T)
    if addend is not None:
        y = y + addend.double()
        raw = raw + EPS32 * (y.abs() + addend.double().abs())
    return y, U * y.abs() + (1 + U) * raw


def mx4_gated(xv, wv):
    """(act, its bound) in fp64; wv's rows are 16 gate rows, their 16 up rows, and so on."""
    K = xv.shape[1]
    I = wv.shape[0] // 2
    f = torch.arange(I)
    rows = f // 16 * 32 + f % 16
    h = xv @ wv.T
    e = K * EPS32 * (xv.abs() @ wv.abs().T)
    g, u, eg, eu = h[:, rows], h[:, rows + 16], e[:, rows], e[:, rows + 16]
    act = silu(g) * u
    pre = 1.1 * u.abs() * eg + silu(g).abs() * eu + 1.1 * eg * eu + 16 * EPS32 * act.abs()
    return act, U * act.abs() + (1 + U) * pre
