"""Operators that train a routed-experts layer: results that would be written over what the call still reads are
refused (no GPU: the addresses are never read)."""
import ctypes

import pytest

NUL = ctypes.c_void_p(None)
WS = ctypes.c_void_p(1 << 60)
M, H, E, K, I = 8, 128, 4, 2, 128
P = M * K
BAD = 1


def far(i):
    return (i + 2) << 40


@pytest.fixture(scope="module")
def lib():
    from invariant_moe_gb300 import _build
    _build.build()
    import invariant_moe_gb300 as bm
    return bm.load_library()


# place among the arguments, bytes
FORWARD = {"x": (0, M * H * 2), "ids": (1, P * 4), "wts": (2, P * 4), "w13": (3, E * 2 * I * H * 2),
           "w2": (4, E * H * I * 2), "out": (5, M * H * 2), "offsets": (6, (E + 1) * 4), "perm": (7, P * 4),
           "slots": (8, M * 4), "x_perm": (9, P * H * 2), "gu": (10, P * 2 * I * 4), "act": (11, P * I * 2)}
BACKWARD = {"dout": (0, M * H * 2), "ids": (1, P * 4), "wts": (2, P * 4), "w13": (3, E * 2 * I * H * 2),
            "w2": (4, E * H * I * 2), "offsets": (5, (E + 1) * 4), "perm": (6, P * 4), "slots": (7, M * 4),
            "x_perm": (8, P * H * 2), "gu": (9, P * 2 * I * 4), "act": (10, P * I * 2), "w_router": (11, E * H * 4),
            "dx": (12, M * H * 2), "dwts": (13, P * 4), "dw13": (14, E * 2 * I * H * 2), "dw2": (15, E * H * I * 2)}


def places(table, over=None):
    """The arguments, each far from the others; over: (name, other): name over other's first bytes, and over its
    last 16."""
    p = [far(i) for i in range(len(table))]
    if over is None:
        return [p]
    name, other = over
    out = []
    for at in (p[table[other][0]], p[table[other][0]] + (table[other][1] - 16) // 16 * 16):
        q = list(p)
        q[table[name][0]] = at
        out.append(q)
    return out


def forward(lib, p):
    return lib.bi_moe_forward_train(*map(ctypes.c_void_p, p), M, H, E, K, I, WS, 1 << 40, NUL)


def backward(lib, p):
    return lib.bi_moe_backward(*map(ctypes.c_void_p, p), 0, M, H, E, K, I, WS, 1 << 40, NUL)


@pytest.mark.parametrize("name", ["out", "offsets", "perm", "slots", "x_perm", "gu", "act"])
def test_forward(lib, name):
    for other in FORWARD:
        if other == name or (name, other) == ("out", "x"):
            continue
        assert all(forward(lib, p) == BAD for p in places(FORWARD, (name, other))), other
        assert name in lib.bi_last_error_message().decode() and "overlap" in lib.bi_last_error_message().decode()


def test_forward_over_part_of_x(lib):
    assert forward(lib, places(FORWARD, ("out", "x"))[1]) == BAD


LATE = ("offsets", "x_perm", "act", "dx", "dwts")


@pytest.mark.parametrize("name", ["dx", "dwts", "dw13", "dw2"])
def test_backward(lib, name):
    for other in BACKWARD:
        if other == name or (name, other) == ("dx", "dout"):
            continue
        if name[:2] == "dw" and name != "dwts" and other not in LATE + ("dw13", "dw2"):
            continue
        assert all(backward(lib, p) == BAD for p in places(BACKWARD, (name, other))), other
        assert name in lib.bi_last_error_message().decode() and "overlap" in lib.bi_last_error_message().decode()


def test_backward_over_part_of_dout(lib):
    assert backward(lib, places(BACKWARD, ("dx", "dout"))[1]) == BAD


# the router's gradient, of bf16 x; places among its arguments
ROUTER = {"dwts": (0, P * 4), "ids": (1, P * 4), "wts": (2, P * 4), "x": (3, M * H * 2), "w": (5, E * H * 4),
          "offsets": (6, (E + 1) * 4), "perm": (7, P * 4), "dx": (8, M * H * 2), "dw": (9, E * H * 4),
          "dbias": (10, E * 4)}


@pytest.mark.parametrize("name", ["dx", "dw", "dbias"])
def test_router(lib, name):
    for other, (at, size) in ROUTER.items():
        if other == name:
            continue
        for start in (0, (size - 16) // 16 * 16):
            p = [far(i) for i in range(11)]
            p[4] = 0  # x is bf16
            p[ROUTER[name][0]] = p[at] + start
            assert lib.bi_router_backward(*[v if i == 4 else ctypes.c_void_p(v) for i, v in enumerate(p)], 0, M, H, E, K,
                                          NUL) == BAD, other
            assert "overlap" in lib.bi_last_error_message().decode()


# layer norm of 3 rows of 37 fp32 values, 48 apart: rows' bytes, then the vectors'
ROWS, WIDTH, LD = 3, 37, 48


def norm(lib, x, w, b, y, mean, rstd):
    p = ctypes.c_void_p
    return lib.bi_layer_norm(p(x), 1, LD, p(w), p(b), 1, ctypes.c_float(1e-5), p(y), LD, p(mean), p(rstd), ROWS, WIDTH,
                             NUL)


def norm_backward(lib, dx, w, mean, rstd, dw, db):
    p = ctypes.c_void_p
    return lib.bi_layer_norm_backward(p(far(20)), LD, p(far(21)), 1, LD, p(w), 1, p(mean), p(rstd), p(dx), LD, p(dw),
                                      p(db), 0, ROWS, WIDTH, WS, 1 << 30, NUL)


# a vector on a row's first and last value, across the start of the next row, and just before the rows
def on_rows(base, size):
    return [base, base + (LD + WIDTH - 1) * 4, base + (2 * LD) * 4 - 4 * (size > 4), base - 4 * (size > 4)]


def test_norm(lib):
    a = [far(i) for i in range(6)]  # x, w, b, y, mean, rstd

    def call(**k):
        v = dict(zip(("x", "w", "b", "y", "mean", "rstd"), a), **k)
        return norm(lib, **v)

    for rows, vectors in (("y", ("w", "b", "mean", "rstd")), ("x", ("mean", "rstd"))):
        for v in vectors:
            for at in on_rows(a["x w b y".split().index(rows)], 12):
                assert call(**{v: at}) == BAD, (rows, v)
                assert "overlap" in lib.bi_last_error_message().decode()
    for v, o in (("mean", "rstd"), ("mean", "w"), ("rstd", "b")):
        assert call(**{v: dict(zip(("w", "b", "rstd"), (a[1], a[2], a[5])))[o] + 8}) == BAD


def test_norm_backward(lib):
    a = {n: far(i) for i, n in enumerate(("dx", "w", "mean", "rstd", "dw", "db"))}
    for v in ("w", "mean", "rstd", "dw", "db"):
        for at in on_rows(a["dx"], 12):
            assert norm_backward(lib, **dict(a, **{v: at})) == BAD, v
            assert "dx overlaps" in lib.bi_last_error_message().decode()
    assert norm_backward(lib, **dict(a, db=a["dw"] + 4)) == BAD
