"""The gated feed-forward block against the fp64 form.

Tolerances, element by element. A product of K terms accumulated in fp32 in any order is off by at most K 2^-23 of the
sum of the terms' magnitudes (2^-23 a step: the tensor cores may truncate). The activation's error is that of its
argument times a slope below 1.2, plus 2^-20 (1 + |g|) of its value for the exponential and the quotient. Operands
rounded to bf16 on the way (h, dg, du) and the results add half a step each, 2^-8 of the value.
"""
import ctypes

import numpy as np
import pytest
import torch

import dynamic_block_sparse_shape_b200 as P
from oracle import layer_oracle as O
from tests.gpu_util import f64, require_gpu

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]
STEP = 2.0 ** -8


def draw(m, d, f, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, k=1.0: (torch.randn(s, generator=g) * k).to(torch.bfloat16).to(device)  # noqa: E731
    return n(m, d), n(f, d, k=d ** -0.5), n(f, d, k=d ** -0.5), n(d, f, k=f ** -0.5), n(m, d)


def mm_err(a, b, ea=0.0, eb=0.0):
    """Error bound of a @ b.T for operands off by at most ea, eb."""
    k = a.shape[1]
    return k * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T) + (
        ea @ np.abs(b).T if np.ndim(ea) else 0.0) + (np.abs(a) @ eb.T if np.ndim(eb) else 0.0)


def close(name, got, want, err):
    tol = err + STEP * (np.abs(want) + err) + 1e-30
    off = np.abs(f64(got) - want)
    assert np.isfinite(f64(got)).all(), name
    assert (off <= tol).all(), f"{name}: {float((off / tol).max()):.3f} of the bound"


def check_fwd(x, wg, wu, wd, act, y, gate, up):
    X, G, U, D = f64(x), f64(wg), f64(wu), f64(wd)
    ry, g, u = O.gated_ffn_fwd(X, G, U, D, act)
    eg, eu = mm_err(X, G), mm_err(X, U)
    if gate is not None:
        close("gate", gate, g, eg)
        close("up", up, u, eu)
    a = O.activation(act, g)
    h = a * u
    eh = 1.2 * eg * (np.abs(u) + eu) + np.abs(a) * eu + 2.0 ** -20 * (1 + np.abs(g)) * np.abs(h)
    eh = eh + STEP * (np.abs(h) + eh)
    close("y", y, ry, mm_err(h, D, ea=eh))


def check_bwd(dy, x, wg, wu, wd, gate, up, act, got):
    DY, X, G, U, D, g, u = (f64(t) for t in (dy, x, wg, wu, wd, gate, up))
    want = O.gated_ffn_bwd(DY, X, G, U, D, g, u, act)
    a, s = O.activation(act, g), O.activation_slope(act, g)
    dh = DY @ D
    edh = mm_err(DY, D.T.copy())
    rel = 2.0 ** -19 * (1 + g * g)  # the slope's polynomial and exponentials
    dg, du, h = dh * u * s, dh * a, a * u
    edg = edh * np.abs(u) * (np.abs(s) + rel) + np.abs(dh * u) * rel
    edu = edh * np.abs(a) + np.abs(dh) * (np.abs(a) + np.abs(g) * 2.0 ** -3) * rel
    eh = (np.abs(a) + np.abs(g) * 2.0 ** -3) * rel * np.abs(u)
    edg, edu, eh = (e + STEP * (np.abs(v) + e) for e, v in ((edg, dg), (edu, du), (eh, h)))
    dx, dwg, dwu, dwd = got
    if dx is not None:
        close("dx", dx, want[0], mm_err(dg, G.T.copy(), ea=edg) + mm_err(du, U.T.copy(), ea=edu))
    if dwg is not None:
        close("dw_gate", dwg, want[1], mm_err(dg.T.copy(), X.T.copy(), ea=edg.T.copy()))
        close("dw_up", dwu, want[2], mm_err(du.T.copy(), X.T.copy(), ea=edu.T.copy()))
        close("dw_down", dwd, want[3], mm_err(DY.T.copy(), h.T.copy(), eb=eh.T.copy()))


# one token, single rows past a tile, widths of 8 values, K of less than a slice, sizes that give pairs of CTAs for
# every product
SIZES = [(1, 8, 8), (1, 64, 128), (2, 72, 136), (3, 520, 264), (8, 2312, 40), (5, 40, 2312), (31, 256, 64), (32, 1096, 200), (33, 200, 1096), (12, 72, 5000), (127, 64, 192), (128, 256, 256), (129, 264, 520),
         (300, 1160, 392), (1000, 136, 2056)]
LARGE = [(700, 1160, 1032), (300, 2312, 1032), (2100, 2312, 2056), (2305, 2304, 1288), (4700, 40, 2056), (9000, 264, 1032)]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,d,f", SIZES)
def test_forward_backward(m, d, f, act):
    require_gpu()
    x, wg, wu, wd, dy = draw(m, d, f, m + d + f)
    ws = P.Workspace("cuda")
    y, g, u = P.gated_ffn_fwd(x, wg, wu, wd, act=act, ws=ws)
    check_fwd(x, wg, wu, wd, act, y, g, u)
    y2, none, _ = P.gated_ffn_fwd(x, wg, wu, wd, act=act, save=False, ws=ws)
    assert none is None and torch.equal(y2, y)
    got = P.gated_ffn_bwd(dy, x, wg, wu, wd, g, u, act=act, ws=ws)
    P.check_device_status(ws)
    check_bwd(dy, x, wg, wu, wd, g, u, act, got)
    one = P.gated_ffn_bwd(dy, x, wg, wu, wd, g, u, act=act, need_dw=False, ws=ws)
    two = P.gated_ffn_bwd(dy, x, wg, wu, wd, g, u, act=act, need_dx=False, ws=ws)
    assert one[1:] == (None, None, None) and two[0] is None
    assert torch.equal(one[0], got[0]) and all(torch.equal(a, b) for a, b in zip(two[1:], got[1:]))


@pytest.mark.gpu
@pytest.mark.parametrize("m,d,f", LARGE)
def test_large_tiles(m, d, f):
    require_gpu()
    x, wg, wu, wd, dy = draw(m, d, f, 5)
    ws = P.Workspace("cuda")
    y, g, u = P.gated_ffn_fwd(x, wg, wu, wd, ws=ws)
    got = P.gated_ffn_bwd(dy, x, wg, wu, wd, g, u, ws=ws)
    P.check_device_status(ws)
    check_fwd(x, wg, wu, wd, "silu", y, g, u)
    check_bwd(dy, x, wg, wu, wd, g, u, "silu", got)
