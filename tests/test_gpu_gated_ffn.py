"""The gated feed-forward block against the fp64 form.

Tolerances, element by element. A product of K terms accumulated in fp32 in any order is off by at most K 2^-23 of the
sum of the terms' magnitudes (2^-23 a step: the tensor cores may truncate). The activation's error is that of its
argument times a slope below 1.2, plus 2^-20 (1 + |g|) of its value for the exponential and the quotient. Operands
rounded to bf16 on the way (h, dg, du) and the results add half a step each, 2^-8 of the value; of at most 32 tokens the
operands' remainders, at most 2^-8 of the value, come along rounded to bf16, which leaves 2^-16.
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


def held(m):
    return STEP if m > 32 else STEP * STEP


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
    eh = eh + held(x.shape[0]) * (np.abs(h) + eh)
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
    edg, edu, eh = (e + held(x.shape[0]) * (np.abs(v) + e) for e, v in ((edg, dg), (edu, du), (eh, h)))
    dx, dwg, dwu, dwd = got
    if dx is not None:
        close("dx", dx, want[0], mm_err(dg, G.T.copy(), ea=edg) + mm_err(du, U.T.copy(), ea=edu))
    if dwg is not None:
        close("dw_gate", dwg, want[1], mm_err(dg.T.copy(), X.T.copy(), ea=edg.T.copy()))
        close("dw_up", dwu, want[2], mm_err(du.T.copy(), X.T.copy(), ea=edu.T.copy()))
        close("dw_down", dwd, want[3], mm_err(DY.T.copy(), h.T.copy(), eb=eh.T.copy()))


# one token, single rows past a tile, widths of 8 values, K of less than a slice, sizes that give pairs of CTAs for
# every product
SIZES = [(1, 8, 8), (1, 64, 128), (2, 72, 136), (3, 520, 264), (8, 2312, 40), (5, 40, 2312), (31, 256, 64),
         (32, 1096, 200), (33, 200, 1096), (12, 72, 5000), (127, 64, 192), (128, 256, 256), (129, 264, 520),
         (300, 1160, 392), (1000, 136, 2056), (7, 2400, 136), (16, 2368, 136), (9, 2400, 72), (17, 72, 72)]
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


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 20, 100, 300, 2100])
def test_views_and_what_lies_around(m):
    """Weights as the halves of one matrix, padded rows everywhere; nothing outside the outputs changes."""
    require_gpu()
    d, f = 264, 136 if m < 2000 else 2056
    x, wg, wu, wd, dy = draw(m, d, f, m)
    both = torch.full((2 * f, d + 24), 9.0, dtype=torch.bfloat16, device="cuda")
    both[:f, :d], both[f:, :d] = wg, wu
    wdp = torch.full((d, f + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    wdp[:, :f] = wd
    buf = torch.full((m + 3, d + 40), -7.0, dtype=torch.bfloat16, device="cuda")
    xp, yp = buf.clone(), buf.clone()
    xp[:m, :d] = x
    ws = P.Workspace("cuda")
    y, g, u = P.gated_ffn_fwd(x, wg, wu, wd, ws=ws)
    got, g2, u2 = P.gated_ffn_fwd(xp[:m, :d], both[:f, :d], both[f:, :d], wdp[:, :f], out=yp[:m, :d], ws=ws)
    assert got.data_ptr() == yp.data_ptr() and torch.equal(got, y) and torch.equal(g, g2) and torch.equal(u, u2)
    assert (yp[m:] == -7).all() and (yp[:, d:] == -7).all()
    P.gated_ffn_fwd(xp[:m, :d], both[:f, :d], both[f:, :d], wdp[:, :f], out=xp[:m, :d], save=False, ws=ws)  # y over x
    assert torch.equal(xp[:m, :d], y) and (xp[m:] == -7).all() and (xp[:, d:] == -7).all()
    dyp = buf.clone()
    dyp[:m, :d] = dy
    xp[:m, :d] = x
    a = P.gated_ffn_bwd(dy, x, wg, wu, wd, g, u, ws=ws)
    b = P.gated_ffn_bwd(dyp[:m, :d], xp[:m, :d], both[:f, :d], both[f:, :d], wdp[:, :f], g, u, ws=ws)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    P.check_device_status(ws)


def _outputs_in(buffers):
    """Views of the middle of canary-filled buffers."""
    return [b[64:64 + n].view(shape) for b, n, shape in buffers]


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 9, 33, 129, 2305])
def test_backward_writes_only_its_outputs(m):
    require_gpu()
    d, f = 328, 1288
    x, wg, wu, wd, dy = draw(m, d, f, 3)
    ws = P.Workspace("cuda")
    _, g, u = P.gated_ffn_fwd(x, wg, wu, wd, ws=ws)
    want = P.gated_ffn_bwd(dy, x, wg, wu, wd, g, u, ws=ws)
    shapes = [(m, d), (f, d), (f, d), (d, f)]
    bufs = [(torch.full((a * b + 128,), 5.0, dtype=torch.bfloat16, device="cuda"), a * b, (a, b)) for a, b in shapes]
    dx, dwg, dwu, dwd = _outputs_in(bufs)
    w, _, _ = P._ffn_weights(wg, wu, wd, "test")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = P.lib().prism_gated_ffn_bwd(ctypes.byref(w), m, 0, 0, p(dy), d, p(x), d, p(g), p(u), p(dx), d, p(dwg), p(dwu),
                                     p(dwd), ws.ptr, ws.nbytes, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for t, r, (b, n, _) in zip((dx, dwg, dwu, dwd), want, bufs):
        assert torch.equal(t, r) and (b[:64] == 5).all() and (b[64 + n:] == 5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 40, 700])
def test_rows_are_apart(m):
    """NaN and infinities of one token stay in its row, whatever tile it shares."""
    require_gpu()
    d, f = 1160, 1032
    x, wg, wu, wd, dy = draw(m, d, f, 4)
    y, g, u = P.gated_ffn_fwd(x, wg, wu, wd)
    bad = m // 2
    x2, dy2 = x.clone(), dy.clone()
    x2[bad] = float("nan")
    y2, g2, u2 = P.gated_ffn_fwd(x2, wg, wu, wd)
    keep = torch.arange(m, device="cuda") != bad
    assert torch.isnan(y2[bad]).all() and torch.equal(y2[keep], y[keep])
    dy2[bad] = float("inf")
    a = P.gated_ffn_bwd(dy, x, wg, wu, wd, g, u, need_dw=False)[0]
    b = P.gated_ffn_bwd(dy2, x, wg, wu, wd, g, u, need_dw=False)[0]
    assert not torch.isfinite(b[bad]).any() and torch.equal(b[keep], a[keep])


@pytest.mark.gpu
def test_empty_streams_and_graphs():
    require_gpu()
    d, f = 256, 512
    x, wg, wu, wd, dy = draw(300, d, f, 6)
    y, g, u = P.gated_ffn_fwd(x[:0], wg, wu, wd)
    assert y.shape == (0, d) and g.shape == (0, f)
    dx, dwg, dwu, dwd = P.gated_ffn_bwd(dy[:0], x[:0], wg, wu, wd, g, u)
    assert dx.shape == (0, d) and all((t == 0).all() for t in (dwg, dwu, dwd))
    assert P.gated_ffn_bwd(dy[:0], x[:0], wg, wu, wd, g, u, need_dw=False)[0].shape == (0, d)
    want = P.gated_ffn_fwd(x, wg, wu, wd)
    wantb = P.gated_ffn_bwd(dy, x, wg, wu, wd, want[1], want[2])
    # another stream, with no workspace given: its memory is not handed on before the stream is done with it
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [P.gated_ffn_fwd(x, wg, wu, wd, stream=side) for _ in range(8)]
    junk = [torch.full((300, f), 3.0, device="cuda") for _ in range(8)]
    side.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want)) and len(junk) == 8
    # two captured graphs that share a workspace, replayed in turn on one stream, after eager calls that grow it
    ws = P.Workspace("cuda")
    graphs = []
    for m in (7, 300):
        xs = x[:m].clone()
        P.gated_ffn_fwd(xs, wg, wu, wd, ws=ws)
        P.gated_ffn_bwd(dy[:m], xs, wg, wu, wd, want[1][:m].clone(), want[2][:m].clone(), ws=ws)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            yy, gg, uu = P.gated_ffn_fwd(xs, wg, wu, wd, ws=ws)
            bb = P.gated_ffn_bwd(dy[:m], xs, wg, wu, wd, gg, uu, ws=ws)
        graphs.append((gr, m, yy, bb))
    held = ws.buf.numel()
    ws.ensure(1 << 26)  # a larger buffer: the graphs' own stays theirs
    junk = [torch.full((held,), 3, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for _ in range(2):
        for gr, m, yy, bb in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert all((j == 3).all() for j in junk)
    for gr, m, yy, bb in graphs:
        r = P.gated_ffn_fwd(x[:m], wg, wu, wd)
        rb = P.gated_ffn_bwd(dy[:m], x[:m], wg, wu, wd, r[1], r[2])
        assert torch.equal(yy, r[0]) and all(torch.equal(a, b) for a, b in zip(bb, rb))
    assert all(torch.equal(a, b) for a, b in zip(wantb, graphs[1][3]))


@pytest.mark.gpu
@pytest.mark.parametrize("m,stride", [(20, 1 << 28), (300, 1 << 24)])
def test_offsets_past_32_bits(m, stride):
    """Tokens more than 2^32 elements apart (10 GB between the first and the last)."""
    require_gpu()
    d, f = 136, 264
    x, wg, wu, wd, dy = draw(m, d, f, 8)
    want = P.gated_ffn_fwd(x, wg, wu, wd)
    wantb = P.gated_ffn_bwd(dy, x, wg, wu, wd, want[1], want[2])
    buf = torch.empty((m - 1) * stride + d, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((m, d), (stride, 1))
    far.copy_(x)
    got = P.gated_ffn_fwd(far, wg, wu, wd)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    gotb = P.gated_ffn_bwd(dy, far, wg, wu, wd, want[1], want[2])
    assert all(torch.equal(a, b) for a, b in zip(gotb, wantb))
    P.gated_ffn_fwd(x, wg, wu, wd, out=far)
    assert torch.equal(far, want[0])


@pytest.mark.parametrize("act", ACTS)
def test_formulas_against_differences(act):
    """The fp64 gradient formulas that the kernels are held to, against central differences of the fp64 forward."""
    r = np.random.default_rng(1)
    m, d, f = 3, 5, 7
    x, wg, wu, wd, dy = r.normal(size=(m, d)), r.normal(size=(f, d)), r.normal(size=(f, d)), r.normal(size=(d, f)), \
        r.normal(size=(m, d))
    _, g, u = O.gated_ffn_fwd(x, wg, wu, wd, act)
    grads = O.gated_ffn_bwd(dy, x, wg, wu, wd, g, u, act)
    loss = lambda *a: float((O.gated_ffn_fwd(*a, act)[0] * dy).sum())  # noqa: E731
    args, h = [x, wg, wu, wd], 1e-6
    for i, grad in enumerate(grads):
        for _ in range(6):
            v = r.normal(size=args[i].shape)
            up, down = [list(args) for _ in range(2)]
            up[i], down[i] = args[i] + h * v, args[i] - h * v
            # truncation h^2 times a third derivative of order 10, rounding 1e-15 / h times the loss of order 100
            assert abs((loss(*up) - loss(*down)) / (2 * h) - float((grad * v).sum())) < 1e-6


def _weights(**change):
    w = P._FfnWeights(1 << 20, 1 << 22, 1 << 24, 64, 64, 128, 64, 128)
    for k, v in change.items():
        setattr(w, k, v)
    return w


def test_refusals():
    """Every refused call returns its status before any CUDA call."""
    from dynamic_block_sparse_shape_b200 import build
    build.build()
    lib, big = P.lib(), 1 << 40
    A = 1 << 30  # activations' addresses from here on, far from the weights

    def fwd(w=None, m=4, act=0, dtype=0, x=A, sx=64, y=A + (1 << 16), sy=64, gate=None, up=None, ws=1 << 34, nb=big):
        return lib.prism_gated_ffn_fwd(ctypes.byref(w or _weights()), m, act, dtype, x, sx, y, sy, gate, up, ws, nb, None)

    def bwd(w=None, m=4, act=0, dtype=0, dy=A, sdy=64, x=A + (1 << 16), sx=64, gate=A + (2 << 16), up=A + (3 << 16),
            dx=A + (4 << 16), sdx=64, g=A + (5 << 16), u=A + (6 << 16), d=A + (7 << 16), ws=1 << 34, nb=big):
        return lib.prism_gated_ffn_bwd(ctypes.byref(w or _weights()), m, act, dtype, dy, sdy, x, sx, gate, up, dx, sdx, g,
                                       u, d, ws, nb, None)

    for call in (fwd, bwd):
        assert call(dtype=1) == 3 and call(act=4) == 1 and call(act=-1) == 1 and call(m=-1) == 1
        assert call(m=(1 << 30) + 1) == 9
        assert call(_weights(d=60, gate_stride=64, up_stride=64)) == 9 and call(_weights(f=132)) == 9
        assert call(_weights(w_gate=None)) == 1 and call(_weights(w_up=(1 << 22) + 8)) == 1
        assert call(_weights(gate_stride=56)) == 1 and call(_weights(down_stride=130)) == 1
        assert call(_weights(up_stride=1 << 31)) == 9
        assert call(x=None) == 1 and call(x=A + (1 << 16) + 8) == 1 and call(sx=60) == 1
        assert call(ws=None) == 4 and call(ws=(1 << 34) + 8) == 4 and call(nb=256) == 4
    assert fwd(y=None) == 1 and fwd(sy=72 + 4) == 1
    assert fwd(gate=A + (2 << 16)) == 1 and fwd(gate=A + (2 << 16), up=A + (2 << 16) + 8) == 1
    assert fwd(gate=A + (2 << 16), up=A + (2 << 16) + 256) == 1  # the projections over one another
    assert fwd(gate=A, up=A + (2 << 16)) == 1 and fwd(gate=1 << 24, up=A + (2 << 16)) == 1  # over x, over a weight
    assert fwd(y=1 << 24) == 1  # y over the second weight
    assert bwd(dx=None, g=None, u=None, d=None) == 1 and bwd(u=None) == 1
    assert bwd(dy=None) == 1 and bwd(gate=None) == 1 and bwd(up=A + 8) == 1 and bwd(sdx=65) == 1
    assert bwd(dx=A) == 1 and bwd(dx=A + (1 << 16) + 128) == 1  # over dy, over part of x
    assert bwd(g=A + (6 << 16)) == 1 and bwd(d=1 << 20) == 1  # outputs over one another, over a weight
    b = ctypes.c_size_t()
    assert lib.prism_gated_ffn_workspace_size(-1, 8, 0, ctypes.byref(b)) == 1
    assert lib.prism_gated_ffn_workspace_size(4, 8, 0, None) == 1
    assert lib.prism_gated_ffn_workspace_size(1 << 31, 8, 0, ctypes.byref(b)) == 9
    assert lib.prism_gated_ffn_workspace_size(1000, 128, 1, ctypes.byref(b)) == 0 and b.value == 256 + 3 * 256000
    x, wg, wu, wd, dy = draw(4, 64, 128, 1, device="cpu")
    for bad in (dict(act="tanh"), dict()):  # an activation that is none; not on a GPU
        with pytest.raises(P.PrismError):
            P.gated_ffn_fwd(x, wg, wu, wd, **bad)
    for args in ((x, wg[:64], wu, wd), (x, wg, wu.t(), wd), (x[:, :32], wg, wu, wd), (x.float(), wg, wu, wd),
                 (x, wg, wu, wd[:, ::2])):
        with pytest.raises(P.PrismError):
            P.gated_ffn_fwd(*args)


def test_refusals_of_shared_memory():
    """y over any weight, and any tensor over the workspace, are refused before any CUDA call."""
    from dynamic_block_sparse_shape_b200 import build
    build.build()
    lib, w = P.lib(), _weights()
    A, far = 1 << 30, 1 << 34
    need = {}
    for backward in (0, 1):
        b = ctypes.c_size_t()
        assert lib.prism_gated_ffn_workspace_size(4, 128, backward, ctypes.byref(b)) == 0
        need[backward] = b.value

    def fwd(x=A, y=A + (1 << 16), gate=A + (2 << 16), up=A + (3 << 16), ws=far):
        return lib.prism_gated_ffn_fwd(ctypes.byref(w), 4, 0, 0, x, 64, y, 64, gate, up, ws, 1 << 40, None)

    def bwd(dy=A, x=A + (1 << 16), gate=A + (2 << 16), up=A + (3 << 16), dx=A + (4 << 16), g=A + (5 << 16),
            u=A + (6 << 16), d=A + (7 << 16), ws=far):
        return lib.prism_gated_ffn_bwd(ctypes.byref(w), 4, 0, 0, dy, 64, x, 64, gate, up, dx, 64, g, u, d, ws, 1 << 40, None)

    for weight, last in ((1 << 20, 128 * 128 - 16), (1 << 22, 128 * 128 - 16), (1 << 24, 64 * 256 - 16)):
        for y in (weight, weight + last, weight - 16):
            assert fwd(y=y) == 1
        for ws in (weight, weight - 256):
            assert fwd(ws=ws) == 1 and bwd(ws=ws) == 1
    for call, names, n in ((fwd, ("x", "y", "gate", "up"), need[0]),
                           (bwd, ("dy", "x", "gate", "up", "dx", "g", "u", "d"), need[1])):
        for name in names:  # over the first and the last bytes that the call uses
            assert call(**{name: far}) == 1 and call(**{name: far + n - 16}) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [8, 20, 40, 300])
def test_far_projections(m, act):
    """Projections up to the type's largest: the activation is g or 0 there and its slope 1 or 0, never NaN from a power
    of g that overflows."""
    require_gpu()
    far = torch.tensor([0.0, -0.0, 3.0, -3.0, 1e12, -1e12, 1.7e19, -1.7e19, 1e25, -1e25, 3e38, -3e38, 1e-30, -1e-30],
                       dtype=torch.bfloat16)
    g = far[torch.arange(m) % len(far)]
    eye = torch.eye(8, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(m, 8, dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = g, 1.0
    wg, wu = torch.zeros(8, 8, dtype=torch.bfloat16), torch.zeros(8, 8, dtype=torch.bfloat16)
    wg[:, 0], wu[:, 1] = 1.0, 0.5
    y, gate, up = P.gated_ffn_fwd(x.cuda(), wg.cuda(), wu.cuda(), eye, act=act)
    assert torch.equal(gate, g.cuda()[:, None].expand(m, 8)) and (up == 0.5).all()
    a, slope = O.activation(act, f64(gate)), O.activation_slope(act, f64(gate))
    # the exponential's 2^-20 (1 + |g|) counts where it is not saturated; one rounding of h and one of y
    tol = (2.0 ** -20 * (1 + np.minimum(np.abs(f64(gate)), 200.0)) + 2 * STEP * (1 + STEP)) * np.abs(a * 0.5) + 2.0 ** -120
    assert (np.abs(f64(y) - a * 0.5) <= tol).all()
    dy = torch.full((m, 8), 2.0 ** -4, dtype=torch.bfloat16, device="cuda")
    dx = P.gated_ffn_bwd(dy, x.cuda(), eye, torch.zeros_like(eye), eye, gate, up, act=act, need_dw=False)[0]
    want = 2.0 ** -4 * 0.5 * slope
    tol = (2.0 ** -19 * (1 + 9.0) + 2 * STEP * (1 + STEP)) * np.maximum(np.abs(want), 2.0 ** -6) + 2.0 ** -120
    assert (np.abs(f64(dx) - want) <= tol).all()


# with SIZES and LARGE, every kernel and split of K that a product can take: see test_every_form_is_reached
FORMS = [(769, 8, 8), (17, 8, 328), (6194, 536, 8), (1973, 864, 8), (1142, 1968, 8), (17, 328, 2176), (1, 328, 9848),
         (17, 2192, 1104), (41, 2392, 520), (26, 200, 9760), (29, 1008, 1096), (28, 856, 2408),
         # pairs of CTAs with K in two parts: the last pair's second CTA with rows of its own, or wholly behind the last
         (780, 1480, 728), (413, 1464, 1216), (643, 1552, 1704), (793, 1408, 1648)]
PRODUCTS = ("gate", "down", "gradient of the gate", "dx", "weight gradients")


def forms(m, d, f):
    """The kernel of each product of a block: CTAs that share a tile, its columns (0: persistent), parts of K; whether
    remainders come along; and of split pairs whether the last one's second CTA has rows."""
    w, a, b = P._FfnWeights(0, 0, 0, d, d, f, d, f), (ctypes.c_int32 * 9)(), (ctypes.c_int32 * 9)()
    assert P.lib().prism_gated_ffn_forms(ctypes.byref(w), m, 0, a) == 0
    assert P.lib().prism_gated_ffn_forms(ctypes.byref(w), m, 1, b) == 0
    found = set()
    for name, c in zip(PRODUCTS, (tuple(x) for x in (a[0:3], a[3:6], b[0:3], b[3:6], b[6:9]))):
        found.add((name, c, m <= 32, 1 <= m % 256 <= 128 if c[:2] == (2, 256) and name != PRODUCTS[4] else None))
    return found


def test_every_form_is_reached():
    """The sizes of this file take every kernel that the choice takes over a wide range, so that a change of the choice
    leaves none of them untested."""
    from dynamic_block_sparse_shape_b200 import build
    build.build()
    reached = set().union(*(forms(*s) for s in SIZES + LARGE + FORMS))
    r = np.random.default_rng(0)
    many = np.exp(r.uniform(np.log([1, 1, 1]), np.log([16384, 512, 1408]), (20000, 3))).round().astype(int)
    missing = {}
    for m, d, f in many:
        for k in forms(int(m), 8 * int(d), 8 * int(f)) - reached:
            missing.setdefault(k, (m, 8 * d, 8 * f))
    assert not missing
    split = {n for n, c, _, _ in reached if c == (2, 256, 2)}
    assert split == set(PRODUCTS)  # pairs that split K, in every product
    w, a = P._FfnWeights(0, 0, 0, 8, 8, 8, 8, 8), (ctypes.c_int32 * 9)()
    call = P.lib().prism_gated_ffn_forms
    assert call(None, 1, 0, a) == 1 and call(ctypes.byref(w), 1, 0, None) == 1 and call(ctypes.byref(w), -1, 0, a) == 1
    a[0] = 7
    assert call(ctypes.byref(w), 0, 1, a) == 0 and list(a) == [0] * 9


@pytest.mark.gpu
@pytest.mark.parametrize("m,d,f", FORMS)
def test_every_form(m, d, f):
    require_gpu()
    act = ACTS[FORMS.index((m, d, f)) % len(ACTS)]
    x, wg, wu, wd, dy = draw(m, d, f, m + d)
    ws = P.Workspace("cuda")
    y, g, u = P.gated_ffn_fwd(x, wg, wu, wd, act=act, ws=ws)
    got = P.gated_ffn_bwd(dy, x, wg, wu, wd, g, u, act=act, ws=ws)
    P.check_device_status(ws)
    check_fwd(x, wg, wu, wd, act, y, g, u)
    check_bwd(dy, x, wg, wu, wd, g, u, act, got)


@pytest.mark.gpu
def test_wide_backward_repeats_itself():
    """The same bits from several hundred calls. A copy of the saved projections of the epilogue's next piece that did not
    wait for the reads of the last one changed a few rows of one call in fifty here."""
    require_gpu()
    m, d, f = 8192, 4096, 11264
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    dy, gate, up, wg, wu, wd = n(m, d), n(m, f), n(m, f), n(f, d), n(f, d), n(d, f)
    ws = P.Workspace("cuda")

    def call(need_dw=False):
        return P.gated_ffn_bwd(dy, dy, wg, wu, wd, gate, up, need_dw=need_dw, ws=ws)

    dx, *dw = call(True)
    off = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(400):
        off += (call()[0] != dx).sum()
    for _ in range(50):
        off += sum((a != b).sum() for a, b in zip(call(True), (dx, *dw)))
    P.check_device_status(ws)
    assert int(off) == 0
