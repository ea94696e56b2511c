"""Rotary positions against the fp64 form.

Tolerances. The angle's fraction of a turn is exact to fp64 rounding and is rounded to fp32 once: an error below
2^-25 turns, so below pi 2^-24 in radians; sin and cos of the library are within 2 ulp (2^-23 at most for values up to
1), the two products and their sum round at most 2 * 2^-24 of the operands' magnitudes. With |x| = max(|x1|, |x2|) the
fp32 result is off by at most (2 (pi + 2 + 2) 2^-24 + ...) |x| < 16 * 2^-24 |m| |x|, and storing it rounds by half a step
of its type (bf16 2^-8 of the value as an upper bound of eps / 2, fp32 2^-24).
"""
import numpy as np
import pytest
import torch

import dynamic_block_sparse_shape_b200 as P
from oracle import layer_oracle as O
from tests.gpu_util import f64, require_gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def check(got, x, angles, layout, magnitude=1.0, transposed=False):
    want = O.rope(f64(x), angles, layout, magnitude, transposed)
    pairs = angles.shape[1]
    xa = np.abs(f64(x))
    big = np.zeros_like(xa)
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + pairs)
        big[..., a] = big[..., b] = np.maximum(xa[..., a], xa[..., b])
    tol = 16 * 2.0 ** -24 * abs(magnitude) * big
    tol = tol + HALF_STEP[x.dtype] * (np.abs(want) + tol) * (big > 0)
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), float((err - tol).max())
    # the channels behind the rotated ones keep their bits
    assert torch.equal(got[..., 2 * pairs:], x[..., 2 * pairs:])


def draw(n, h, d, dtype, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((n, h, d), generator=g).to(dtype).to(device)


CASES = [
    # dims, head_dim, hq, hk, grid
    ((44, 42, 42), 128, 24, 24, (3, 5, 7)),
    ((16, 12, 12), 64, 12, 4, (13, 3, 5)),
    ((2, 0, 0), 64, 1, 1, (1, 1, 1)),
    ((0, 2, 4), 6, 3, 1, (2, 3, 4)),
    ((10, 6, 2), 48, 5, 2, (1, 9, 31)),
    ((86, 86, 84), 256, 2, 2, (4, 4, 9)),
    ((6, 10, 10), 80, 32, 8, (2, 17, 33)),
    # halves of 13, 18 and 20 channels under many tokens; a token of more than a CTA's shared memory
    ((10, 8, 8), 64, 3, 1, (17, 9, 11)),
    ((12, 12, 12), 40, 6, 2, (5, 21, 40)),
    ((20, 10, 10), 64, 20, 4, (16, 20, 16)),
    ((84, 84, 86), 256, 50, 10, (1, 3, 5)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dims,d,hq,hk,grid", CASES)
def test_grid(dims, d, hq, hk, grid, dtype, layout):
    require_gpu()
    n = int(np.prod(grid))
    q, k = draw(n, hq, d, dtype, 1), draw(n, hk, d, dtype, 2)
    spec = P.RopeSpec(dims, layout=layout)
    ang = O.rope_angles(dims, grid=grid)
    for fn, tr in ((P.rope, False), (P.rope_bwd, True)):
        yq, yk = fn(q, k, spec, grid=grid)
        check(yq, q, ang, layout, transposed=tr)
        check(yk, k, ang, layout, transposed=tr)
        # in place: the same bits
        q2, k2 = q.clone(), k.clone()
        fn(q2, k2, spec, grid=grid, out=(q2, k2))
        assert torch.equal(q2, yq) and torch.equal(k2, yk)


@pytest.mark.gpu
@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", {"factor": 4.0}), ("ntk", {"factor": 8.0}),
                                        ("yarn", {"factor": 8.0, "trained_len": 4096.0}),
                                        ("yarn", {"factor": 2.0, "trained_len": 100.0})])
@pytest.mark.parametrize("n,rot,d,layout", [(1, 64, 128, "half"), (7, 26, 48, "half"), (129, 128, 128, "interleaved"),
                                            (3000, 2, 96, "interleaved"), (33, 256, 256, "half")])
def test_positions(n, rot, d, layout, scaling, kw):
    """Given positions over the whole int32 range, single tokens among them, grouped heads."""
    require_gpu()
    g = torch.Generator().manual_seed(n)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, 1), generator=g).to(torch.int32)
    pos[0] = 2 ** 31 - 1
    if n > 1:
        pos[1], pos[-1] = 0, -2 ** 31
    q, k = draw(n, 8, d, torch.float32, 3), draw(n, 2, d, torch.float32, 4)
    spec = P.RopeSpec((rot,), layout=layout, theta=500000.0, scaling=scaling, **kw)
    ang = O.rope_angles((rot,), positions=pos.numpy(), theta=500000.0, scaling=scaling, **kw)
    yq, yk = P.rope(q, k, spec, positions=pos.cuda())
    # at 2^31 radians one fp64 rounding is 2^-22 radians, and either side rounds about seven times on its way (the power
    # twice that, the stretching, the scale, the product): 16 * 2^-22 = 2^-18 radians, times |x1| + |x2| <= 2 |x|
    for y, x in ((yq, q), (yk, k)):
        want = O.rope(f64(x), ang, layout, spec.magnitude)
        big = np.abs(f64(x)).max(axis=-1, keepdims=True)
        assert (np.abs(f64(y) - want) <= spec.magnitude * big * (2.0 ** -17 + 17 * 2.0 ** -24)).all()


@pytest.mark.gpu
def test_index_scale_offset_magnitude():
    """A one-axis spec without positions takes the token's index; fractional scale, offset and magnitude."""
    require_gpu()
    x = draw(1000, 3, 64, torch.float32, 5)
    spec = P.RopeSpec((64,), pos_scale=(21.533203125 / 6.0,), pos_offset=(-17.25,), magnitude=0.5)
    y, none = P.rope(x, None, spec)
    assert none is None
    check(y, x, O.rope_angles((64,), n=1000, pos_scale=(21.533203125 / 6.0,), pos_offset=(-17.25,)), "interleaved", 0.5)
    # the transposed rotation is the gradient: <R x, y> = <x, R^T y>, and differences of a sum agree with it
    w = draw(1000, 3, 64, torch.float32, 6)
    g, _ = P.rope_bwd(w, None, spec)
    lhs, rhs = float((f64(y) * f64(w)).sum()), float((f64(x) * f64(g)).sum())
    assert abs(lhs - rhs) <= 32 * 2.0 ** -24 * float(np.abs(f64(x) * f64(g)).sum())
    e = torch.zeros_like(x)
    e[17, 1, 5] = 1.0
    up, _ = P.rope(x + e, None, spec)
    diff = float(((f64(up) - f64(y)) * f64(w)).sum())
    # a rotation is linear: the difference of step 1 is the derivative, up to the roundings of two results of size 4
    assert abs(diff - float(g[17, 1, 5])) <= 4 * 64 * 2.0 ** -22


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_strides_and_alignment(dtype, layout, shift):
    """Views of a packed QKV buffer at any offset of whole elements, rotated in place: the rest stays as it was."""
    require_gpu()
    n, h, d, hk = 50, 6, 32, 2
    width = (h + 2 * hk) * d + 5 + shift
    base = draw(n + 1, 1, width, dtype, 7).view(-1)
    was = base.clone()
    rows = base[shift:shift + n * width].view(n, width)
    q = rows[:, :h * d].unflatten(1, (h, d))
    k = rows[:, h * d:(h + hk) * d].unflatten(1, (hk, d))
    spec = P.RopeSpec((12, 6, 6), layout=layout)
    grid = (2, 5, 5)
    ang = O.rope_angles((12, 6, 6), grid=grid)
    q0, k0 = q.clone(), k.clone()
    P.rope(q, k, spec, grid=grid, out=(q, k))
    check(q.contiguous(), q0, ang, layout)
    check(k.contiguous(), k0, ang, layout)
    rest = torch.ones_like(base, dtype=torch.bool)
    rest[shift:shift + n * width].view(n, width)[:, :(h + hk) * d] = False
    assert torch.equal(base[rest], was[rest])
    # out of place with other strides
    out = torch.full((n, h + 1, d), 7.0, dtype=dtype, device="cuda")[:, 1:]
    P.rope(q0, None, spec, grid=grid, out=out)
    assert torch.equal(out, q)


@pytest.mark.gpu
def test_nonfinite_channels_stay_apart():
    """Infinities and NaN in channels behind the rotated ones, and in one pair, touch nothing else."""
    require_gpu()
    x = draw(20, 2, 64, torch.bfloat16, 8)
    y0, _ = P.rope(x, None, P.RopeSpec((18,)))
    x2 = x.clone()
    x2[:, :, 18:] = float("nan")
    x2[3, 1, 40] = float("inf")
    x2[5, 0, 4] = float("inf")
    y, _ = P.rope(x2, None, P.RopeSpec((18,)))
    assert torch.equal(y[..., 18:].view(torch.int16), x2[..., 18:].view(torch.int16))
    same = torch.ones_like(y[..., :18], dtype=torch.bool)
    same[5, 0, 4:6] = False
    assert torch.equal(y[..., :18][same], y0[..., :18][same])


@pytest.mark.gpu
def test_streams_graph_and_empty():
    require_gpu()
    spec = P.RopeSpec((44, 42, 42))
    grid = (2, 9, 11)
    q, k = draw(198, 24, 128, torch.bfloat16, 9), draw(198, 24, 128, torch.bfloat16, 10)
    want = P.rope(q, k, spec, grid=grid)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = P.rope(q, k, spec, grid=grid, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = P.rope(q, k, spec, grid=grid)
    q.copy_(draw(198, 24, 128, torch.bfloat16, 11))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], P.rope(q, k, spec, grid=grid)[0]) and torch.equal(out[1], want[1])
    y, z = P.rope(q[:0], k[:0], spec, grid=(0, 9, 11))
    assert y.shape == (0, 24, 128) and z.shape == (0, 24, 128)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A tensor of more than 2^32 elements between its first and last token."""
    require_gpu()
    stride = 1 << 22
    n = 1100  # 1100 * 2^22 > 2^32 elements, 9.2 GB in bf16
    buf = torch.zeros(n * stride, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((n, 2, 64), (stride, 64, 1))
    v = draw(n, 2, 64, torch.bfloat16, 12)
    x.copy_(v)
    spec = P.RopeSpec((64,), layout="half")
    P.rope(x, None, spec, out=x)
    check(x.contiguous(), v, O.rope_angles((64,), n=n), "half")


def _call(params=None, grid=None, pos=None, n=4, q=1 << 20, qo=1 << 21, hq=2, sq=128, so=128, k=None, ko=None, hk=0,
          sk=0, sko=0, dtype=0, d=64, **change):
    import ctypes
    spec = P.RopeSpec((64,)) if params is None else params
    c = P._RopeParams.from_buffer_copy(spec._c)
    for key, v in change.items():
        setattr(c, key, v)
    p = lambda a: None if a is None else ctypes.c_void_p(a)  # noqa: E731
    g = None if grid is None else ctypes.byref(P._Dim3(*grid))
    return P.lib().prism_rope(ctypes.byref(c), g, p(pos), n, p(q), p(qo), hq, sq, so, p(k), p(ko), hk, sk, sko, dtype, d,
                              0, None)


def test_refusals():
    """Every refused call returns its status before any CUDA call."""
    from dynamic_block_sparse_shape_b200 import build
    build.build()
    three = P.RopeSpec((20, 22, 22))
    assert _call(q=None) == 1 and _call(qo=None) == 1
    assert _call(dtype=2) == 3
    assert _call(d=63) == 9 and _call(d=258) == 9 and _call(d=62) == 1  # 64 rotated channels in 62
    assert _call(sq=127) == 1 and _call(so=64) == 1
    assert _call(sq=1 << 32) == 9
    assert _call(n=-1) == 1 and _call(n=(1 << 30) + 1) == 9
    assert _call(q=(1 << 20) + 1) == 1 and _call(dtype=1, q=(1 << 20) + 2) == 1 and _call(pos=(1 << 20) + 2) == 1
    assert _call(hq=0) == 1 and _call(k=1 << 22, ko=1 << 23, hk=0, sk=128, sko=128) == 1
    assert _call(k=1 << 22, ko=None, hk=1, sk=128, sko=128) == 1
    assert _call(three) == 1 and _call(three, grid=(1, 2, 3)) == 2 and _call(three, grid=(-1, -2, 2)) == 1
    assert _call(layout=2) == 1 and _call(scaling=4) == 1 and _call(n_axes=2) == 1
    assert _call(theta=1.0) == 1 and _call(theta=float("nan")) == 1 and _call(theta=float("inf")) == 1
    assert _call(scaling=1, factor=0.0) == 1 and _call(scaling=3, factor=2.0, trained_len=0.0) == 1
    assert _call(magnitude=float("inf")) == 1
    # outputs over other tensors: partly over the own input, over the other input, over the other output
    assert _call(qo=(1 << 20) + 256) == 1
    assert _call(qo=1 << 20, so=256) == 1
    assert _call(k=1 << 21, ko=1 << 22, hk=2, sk=128, sko=128) == 1
    assert _call(k=1 << 22, ko=(1 << 21) + 128, hk=2, sk=128, sko=128) == 1
    assert _call(pos=(1 << 21) + 512) == 1  # the output over the positions
    assert _call(n=0) == 0
    for bad in (dict(layout="halves"), dict(scaling="other"), dict(pos_scale=(1.0, 2.0)),
                dict(scaling="yarn", factor=0.0)):
        with pytest.raises(P.PrismError):
            P.RopeSpec((64,), **bad)
    with pytest.raises(P.PrismError):
        P.RopeSpec((64, 2))
    with pytest.raises(P.PrismError):  # not on a GPU
        P.rope(torch.zeros(1, 1, 64), None, P.RopeSpec((64,)))


@pytest.mark.parametrize("call", [P.rope, P.rope_bwd])
def test_refusals_of_positions(call):
    """Positions of three axes come as [tokens, axes]: the same number of values in another shape is not taken."""
    x, spec = torch.zeros(5, 2, 16), P.RopeSpec((4, 4, 4))
    good = torch.zeros(5, 3, dtype=torch.int32)
    for bad in (good.t().contiguous(), good.view(15), good.view(1, 5, 3), good[:4], good.t().contiguous().t()):
        with pytest.raises(P.PrismError, match="positions"):
            call(x, None, spec, positions=bad)
    with pytest.raises(P.PrismError, match="positions"):
        call(x, None, spec, positions=good.long())
    one = P.RopeSpec((8,))
    for fine, s in ((good, spec), (good[:, 0].contiguous(), one), (torch.zeros(1, 5, dtype=torch.int32), one)):
        with pytest.raises(P.PrismError, match="CUDA device"):  # taken as far as that goes without a GPU
            call(x, None, s, positions=fine)


def test_magnitude_of_a_stretched_context():
    """0.1 ln(factor) + 1 belongs to stretched contexts; one that is not stretched, or shortened, keeps its magnitude."""
    for factor, want in ((8.0, 0.1 * np.log(8.0) + 1), (1.0, 1.0), (0.5, 1.0), (1e-6, 1.0)):
        assert abs(P.RopeSpec((8,), scaling="yarn", factor=factor).magnitude - want) < 1e-15
    assert P.RopeSpec((8,), scaling="yarn", factor=0.5, magnitude=0.75).magnitude == 0.75
    assert P.RopeSpec((8,), scaling="linear", factor=8.0).magnitude == 1.0
    with pytest.raises(P.PrismError):
        P.RopeSpec((8,), scaling="yarn", factor=0.0)
