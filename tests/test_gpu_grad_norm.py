"""Global gradient norm and clipping against the fp64 form.

Tolerances. A sum of squares is added in fp32 over at most 16 terms a chain, then in fp64: at most 17 roundings of
2^-24 of a sum of positive terms, half of that in its root, and the fp32 result rounds by 2^-24: below 16 * 2^-24 of
the norm. The factor is formed from the fp64 norm, so it is off by that much and 2^-24 for its own rounding; the product
and the storing round by half a step each.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import dynamic_block_sparse_shape_b200 as P
from oracle import layer_oracle as O
from tests.gpu_util import f64, require_gpu

NORM_TOL = 16 * 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def tensors(sizes, seed, kinds=(torch.bfloat16, torch.float32), scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(kinds[i % len(kinds)]).cuda() for i, n in enumerate(sizes)]


def check(got, was, factor):
    for a, b in zip(got, was):
        want = f64(b) * factor
        tol = (NORM_TOL + 2 * 2.0 ** -24) * np.abs(want)
        tol = tol + HALF_STEP[b.dtype] * (np.abs(want) + tol) + (2.0 ** -134 if b.dtype == torch.bfloat16 else 2.0 ** -150)
        assert (np.abs(f64(a) - want) <= tol).all()


LISTS = [[1], [0, 1, 0], [5, 3], [4096], [8192, 8193, 8191], [0], [40001, 7, 123457, 1, 2],
         list(range(1, 41)), list(range(0, 950)), [3000001, 17, 5000000]]


@pytest.mark.gpu
@pytest.mark.parametrize("kinds", [(torch.bfloat16,), (torch.float32,), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{sum(s)}")
def test_norm_and_clip(sizes, kinds):
    require_gpu()
    g = tensors(sizes, len(sizes), kinds)
    ref = O.grad_norm([f64(t) for t in g])
    ws = P.Workspace("cuda")
    n = P.grad_norm(g, ws=ws)
    assert abs(float(n) - ref) <= NORM_TOL * ref
    top = P.grad_norm(g, ord=math.inf, ws=ws)
    assert float(top) == O.grad_norm([f64(t) for t in g], math.inf)  # a maximum rounds nothing
    for ratio in (0.3, 2.0):
        limit = ratio * ref if ref else 1.0
        out = [torch.full_like(t, 5.0) for t in g]
        was = [t.clone() for t in g]
        n2 = P.clip_grad_norm(g, limit, out=out, ws=ws)
        assert float(n2) == float(n)
        assert all(torch.equal(a, b) for a, b in zip(g, was))
        check(out, was, O.clip_factor(ref, limit))
        if ratio > 1:
            assert all(torch.equal(a, b) for a, b in zip(out, was))
        g2 = [t.clone() for t in g]
        P.clip_grad_norm(P.GradList(g2), limit, ws=ws)  # in place: the same bits
        assert all(torch.equal(a, b) for a, b in zip(g2, out))
        g3 = [t.clone() for t in g]
        P.scale_grads(g3, n, limit)  # from the norm rounded to fp32
        check(g3, was, O.clip_factor(ref, limit))


@pytest.mark.gpu
@pytest.mark.parametrize("shift_in,shift_out", [(0, 0), (1, 1), (3, 0), (0, 5), (7, 2), (9, 1)])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_alignment(kind, shift_in, shift_out):
    """Tensors at any offset of whole elements; what lies around the outputs stays."""
    require_gpu()
    for n in (1, 2, 7, 8, 9, 1000, 4099, 20000):
        src = tensors([n + 32], n, (kind,))[0]
        dst = torch.full((n + 32,), -3.0, dtype=kind, device="cuda")
        a, b = src[shift_in:shift_in + n], dst[shift_out:shift_out + n]
        ref = O.grad_norm([f64(a)])
        norm = P.clip_grad_norm([a], 0.5 * ref, out=[b])
        assert abs(float(norm) - ref) <= NORM_TOL * ref
        check([b], [a], O.clip_factor(ref, 0.5 * ref))
        assert (dst[:shift_out] == -3).all() and (dst[shift_out + n:] == -3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-18, 1e18, 1e25, 3e35])
def test_far_magnitudes(scale):
    """Squares below the smallest and above the largest fp32 number still count."""
    require_gpu()
    for sizes in ([1000], [5, 12345], [300000]):
        g = tensors(sizes, 3, (torch.float32, torch.bfloat16), scale)
        ref = O.grad_norm([f64(t) for t in g])
        n = P.clip_grad_norm(g, ref / 2, eps=0.0, out=[torch.empty_like(t) for t in g])
        assert ref < 3e38 and abs(float(n) - ref) <= NORM_TOL * ref
    mixed = [torch.full((100,), 1e-25, device="cuda"), torch.full((3,), 2e-25, device="cuda")]
    ref = O.grad_norm([f64(t) for t in mixed])
    assert abs(float(P.grad_norm(mixed)) - ref) <= NORM_TOL * ref


@pytest.mark.gpu
def test_nonfinite_and_empty():
    require_gpu()
    assert float(P.grad_norm([])) == 0.0 and float(P.clip_grad_norm([], 1.0)) == 0.0
    e = torch.empty(0, device="cuda")
    assert float(P.clip_grad_norm([e], 1.0)) == 0.0
    for o in (2, math.inf):
        g = tensors([100, 20000], 5)
        g[1][777] = float("nan")
        assert math.isnan(float(P.grad_norm(g, ord=o)))
        P.clip_grad_norm(g, 1.0, ord=o)
        assert all(torch.isnan(t).all() for t in g)
        g = tensors([100, 20000], 5)
        g[0][5] = -float("inf")
        assert float(P.grad_norm(g, ord=o)) == math.inf
        P.clip_grad_norm(g, 1.0, ord=o)
        assert torch.isnan(g[0][5]) and (g[1] == 0).all()
    z = [torch.zeros(5000, device="cuda")]
    assert float(P.clip_grad_norm(z, 0.0)) == 0.0 and (z[0] == 0).all()
    g = tensors([1000], 6, (torch.float32,))
    was = g[0].clone()
    P.clip_grad_norm(g, math.inf)
    assert torch.equal(g[0], was)
    # a tensor listed twice counts twice in a norm, and cannot be scaled
    n1 = float(P.grad_norm(g))
    assert abs(float(P.grad_norm(g + g)) - math.sqrt(2) * n1) <= 2 * NORM_TOL * n1
    with pytest.raises(P.PrismError) as err:
        P.clip_grad_norm(g + g, 1.0)
    assert err.value.status == 1 and torch.equal(g[0], was)


@pytest.mark.gpu
def test_dense_in_any_order_and_zeros():
    require_gpu()
    g = [t.view(40, 30, 50) for t in tensors([60000, 60000], 12)]
    turned = [g[0].permute(2, 0, 1), g[1].transpose(0, 2)]
    ref = O.grad_norm([f64(t) for t in g])
    norm = P.clip_grad_norm(turned, ref / 4)
    assert abs(float(norm) - ref) <= NORM_TOL * ref
    assert abs(O.grad_norm([f64(t) for t in g]) - ref / 4) <= 2.0 ** -8 * ref / 4
    # zeros around one value, and values that a square loses in fp32
    z = torch.zeros(100000, device="cuda")
    z[777] = 3.0
    assert float(P.grad_norm([z, torch.zeros_like(z)])) == 3.0
    z[777] = 2.0 ** -100
    assert float(P.grad_norm([z])) == 2.0 ** -100
    z[777] = float("nan")
    was = torch.arange(5.0, device="cuda")
    keep = was.clone()
    P.clip_grad_norm([z, was], math.inf)  # nothing to clip to: whatever the norm
    assert torch.equal(was, keep)


@pytest.mark.gpu
def test_same_bits_stream_and_graph():
    require_gpu()
    g = tensors([1000003, 17, 250000], 7)
    ws = P.Workspace("cuda")
    first = P.grad_norm(g, ws=ws)
    for _ in range(5):
        assert torch.equal(P.grad_norm(g, ws=ws), first)
    out = [torch.empty_like(t) for t in g]
    want = [torch.empty_like(t) for t in g]
    lst, ref = P.GradList(g, out=out), P.GradList(g, out=want)
    P.clip_grad_norm(ref, 10.0, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = P.clip_grad_norm(lst, 10.0, stream=side)
    side.synchronize()
    assert torch.equal(n, first) and all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = P.clip_grad_norm(lst, 10.0, ws=ws)
    g[0].mul_(3.0)
    graph.replay()
    P.clip_grad_norm(ref, 10.0)
    torch.cuda.synchronize()
    now = O.grad_norm([f64(t) for t in g])  # tripling 1000003 of 1250020 squares of one size: about 2.72 times the first
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and abs(float(n) - now) <= NORM_TOL * now


def _raw(call, entries, *rest):
    arr = (P._Tensor * max(1, len(entries)))(*entries)
    return getattr(P.lib(), call)(arr, len(entries), *rest)


def test_refusals():
    """Every refused call returns its status before any CUDA call."""
    from dynamic_block_sparse_shape_b200 import build
    build.build()
    p, ws, ok = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 24), (1 << 21, None, 100, 0, 0)
    big = 1 << 30
    norm = lambda e, *a: _raw("prism_grad_norm", e, *a)  # noqa: E731
    clip = lambda e, m=1.0, eps=1e-6: _raw("prism_grad_clip", e, 0, m, eps, p, ws, big, None)  # noqa: E731
    scale = lambda e, m=1.0, eps=1e-6, n=p: _raw("prism_grad_scale", e, n, m, eps, None)  # noqa: E731
    assert norm([ok], 0, None, ws, big, None) == 1
    assert norm([ok], 2, p, ws, big, None) == 1
    assert norm([ok], 0, p, None, big, None) == 4 and norm([ok], 0, p, ws, 256, None) == 4
    assert norm([ok], 0, p, ctypes.c_void_p((1 << 24) + 8), big, None) == 4
    assert norm([(1 << 21, None, 100, 2, 0)], 0, p, ws, big, None) == 3
    assert norm([(None, None, 100, 0, 0)], 0, p, ws, big, None) == 1
    assert norm([((1 << 21) + 1, None, 100, 0, 0)], 0, p, ws, big, None) == 1
    assert norm([((1 << 21) + 2, None, 100, 1, 0)], 0, p, ws, big, None) == 1
    assert norm([(1 << 21, None, -1, 0, 0)], 0, p, ws, big, None) == 1
    assert norm([(1 << 21, None, 1 << 44, 0, 0)], 0, p, ws, big, None) == 9
    for f in (clip, scale):
        assert f([ok], float("nan")) == 1 and f([ok], -1.0) == 1 and f([ok], 1.0, -1.0) == 1
        assert f([ok, ok]) == 1  # the same tensor twice
        assert f([ok, ((1 << 21) + 198, None, 10, 0, 0)]) == 1  # two that meet
        assert f([(1 << 21, (1 << 21) + 4, 100, 0, 0)]) == 1  # over its own input, shifted
        assert f([(1 << 21, 1 << 22, 100, 0, 0), (1 << 22, 1 << 23, 100, 0, 0)]) == 1  # over the next one's input
        assert f([(1 << 21, 1 << 22, 100, 0, 0), (1 << 23, 1 << 22, 100, 0, 0)]) == 1  # two outputs in one place
        assert f([(1 << 21, (1 << 22) + 1, 100, 0, 0)]) == 1
    assert scale([ok], n=None) == 1
    b = ctypes.c_size_t()
    assert P.lib().prism_grad_norm_workspace_size(-1, ctypes.byref(b)) == 1
    assert P.lib().prism_grad_norm_workspace_size((1 << 20) + 1, ctypes.byref(b)) == 9
    assert scale([((1 << 20), None, 100, 0, 0)]) == 1  # over the norm itself
    with pytest.raises(P.PrismError):
        P.GradList([torch.zeros(4, 4).t()[1:]])
    with pytest.raises(P.PrismError):
        P.GradList([torch.zeros(4, 6)], out=[torch.zeros(6, 4).t()])
    with pytest.raises(P.PrismError):
        P.GradList([torch.zeros(4)], out=[])
    with pytest.raises(P.PrismError):
        P.GradList([torch.zeros(4, dtype=torch.float16)])
    with pytest.raises(P.PrismError):
        P.grad_norm([torch.zeros(4)], ord=3)


def test_refusals_of_shared_memory():
    """The norm or the workspace over a tensor or over one another, before any CUDA call."""
    from dynamic_block_sparse_shape_b200 import build
    build.build()
    ws, norm, big = 1 << 24, 1 << 20, 1 << 30
    b = ctypes.c_size_t()
    assert P.lib().prism_grad_norm_workspace_size(1, ctypes.byref(b)) == 0
    calls = [lambda e, n=norm: _raw("prism_grad_norm", e, 0, n, ws, big, None),
             lambda e, n=norm: _raw("prism_grad_clip", e, 0, 1.0, 1e-6, n, ws, big, None)]
    for call in calls:
        for at in (ws, ws - 196, ws + b.value - 4):
            assert call([(at, None, 100, 0, 0)]) == 1
        assert call([(norm, None, 100, 0, 0)]) == 1 and call([(norm - 196, None, 100, 0, 0)]) == 1
        assert call([(1 << 21, None, 100, 0, 0)], ws + 4) == 1 and call([], ws + b.value - 4) == 1
    for at in (ws, ws - 196, ws + b.value - 4, norm):
        assert calls[1]([(1 << 21, at, 100, 0, 0)]) == 1  # where the scaled values go


@pytest.mark.gpu
@pytest.mark.parametrize("n", [100, 300000])
def test_nothing_to_scale_by(n):
    """A norm of 0 and eps = 0 leave the values whatever the bound, 0 among them: no 0 / 0."""
    require_gpu()
    for limit in (0.0, 1.0):
        z = [torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")]
        assert float(P.clip_grad_norm(z, limit, eps=0.0)) == 0.0 and all((t == 0).all() for t in z)
        one = [torch.ones(n, device="cuda")]
        P.scale_grads(one, torch.zeros((), device="cuda"), limit, eps=0.0)
        assert (one[0] == 1).all()
    one = [torch.ones(n, device="cuda")]
    P.clip_grad_norm(one, 0.0, eps=0.0)
    assert (one[0] == 0).all()
