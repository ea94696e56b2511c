"""Calls on a given stream while the caller's own stream is busy.

Nothing that a call allocates or clears may wait for, or land among, the work that the caller's current stream still has
queued: a call on an idle stream gives the same bits as ever, and is done before that queue is.
"""
import math

import pytest
import torch

import dynamic_block_sparse_shape_b200 as P
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


class Busy:
    """Some tens of milliseconds of ordinary work queued on the current stream, over its own gigabyte."""

    def __init__(self, rounds=150):
        self.x = torch.ones(1 << 28, device="cuda")
        self.rounds, self.end = rounds, torch.cuda.Event()

    def __enter__(self):
        torch.cuda.synchronize()
        for _ in range(self.rounds):
            self.x.mul_(1.0)
        self.end.record()
        return self

    def __exit__(self, *exc):
        torch.cuda.synchronize()


def soil(*streams):
    """Leaves memory full of ones among the allocator's free blocks of each stream."""
    for s in streams:
        with torch.cuda.stream(s):
            junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 20, 1 << 21, 1 << 25, 1 << 27)]
        torch.cuda.synchronize()
        del junk


def flat(r):
    if torch.is_tensor(r):
        return [r]
    if isinstance(r, dict):
        r = list(r.values())
    return [t for x in r if torch.is_tensor(x) or isinstance(x, (tuple, list)) for t in flat(x)]


def same_beside(call, ws=None):
    """`call(stream)` on a side stream beside a busy current one gives the bits that it gives by itself."""
    want = [t.clone() for t in flat(call(None, None))]
    side = torch.cuda.Stream()
    soil(side, torch.cuda.current_stream())
    call(side, None)  # its memory is the allocator's from here on, not the driver's
    soil(side)
    with Busy() as busy:
        got = flat(call(side, ws))
        side.synchronize()
        assert not busy.end.query()  # otherwise nothing was shown
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
    if ws is not None:
        P.check_device_status(ws)


def ffn(m, d, f):
    g = torch.Generator().manual_seed(m)
    n = lambda *s, k=1.0: (torch.randn(s, generator=g) * k).to(torch.bfloat16).cuda()  # noqa: E731
    return n(m, d), n(f, d, k=d ** -0.5), n(f, d, k=d ** -0.5), n(d, f, k=f ** -0.5), n(m, d)


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("m,d,f", [(1, 256, 512), (33, 256, 512), (300, 1160, 392), (2100, 2312, 2056)])
def test_feed_forward(m, d, f, kept):
    """Without a workspace, and with one that has to grow in the call."""
    require_gpu()
    x, wg, wu, wd, dy = ffn(m, d, f)
    same_beside(lambda s, ws: P.gated_ffn_fwd(x, wg, wu, wd, ws=ws, stream=s), P.Workspace("cuda", 256) if kept else None)
    _, g, u = P.gated_ffn_fwd(x, wg, wu, wd)
    same_beside(lambda s, ws: P.gated_ffn_bwd(dy, x, wg, wu, wd, g, u, ws=ws, stream=s),
                P.Workspace("cuda", 256) if kept else None)


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("sizes", [[1000], [3000001, 17, 5000000], [4001] * 950])
def test_clipping(sizes, kept):
    require_gpu()
    g = torch.Generator().manual_seed(len(sizes))
    grads = [torch.randn(n, generator=g).cuda() for n in sizes]
    out = [torch.empty_like(t) for t in grads]

    def call(s, ws):
        norm = P.clip_grad_norm(P.GradList(grads, out), 1.0, ws=ws, stream=s)
        return [P.grad_norm(grads, ord=math.inf, ws=ws, stream=s), norm] + out

    same_beside(call, P.Workspace("cuda", 256) if kept else None)


def test_rotation():
    require_gpu()
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn((32 * 9 * 16, h, 128), generator=g).to(torch.bfloat16).cuda() for h in (12, 4))
    spec = P.RopeSpec((44, 42, 42))
    same_beside(lambda s, ws: P.rope(q, k, spec, grid=(32, 9, 16), stream=s))


@pytest.mark.parametrize("kept", [False, True])
def test_attention(kept):
    """Zone shapes, pooling, selection and both attention passes."""
    require_gpu()
    g = torch.Generator().manual_seed(2)
    grid = (8, 16, 24)
    geo = P.Geometry(grid, (8, 8, 8), ((4, 4, 4), (1, 8, 8)))
    n = grid[0] * grid[1] * grid[2]
    q, k, v, do = (torch.randn((n, 2, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    feat = torch.randn((n, 128), generator=g).cuda()
    sc = 0.125

    def call(s, ws):
        kw = dict(ws=ws, stream=s)
        zs, margin = P.zone_shapes(geo, feat=feat, **kw)
        qp, kp = P.block_pool(geo, zs, q, k, **kw)
        bias = P.block_audio_bias(geo, zs, feat, 0.5, **kw)
        one = P.block_select(qp, kp, sc, 2, 0.4, **kw)
        sel = P.block_select_ex(qp, kp, sc, 3, 0.3, key_bias=bias, **kw)
        o, lse = P.bsa_fwd(geo, zs, q, k, v, sc, sel["row_ptr"], sel["col_idx"], **kw)
        d = P.bsa_bwd(geo, zs, q, k, v, o, lse, do, sc, sel["row_ptr"], sel["col_idx"], sel["total"], **kw)
        return [zs, margin, qp, kp, bias, flat(one), flat(sel), o, lse, list(d)]

    same_beside(call, P.Workspace("cuda", 256) if kept else None)


def test_memory_stays_with_the_streams_that_use_it():
    """A shared workspace that another stream still works in is not handed on when it grows."""
    require_gpu()
    x, wg, wu, wd, dy = ffn(300, 1160, 392)
    want = P.gated_ffn_fwd(x, wg, wu, wd)
    ws = P.Workspace("cuda", 1 << 22)
    junk = torch.ones(1 << 28, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(100):
            junk.mul_(1.0)
        got = P.gated_ffn_fwd(x, wg, wu, wd, ws=ws)
    held = ws.buf.data_ptr()
    ws.ensure(1 << 24)
    again = [torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert all(not t.data_ptr() <= held < t.data_ptr() + t.numel() for t in again)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_forked_inside_a_capture():
    """A call on a side stream that joins the captured one: with a workspace, and without one."""
    require_gpu()
    x, wg, wu, wd, dy = ffn(300, 1160, 392)
    grads = [torch.ones(n, device="cuda") for n in (1000, 300000)]
    ws = P.Workspace("cuda")
    want = P.gated_ffn_fwd(x, wg, wu, wd, ws=ws)
    wantb = P.gated_ffn_bwd(dy, x, wg, wu, wd, want[1], want[2], ws=ws)
    norm = P.grad_norm(grads)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = P.gated_ffn_fwd(x, wg, wu, wd, stream=side)
        gotb = P.gated_ffn_bwd(dy, x, wg, wu, wd, got[1], got[2], ws=ws, stream=side)
        n = P.grad_norm(grads, stream=side)
        here.wait_stream(side)
        y2 = got[0] + 0
    junk = [torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for _ in range(3):
        for t in (*got, *gotb, n, y2):
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, *gotb, n, y2), (*want, *wantb, norm, want[0])))
    assert all((j == 255).all() for j in junk)
    P.check_device_status(ws)
    P.check_device_status()


def test_two_threads_at_once():
    """Calls from several host threads, each on a stream and with memory of its own."""
    require_gpu()
    import threading
    sizes = [(1, 256, 512), (33, 256, 512), (300, 1160, 392), (900, 520, 264)]
    data = [ffn(*s) for s in sizes]
    spec = P.RopeSpec((44, 42, 42))
    q = torch.randn((360, 4, 128), device="cuda")

    def work(x, wg, wu, wd, dy, s):
        y, g, u = P.gated_ffn_fwd(x, wg, wu, wd, stream=s)
        r = [y, g, u, *P.gated_ffn_bwd(dy, x, wg, wu, wd, g, u, stream=s), P.rope(q, None, spec, grid=(4, 9, 10), stream=s)[0]]
        return r + [P.grad_norm([y, g, u], stream=s)]

    want = [work(*d, None) for d in data]
    torch.cuda.synchronize()
    off = []

    def run(i):
        s = torch.cuda.Stream()
        for _ in range(40):
            got = work(*data[i], s)
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                off.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(data))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not off
    P.check_device_status()
