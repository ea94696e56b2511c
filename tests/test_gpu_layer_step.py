"""The operators around the attention together with it, as one training step of a layer uses them: rotation of Q and
K, zone shapes, pooling, selection, attention, feed-forward, their backward passes, and the clipping of the gradients.

The attention is held to the stated tolerance of its own tests (max-abs 2e-2, mean-abs 2e-3 at unit scale); the rotation
before and after it is exact to bf16 rounding. Each stage's reference starts from the values that the stage was given.
"""
import math

import numpy as np
import pytest
import torch

import dynamic_block_sparse_shape_b200 as P
from oracle import layer_oracle as L
from oracle import prism_oracle as O
from tests.gpu_util import assert_close, f64, mask_bits_to_bool, require_gpu

GRID, ZONE, HEADS, D = (4, 8, 16), (4, 8, 8), 2, 64


def _step(x, weights, spec, geo, ws, stream=None):
    """One layer's step on the GPU: outputs and gradients by name."""
    n = x["q"].shape[0]
    sc = 1.0 / math.sqrt(D)
    q, k = P.rope(x["q"], x["k"], spec, grid=GRID, stream=stream)
    zs, _ = P.zone_shapes(geo, ws=ws, stream=stream)
    qp, kp = P.block_pool(geo, zs, q, k, ws=ws, stream=stream)
    sel = P.block_select(qp, kp, sc, 2, 0.5, ws=ws, stream=stream)
    o_lo = torch.empty_like(q)
    o, lse = P.bsa_fwd(geo, zs, q, k, x["v"], sc, sel["row_ptr"], sel["col_idx"], ws=ws, o_lo=o_lo, stream=stream)
    h = o.reshape(n, HEADS * D)
    y, gate, up = P.gated_ffn_fwd(h, *weights, act="gelu_tanh", ws=ws, stream=stream)
    dh, dwg, dwu, dwd = P.gated_ffn_bwd(x["dy"], h, *weights, gate, up, act="gelu_tanh", ws=ws, stream=stream)
    do = dh.view(n, HEADS, D)
    dqr, dkr, dv = P.bsa_bwd(geo, zs, q, k, x["v"], o, lse, do, sc, sel["row_ptr"], sel["col_idx"], sel["total"], ws=ws,
                             o_lo=o_lo, stream=stream)
    dq, dk = P.rope_bwd(dqr, dkr, spec, grid=GRID, stream=stream)
    r = dict(q=q, k=k, zs=zs, sel=sel, o=o, lse=lse, y=y, gate=gate, up=up, do=do, dqr=dqr, dkr=dkr)
    grads = dict(dq=dq, dk=dk, dv=dv, dwg=dwg, dwu=dwu, dwd=dwd)
    r["before"] = {name: t.clone() for name, t in grads.items()}
    r["norm"] = P.clip_grad_norm(list(grads.values()), 0.5, ws=ws, stream=stream)
    r["grads"] = grads
    return r


def _inputs():
    g = torch.Generator().manual_seed(3)
    n = GRID[0] * GRID[1] * GRID[2]
    b = lambda *s, k=1.0: (torch.randn(s, generator=g) * k).to(torch.bfloat16).cuda()  # noqa: E731
    x = {name: b(n, HEADS, D) for name in ("q", "k", "v")}
    x["dy"] = b(n, HEADS * D)
    c, f = HEADS * D, 208
    return x, (b(f, c, k=c ** -0.5), b(f, c, k=c ** -0.5), b(c, f, k=f ** -0.5))


@pytest.mark.gpu
def test_step_against_fp64():
    require_gpu()
    x, weights = _inputs()
    spec = P.RopeSpec((22, 20, 22), layout="half")
    geo = P.Geometry(GRID, ZONE, ((4, 4, 4),))
    ws = P.Workspace("cuda")
    r = _step(x, weights, spec, geo, ws)
    torch.cuda.synchronize()
    P.check_device_status(ws)
    ang = L.rope_angles((22, 20, 22), grid=GRID)
    for name in ("q", "k"):
        want = L.rope(f64(x[name]), ang, "half")
        assert (np.abs(f64(r[name]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * (1 + 2.0 ** -8) * np.abs(f64(x[name])).max()).all()
    # the selection from the rotated rows, the attention over it
    idx, _, _ = O.zone_shapes(GRID, ZONE, geo.cand)
    blocks = O.block_tokens(GRID, ZONE, geo.cand, idx)
    Q, K, V = f64(r["q"]), f64(r["k"]), f64(x["v"])
    sc = 1.0 / math.sqrt(D)
    mask = mask_bits_to_bool(r["sel"]["mask"], blocks.shape[0])
    ref = O.block_select(O.block_pool(Q, blocks), O.block_pool(K, blocks), sc, 2, 0.5)
    assert (mask.sum(-1) >= 2).all() and (mask == ref["mask"]).mean() > 0.99  # a boundary block may change places
    allowed = O.token_mask(mask, blocks, Q.shape[0])
    o, lse = O.masked_attention_fwd(Q, K, V, allowed, sc)
    assert_close("O", f64(r["o"]), o)
    # the feed-forward block on what the attention gave it
    h = f64(r["o"]).reshape(Q.shape[0], -1)
    W = [f64(w) for w in weights]
    y, g, u = L.gated_ffn_fwd(h, *W, "gelu_tanh")
    assert_close("y", f64(r["y"]), y)
    dh, dwg, dwu, dwd = L.gated_ffn_bwd(f64(x["dy"]), h, *W, f64(r["gate"]), f64(r["up"]), "gelu_tanh")
    do = f64(r["do"])
    assert_close("dO", do.reshape(dh.shape), dh, atol_max=4e-2, atol_mean=4e-3)  # of rms 2: the stated bound scaled
    b = {k: f64(v) for k, v in r["before"].items()}
    for name, want in (("dwg", dwg), ("dwu", dwu), ("dwd", dwd)):
        rel = np.linalg.norm(b[name] - want) / np.linalg.norm(want)
        assert rel <= 2 * 2.0 ** -8, (name, rel)  # two roundings of half a bf16 step each
    dq, dk, dv = O.masked_attention_bwd(Q, K, V, f64(r["o"]), f64(r["lse"]), do, allowed, sc)
    for name, want in (("dqr", dq), ("dkr", dk)):
        assert_close(name, f64(r[name]), want, atol_max=4e-2, atol_mean=4e-3)
    assert_close("dv", b["dv"], dv, atol_max=4e-2, atol_mean=4e-3)
    for name, src in (("dq", "dqr"), ("dk", "dkr")):
        want = L.rope(f64(r[src]), ang, "half", transposed=True)
        assert (np.abs(b[name] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * (1 + 2.0 ** -8) * np.abs(f64(r[src])).max()).all()
    # the clipping of all six
    norm = L.grad_norm(list(b.values()))
    assert abs(float(r["norm"]) - norm) <= 2.0 ** -20 * norm
    for name, t in r["grads"].items():
        want = b[name] * L.clip_factor(norm, 0.5)
        assert (np.abs(f64(t) - want) <= 2.0 ** -8 * np.abs(want) + 1e-30).all(), name


@pytest.mark.gpu
def test_step_is_the_same_every_time():
    """The same bits again, on another stream and with a shared workspace that other sizes used in between."""
    require_gpu()
    x, weights = _inputs()
    spec = P.RopeSpec((22, 20, 22), layout="half")
    geo = P.Geometry(GRID, ZONE, ((4, 4, 4),))
    ws = P.Workspace("cuda")
    first = _step(x, weights, spec, geo, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = _step(x, weights, spec, geo, ws)
    side.synchronize()
    assert torch.equal(first["y"], again["y"]) and torch.equal(first["norm"], again["norm"])
    for name in first["grads"]:
        assert torch.equal(first["grads"][name], again["grads"][name]), name


@pytest.mark.gpu
def test_sharded_clipping():
    """Two head shards: the norm from the shards' norms, then each shard scaled, equals clipping the whole."""
    require_gpu()
    from dynamic_block_sparse_shape_b200.shard import head_shard
    g = torch.Generator().manual_seed(9)
    whole = torch.randn((500, 5, 64), generator=g).to(torch.bfloat16).cuda()
    parts = [whole[:, slice(*head_shard(5, 2, r))].contiguous() for r in range(2)]
    norm = P.grad_norm([whole])
    both = torch.stack([P.grad_norm([p]) for p in parts]).square().sum().sqrt()
    # each rank's fp32 norm is off by 16 * 2^-24 at most, squares, sum and root by three roundings more
    assert abs(float(both) - float(norm)) <= 40 * 2.0 ** -24 * float(norm)
    for p in parts:
        P.scale_grads([p], both, 1.0)
    P.clip_grad_norm([whole], 1.0)
    for r, p in enumerate(parts):
        want = whole[:, slice(*head_shard(5, 2, r))]
        # factors 40 * 2^-24 apart round to neighbouring bf16 values at most
        assert ((p.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs()).all()


@pytest.mark.gpu
def test_step_after_other_sizes():
    """The same bits again after other sizes, smaller and larger, used the shared workspace in between and let it grow."""
    require_gpu()
    x, weights = _inputs()
    spec = P.RopeSpec((22, 20, 22), layout="half")
    geo = P.Geometry(GRID, ZONE, ((4, 4, 4),))
    ws = P.Workspace("cuda", 256)
    first = _step(x, weights, spec, geo, ws)
    b = lambda *s: torch.full(s, 0.5, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for m, c, f in ((3, 64, 128), (3000, 264, 1032), (40, 2312, 72)):
        y, gate, up = P.gated_ffn_fwd(b(m, c), b(f, c), b(f, c), b(c, f), ws=ws)
        P.gated_ffn_bwd(y, b(m, c), b(f, c), b(f, c), b(c, f), gate, up, ws=ws)
    P.clip_grad_norm([b(n) for n in range(1, 2000)], 1.0, ws=ws)
    again = _step(x, weights, spec, geo, ws)
    P.check_device_status(ws)
    assert torch.equal(first["y"], again["y"]) and torch.equal(first["norm"], again["norm"])
    for name in first["grads"]:
        assert torch.equal(first["grads"][name], again["grads"][name]), name


@pytest.mark.gpu
def test_step_as_replayed_graphs():
    """What lies before and behind the selection (which hands its total to the host) as two captured graphs that share a
    workspace: replayed with other inputs they give an eager step's bits."""
    require_gpu()
    x, weights = _inputs()
    spec = P.RopeSpec((22, 20, 22), layout="half")
    geo = P.Geometry(GRID, ZONE, ((4, 4, 4),))
    ws, sc, n = P.Workspace("cuda"), 1.0 / math.sqrt(D), x["q"].shape[0]
    first = _step(x, weights, spec, geo, ws)  # grows the workspace, loads the kernels
    sel = first["sel"]
    torch.cuda.synchronize()
    before, behind = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(before):
        q, k = P.rope(x["q"], x["k"], spec, grid=GRID)
        zs, _ = P.zone_shapes(geo, ws=ws)
        qp, kp = P.block_pool(geo, zs, q, k, ws=ws)
    with torch.cuda.graph(behind):
        o_lo = torch.empty_like(q)
        o, lse = P.bsa_fwd(geo, zs, q, k, x["v"], sc, sel["row_ptr"], sel["col_idx"], ws=ws, o_lo=o_lo)
        h = o.reshape(n, HEADS * D)
        y, gate, up = P.gated_ffn_fwd(h, *weights, act="gelu_tanh", ws=ws)
        dh, dwg, dwu, dwd = P.gated_ffn_bwd(x["dy"], h, *weights, gate, up, act="gelu_tanh", ws=ws)
        dqr, dkr, dv = P.bsa_bwd(geo, zs, q, k, x["v"], o, lse, dh.view(n, HEADS, D), sc, sel["row_ptr"], sel["col_idx"],
                                 sel["total"], ws=ws, o_lo=o_lo)
        dq, dk = P.rope_bwd(dqr, dkr, spec, grid=GRID)
        grads = dict(dq=dq, dk=dk, dv=dv, dwg=dwg, dwu=dwu, dwd=dwd)
        norm = P.clip_grad_norm(list(grads.values()), 0.5, ws=ws)
    for scale in (1.0, -0.5):  # q and k, and so the selection, stay
        x["v"].mul_(scale)
        x["dy"].mul_(scale)
        want = _step(x, weights, spec, geo, P.Workspace("cuda"))
        before.replay()
        again = P.block_select(qp, kp, sc, 2, 0.5, ws=ws)
        assert torch.equal(again["col_idx"], sel["col_idx"]) and torch.equal(again["row_ptr"], sel["row_ptr"])
        behind.replay()
        torch.cuda.synchronize()
        P.check_device_status(ws)
        assert torch.equal(y, want["y"]) and torch.equal(norm, want["norm"])
        for name in grads:
            assert torch.equal(grads[name], want["grads"][name]), (name, scale)
