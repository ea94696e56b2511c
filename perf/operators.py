"""Cases that measure the operators around the block-sparse attention of one layer's training step.

Three operators, forward and backward where they have one:

* ``rope``: rotary positions of Q and K, over the (t, h, w) token grid of the video latents or at given positions,
  before pooling, scoring and attention read them (and the transposed rotation of dQ and dK after the backward);
* ``ffn``: the gated feed-forward block behind the attention, y = (act(x Wg^T) * (x Wu^T)) Wd^T;
* ``clip``: the global L2 norm of the step's gradients and their clipping.

``run`` computes a case in plain torch operations, or with ``own`` set by the framework's own calls. ``exact`` gives
the same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of a streamed generation: K and Q of a grouped-head layout, half of the head rotated,
        # at a far position of an extended context
        {"name": "rope one token", "op": "rope", "bwd": False, "tokens": 1, "t": 0, "h": 0, "w": 0, "far": 1 << 20,
         "hq": 24, "hk": 8, "d": 128, "layout": "half", "a0": 64, "a1": 0, "a2": 0, "theta": 500000.0,
         "scaling": "yarn", "factor": 8.0, "type": "bf16"},
        # a 32-bit layer on a small clipped grid, odd in every axis, part of a 64-wide head
        {"name": "rope odd grid fp32", "op": "rope", "bwd": False, "tokens": 13 * 23 * 37, "t": 13, "h": 23, "w": 37,
         "far": 0, "hq": 12, "hk": 4, "d": 64, "layout": "half", "a0": 16, "a1": 12, "a2": 12, "theta": 10000.0,
         "scaling": "none", "factor": 1.0, "type": "fp32"},
        # the real 720p latent grid, every channel rotated, the axes' shares as a video transformer splits them
        {"name": "rope 720p latent", "op": "rope", "bwd": False, "tokens": 16 * 45 * 80, "t": 16, "h": 45, "w": 80,
         "far": 0, "hq": 24, "hk": 24, "d": 128, "layout": "interleaved", "a0": 44, "a1": 42, "a2": 42,
         "theta": 10000.0, "scaling": "none", "factor": 1.0, "type": "bf16"},
        # the gradients of Q and K of the 2K training step
        {"name": "rope 2k backward", "op": "rope", "bwd": True, "tokens": 32 * 72 * 128, "t": 32, "h": 72, "w": 128,
         "far": 0, "hq": 24, "hk": 24, "d": 128, "layout": "interleaved", "a0": 44, "a1": 42, "a2": 42,
         "theta": 10000.0, "scaling": "none", "factor": 1.0, "type": "bf16"},
        # a single token through the block: the weights' bytes are the cost
        {"name": "ffn one token", "op": "ffn", "bwd": False, "save": False, "m": 1, "d": 2048, "f": 5632, "act": "silu"},
        # a ragged batch of a small layer (widths that are no multiple of any tile), activations saved for training
        {"name": "ffn ragged", "op": "ffn", "bwd": False, "save": True, "m": 1237, "d": 1160, "f": 3112,
         "act": "gelu_tanh"},
        # one chunk of video tokens through a wide layer
        {"name": "ffn wide", "op": "ffn", "bwd": False, "save": True, "m": 16384, "d": 4096, "f": 11264, "act": "silu"},
        # the backward pass of a small layer over an odd number of tokens
        {"name": "ffn ragged backward", "op": "ffn", "bwd": True, "save": True, "m": 1999, "d": 1536, "f": 4104,
         "act": "gelu"},
        # the backward pass of the wide layer
        {"name": "ffn wide backward", "op": "ffn", "bwd": True, "save": True, "m": 8192, "d": 4096, "f": 11264,
         "act": "silu"},
        # the gradients of a small adapter: latency
        {"name": "clip few small", "op": "clip", "tensors": 6, "total": 40001, "mix": "fp32", "sizes": 1, "ratio": 0.7},
        # the gradients of a few layers, hundreds of tensors from single values to matrices, both types
        {"name": "clip many mixed", "op": "clip", "tensors": 411, "total": 60000007, "mix": "both", "sizes": 2,
         "ratio": 0.3},
        # a large model's gradients, larger than any cache
        {"name": "clip large", "op": "clip", "tensors": 64, "total": 600000000, "mix": "bf16", "sizes": 3, "ratio": 0.6},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "ffn", "clip"))
    if op == "rope":
        d = rng.choice((32, 48, 64, 80, 96, 128, 256))
        hq = rng.randint(1, 32)
        hk = rng.choice([h for h in (1, 2, 4, 8, hq) if h <= hq])
        kind = rng.choice(("bf16", "bf16", "fp32"))
        most = 2 * 294912 * 24 * 128 // (2 if kind == "fp32" else 1)
        top = max(2, min(294912, most // ((hq + hk) * d)))
        far = 0
        if rng.random() < 0.5:  # a grid
            t = rng.randint(1, 32)
            h = rng.randint(1, max(1, min(90, top // t)))
            w = rng.randint(1, max(1, min(160, top // (t * h))))
            tokens = t * h * w
            rot = rng.randint(3, d // 2) * 2
            a1 = 2 * rng.randint(1, rot // 6)
            a2 = 2 * rng.randint(1, rot // 6)
            a0 = rot - a1 - a2
        else:  # given positions
            t = h = w = 0
            tokens = _log(rng, 1, top)
            far = _log(rng, 1, 1 << 24)
            a0, a1, a2 = rng.randint(1, d // 2) * 2, 0, 0
        return {"op": op, "bwd": rng.random() < 0.5, "tokens": tokens, "t": t, "h": h, "w": w, "far": far, "hq": hq,
                "hk": hk, "d": d, "layout": rng.choice(("half", "interleaved")), "a0": a0, "a1": a1, "a2": a2,
                "theta": rng.choice((10000.0, 500000.0)), "scaling": rng.choice(("none", "linear", "ntk", "yarn")),
                "factor": rng.choice((2.0, 4.0, 8.0)), "type": kind}
    if op == "ffn":
        bwd = rng.random() < 0.5
        m = _log(rng, 1, 16384)
        d = 8 * _log(rng, 8, 512)
        f = 8 * _log(rng, 16, 1408)
        if bwd:
            m = min(m, 8192)
        return {"op": op, "bwd": bwd, "save": bwd or rng.random() < 0.5, "m": m, "d": d, "f": f,
                "act": rng.choice(("silu", "gelu", "gelu_tanh", "relu"))}
    return {"op": op, "tensors": _log(rng, 1, 600), "total": _log(rng, 1000, 400000000),
            "mix": rng.choice(("bf16", "fp32", "both")), "sizes": rng.randint(1, 10 ** 6),
            "ratio": rng.choice((0.1, 0.6, 2.0))}


# ------------------------------------------------------------------ inputs
def _sizes(case):
    """Sizes of the gradients: log-uniform shares of the total, single values and odd lengths among them."""
    rng = random.Random(case["sizes"])
    share = [math.exp(rng.uniform(0.0, 8.0)) for _ in range(case["tensors"])]
    return [max(1, int(case["total"] * s / sum(share))) for s in share]


def _gradient_types(case):
    rng = random.Random(case["sizes"] + 1)
    one = {"bf16": ("bf16",), "fp32": ("fp32",), "both": ("bf16", "fp32")}[case["mix"]]
    return [TYPES[rng.choice(one)] for _ in range(case["tensors"])]


def _buckets(sizes, kinds):
    """A bucket of zeros for each type, and each tensor's place in them."""
    kept = sorted(set(kinds), key=str)
    padded = [-(-n // 64) * 64 for n in sizes]
    start = [sum(p for p, k in zip(padded[:i], kinds) if k == kinds[i]) for i in range(len(sizes))]
    flat = {k: torch.zeros(sum(p for p, q in zip(padded, kinds) if q == k), dtype=k, device=DEVICE) for k in kept}
    return [flat[k] for k in kept], [flat[k][a:a + n] for a, n, k in zip(start, sizes, kinds)]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))

    def normal(shape, kind, scale=1.0):
        return torch.randn(shape, generator=g, device=DEVICE).mul_(scale).to(kind)

    s = dict(case)
    if case["op"] == "rope":
        kind = TYPES[case["type"]]
        s["q"] = normal((case["tokens"], case["hq"], case["d"]), kind)
        s["k"] = normal((case["tokens"], case["hk"], case["d"]), kind)
        s["axis"] = torch.tensor([a for a, _ in _pairs(case)], device=DEVICE)
        s["freq"] = torch.tensor([f for _, f in _pairs(case)], dtype=torch.float64, device=DEVICE)
        s["positions"] = None
        if not case["t"]:  # the tokens of several sequences: any order, any position up to the context's end
            s["positions"] = torch.randint(0, case["far"], (case["tokens"], 1), generator=g, device=DEVICE,
                                           dtype=torch.int32)
    elif case["op"] == "ffn":
        m, d, f, b = case["m"], case["d"], case["f"], torch.bfloat16
        s["x"] = normal((m, d), b)
        s["wg"] = normal((f, d), b, d ** -0.5)
        s["wu"] = normal((f, d), b, d ** -0.5)
        s["wd"] = normal((d, f), b, f ** -0.5)
        if case["bwd"]:  # the projections that the forward pass saved, and the gradient that comes back
            s["g"] = (s["x"].float() @ s["wg"].float().T).to(b)
            s["u"] = (s["x"].float() @ s["wu"].float().T).to(b)
            s["dy"] = normal((m, d), b, 1e-2)
    else:
        s["grads"] = [normal((n,), kind, 10.0 ** -(i % 4)) for i, (n, kind) in
                      enumerate(zip(_sizes(case), _gradient_types(case)))]
        # the clipped gradients go into one bucket for each type, every tensor on a 128-byte border
        s["buckets"], s["clipped"] = _buckets([x.numel() for x in s["grads"]], [x.dtype for x in s["grads"]])
        # the bound that a training run sets, against the norm that these gradients have about
        norm = math.sqrt(sum(n * 100.0 ** -(i % 4) for i, n in enumerate(_sizes(case))))
        s["max_norm"] = case["ratio"] * norm
    return s


# ------------------------------------------------------------------ plain forms
_TRAINED = 4096.0  # the context length that the unscaled frequencies were trained for


def _ramp(theta, n, j):
    """Share of the stretched frequency in pair j of an axis of n channels: pairs that turn more than 32 times over
    the trained length keep theirs, those below one turn are stretched, a ramp over the pair's index between."""
    at = lambda turns: n * math.log(_TRAINED / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), n - 1)
    return min(max((j - low) / max(high - low, 0.001), 0.0), 1.0)


def _frequency(case, n, j):
    """Angle per position of pair j of an axis of n channels."""
    kind, factor = case["scaling"], case["factor"]
    theta = case["theta"] * (factor ** (n / (n - 2)) if kind == "ntk" and n > 2 else 1.0)
    f = theta ** (-2.0 * j / n)
    share = {"linear": 1.0, "yarn": _ramp(theta, n, j) if kind == "yarn" else 0.0}.get(kind, 0.0)
    return f / factor * share + f * (1.0 - share)


def _pairs(case):
    """(axis, frequency) of every pair: those of axis 0, then axis 1, then axis 2."""
    return [(a, _frequency(case, n, j)) for a, n in enumerate((case["a0"], case["a1"], case["a2"]))
            for j in range(n // 2)]


def _stretch(case):
    """The factor on rotated channels that goes with the stretched frequencies."""
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0


def _angles(s):
    """Angle of every token and pair in 64 bits."""
    positions = s["positions"]
    if positions is None:
        n = torch.arange(s["tokens"], device=DEVICE)
        hw = s["h"] * s["w"]
        positions = torch.stack([n // hw, n % hw // s["w"], n % s["w"]], 1)
    return positions.expand(-1, 3)[:, s["axis"]].double() * s["freq"]


def _rotate(case, x, cos, sin):
    """Rotated pairs in 32 bits, rounded once; the channels behind the rotated ones as they were."""
    rot = case["a0"] + case["a1"] + case["a2"]
    y = x.clone()
    if case["layout"] == "half":
        one, two = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        one, two = slice(0, rot, 2), slice(1, rot, 2)
    a, b = x[..., one].float(), x[..., two].float()
    y[..., one] = (a * cos - b * sin).to(x.dtype)
    y[..., two] = (b * cos + a * sin).to(x.dtype)
    return y


def _activation(act, g):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    return g.clamp(min=0), (g > 0).to(g.dtype)


def _ffn(s):
    g, u = s["x"].float() @ s["wg"].float().T, s["x"].float() @ s["wu"].float().T
    y = ((_activation(s["act"], g)[0] * u) @ s["wd"].float().T).to(s["x"].dtype)
    return (y, g.to(y.dtype), u.to(y.dtype)) if s["save"] else (y,)


def _ffn_backward(s):
    b = s["x"].dtype
    x, g, u, dy = s["x"].float(), s["g"].float(), s["u"].float(), s["dy"].float()
    a, slope = _activation(s["act"], g)
    dh = dy @ s["wd"].float()
    dg, du = dh * u * slope, dh * a
    dx = dg @ s["wg"].float() + du @ s["wu"].float()
    return dx.to(b), (dg.T @ x).to(b), (du.T @ x).to(b), (dy.T @ (a * u)).to(b)


def _clip(s):
    norm = torch.stack([x.double().square().sum() for x in s["grads"]]).sum().sqrt()
    factor = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    _ = [y.copy_(x.float() * factor) for x, y in zip(s["grads"], s["clipped"])]
    return norm.float(), s["buckets"]


# ------------------------------------------------------------------ one pass
def _spec(s):
    """The framework's description of the rotation, made once by a program that keeps it."""
    import dynamic_block_sparse_shape_b200 as P
    dims = (s["a0"], s["a1"], s["a2"]) if s["t"] else (s["a0"],)
    return P.RopeSpec(dims, layout=s["layout"], theta=s["theta"], scaling=s["scaling"], factor=s["factor"],
                      trained_len=_TRAINED)


def _run_own(s):
    import dynamic_block_sparse_shape_b200 as P
    if s["op"] == "rope":
        if "spec" not in s:
            s["spec"] = _spec(s)
        call = P.rope_bwd if s["bwd"] else P.rope
        grid = (s["t"], s["h"], s["w"]) if s["t"] else None
        return call(s["q"], s["k"], s["spec"], grid=grid, positions=s["positions"])
    if "ws" not in s:
        s["ws"] = P.Workspace(DEVICE)
    if s["op"] == "clip":
        if "list" not in s:  # gradients that stay in place from step to step: laid out once
            s["list"] = P.GradList(s["grads"], out=s["clipped"])
        norm = P.clip_grad_norm(s["list"], s["max_norm"], ws=s["ws"])
        return norm, s["buckets"]
    if s["bwd"]:
        return P.gated_ffn_bwd(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], s["g"], s["u"], act=s["act"], ws=s["ws"])
    y, g, u = P.gated_ffn_fwd(s["x"], s["wg"], s["wu"], s["wd"], act=s["act"], save=s["save"], ws=s["ws"])
    return (y, g, u) if s["save"] else (y,)


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "rope":
        turn = _angles(state)
        m = _stretch(state)
        cos, sin = (torch.cos(turn) * m).float()[:, None], (torch.sin(turn) * m).float()[:, None]
        if state["bwd"]:
            sin = -sin
        return _rotate(state, state["q"], cos, sin), _rotate(state, state["k"], cos, sin)
    if state["op"] == "clip":
        return _clip(state)
    return _ffn_backward(state) if state["bwd"] else _ffn(state)


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * (case["hq"] + case["hk"])
        rot = case["a0"] + case["a1"] + case["a2"]
        size = 2 if case["type"] == "bf16" else 4
        return {"bytes": 2 * n * case["d"] * size + (0 if case["t"] else 4 * case["tokens"]), "flops": 3 * n * rot}
    if case["op"] == "ffn":
        m, d, f = case["m"], case["d"], case["f"]
        if case["bwd"]:  # dy, x, g, u and the weights in; dx and the weights' gradients out; dh, dx and dW products
            return {"bytes": 2 * (3 * m * d + 2 * m * f + 6 * d * f), "flops": 12 * m * d * f}
        return {"bytes": 2 * (2 * m * d + 3 * d * f + (2 * m * f if case["save"] else 0)), "flops": 6 * m * d * f}
    moved = sum(n * k.itemsize for n, k in zip(_sizes(case), _gradient_types(case)))
    return {"bytes": 2 * moved, "flops": 3 * sum(_sizes(case))}


# ------------------------------------------------------------------ 64 bits
def _exact_frequencies(case, n):
    """The frequencies of one axis of n channels, as a tensor over its pairs."""
    j = torch.arange(n // 2, dtype=torch.float64, device=DEVICE)
    theta = math.log(case["theta"])
    if case["scaling"] == "ntk" and n > 2:
        theta += math.log(case["factor"]) * n / (n - 2)
    f = torch.exp(-2 * j / max(n, 1) * theta)
    if case["scaling"] == "linear":
        return f / case["factor"]
    if case["scaling"] == "yarn":
        border = [n / (2 * theta) * math.log(_TRAINED / (2 * math.pi * turns)) for turns in (32, 1)]
        low, high = max(math.floor(border[0]), 0), min(math.ceil(border[1]), n - 1)
        stretched = ((j - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (1 - stretched + stretched / case["factor"])
    return f


def _exact_rope(case, s):
    dims = (case["a0"], case["a1"], case["a2"])
    rot = sum(dims)
    if s["positions"] is None:
        ax = [torch.arange(case[c], dtype=torch.float64, device=DEVICE) for c in ("t", "h", "w")]
        place = torch.cartesian_prod(*ax)
    else:
        place = s["positions"].double().expand(-1, 3)
    turn = torch.cat([place[:, a, None] * _exact_frequencies(case, n) for a, n in enumerate(dims)], 1)
    stretch = 1.0 + math.log(case["factor"]) / 10 if case["scaling"] == "yarn" else 1.0
    w = torch.polar(torch.full_like(turn, stretch), -turn if case["bwd"] else turn)[:, None]

    def one(x):
        x = x.double()
        if case["layout"] == "half":
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * w
            return torch.cat([z.real, z.imag, x[..., rot:]], -1)
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * w
        return torch.cat([torch.view_as_real(z).flatten(-2), x[..., rot:]], -1)

    return one(s["q"]), one(s["k"])


def _exact_slope(act, g):
    """act'(g) by differentiating the activation's definition."""
    g = g.detach().requires_grad_()
    with torch.enable_grad():
        y = _exact_act(act, g)
        return torch.autograd.grad(y.sum(), g)[0]


def _exact_act(act, g):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return torch.nn.functional.gelu(g)
    if act == "gelu_tanh":
        return torch.nn.functional.gelu(g, approximate="tanh")
    return torch.relu(g)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "clip":
        total = math.sqrt(math.fsum(float(torch.dot(v, v)) for v in (x.double() for x in s["grads"])))
        factor = min(1.0, s["max_norm"] / (total + 1e-6))
        wide, place = _buckets([x.numel() for x in s["grads"]], [x.dtype for x in s["grads"]])
        wide = [b.double() for b in wide]
        at = {b.dtype: [p.storage_offset() for p in place if p.dtype == b.dtype] for b in s["buckets"]}
        for b, kind in zip(wide, (b.dtype for b in s["buckets"])):
            for a, x in zip(at[kind], [x for x in s["grads"] if x.dtype == kind]):
                b[a:a + x.numel()] = x.double() * factor
        return torch.tensor(total, dtype=torch.float64), wide
    D = {k: s[k].double() for k in ("x", "wg", "wu", "wd")}
    if not case["bwd"]:
        g, u = torch.einsum("md,fd->mf", D["x"], D["wg"]), torch.einsum("md,fd->mf", D["x"], D["wu"])
        y = torch.einsum("mf,df->md", _exact_act(case["act"], g) * u, D["wd"])
        return (y, g, u) if case["save"] else (y,)
    g, u, dy = s["g"].double(), s["u"].double(), s["dy"].double()
    dh = torch.einsum("md,df->mf", dy, D["wd"])
    dg, du = dh * u * _exact_slope(case["act"], g), dh * _exact_act(case["act"], g)
    h = _exact_act(case["act"], g) * u
    return (torch.einsum("mf,fd->md", dg, D["wg"]) + torch.einsum("mf,fd->md", du, D["wu"]),
            torch.einsum("mf,md->fd", dg, D["x"]), torch.einsum("mf,md->fd", du, D["x"]),
            torch.einsum("md,mf->df", dy, h))
