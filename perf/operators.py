"""Performance cases of the feed-forward operators.

Three operators that make up the feed-forward half of a transformer layer, in
both directions, and the clipping of its gradients:

  linear     Z = X W^T + b;  Y = act(Z) + R
  glu        G = X Wg^T + bg;  U = X Wu^T + bu;  H = act(G) * U
  grad_clip  norm = sqrt(sum g^2) over many tensors;  out = g * min(1, max_norm / (norm + 1e-6))

`listed()` holds fixed cases, `draw()` gives more of the same ranges,
`prepare()` makes the inputs on the GPU, `run()` makes one pass in the
operators' plain form (or, where `own` is true, through the library), and
`exact()` gives the outputs in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6  # added to the norm before the division


def listed():
    return [
        # one token through a square projection with bias and residual (the projection that closes a layer while serving)
        case_linear("token", "fwd", 1, 4096, 4096, "bf16", "none", bias=True, residual=True),
        # a few tokens at once through the widening projection: a small serving batch
        case_linear("batch", "fwd", 24, 8192, 2048, "f16", "gelu", bias=True),
        # a long prompt, or a training batch, through the widening projection; Z kept for the backward pass
        case_linear("prompt", "fwd", 8192, 16384, 4096, "bf16", "gelu_tanh", bias=True, save=True),
        # scores over an odd number of symbols, in fp32
        case_linear("scores", "fwd", 1000, 32003, 1024, "f16", "none", y="f32"),
        # a training step's backward pass through the projection
        case_linear("train", "bwd", 4096, 8192, 4096, "bf16", "gelu", bias=True),
        # the same with sizes that fit no tile, rows of odd length
        case_linear("ragged", "bwd", 777, 1001, 1128, "f16", "silu", bias=True),
        # one token through the gated block's two projections
        case_glu("token", "fwd", 1, 10944, 4096, "bf16", "silu"),
        # a ragged handful of tokens, as speculative decoding or a small batch gives
        case_glu("ragged", "fwd", 131, 5000, 2056, "f16", "gelu_tanh", bias=True),
        # a training batch forward, both projections kept
        case_glu("prompt", "fwd", 4096, 10944, 4096, "bf16", "silu", save=True),
        # and its backward pass
        case_glu("train", "bwd", 4096, 10944, 4096, "bf16", "silu"),
        # the gradients of a small model: many short vectors among its matrices
        case_clip("small", 40, 4096, 1 << 18, "mixed", 0.3),
        # the gradients of several wide layers
        case_clip("large", 36, 4096, 1 << 24, "bf16", 0.3),
    ]


def case_linear(name, way, m, n, k, kind, act, bias=False, residual=False, save=False, y=None):
    return {"name": "linear_%s_%s" % (way, name), "op": "linear", "way": way, "m": m, "n": n, "k": k, "type": kind, "act": act,
            "bias": bias, "residual": residual, "save": save, "y": y or kind}


def case_glu(name, way, m, f, k, kind, act, bias=False, save=False):
    return {"name": "glu_%s_%s" % (way, name), "op": "glu", "way": way, "m": m, "n": f, "k": k, "type": kind, "act": act,
            "bias": bias, "save": save}


def case_clip(name, tensors, shortest, longest, kind, share):
    return {"name": "clip_%s" % name, "op": "clip", "tensors": tensors, "shortest": shortest, "longest": longest, "type": kind, "share": share}


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A row length: most are multiples of 64 or 8, some are odd."""
    v = _spread(rng, low, high)
    step = rng.choice((64, 64, 8, 1))
    return max(low, v // step * step)


def draw(rng):
    op = rng.choice(("linear", "linear", "glu", "glu", "clip"))
    if op == "clip":
        tensors = _spread(rng, 2, 60)
        longest = min(_spread(rng, 1 << 12, 1 << 24), (36 << 22) // tensors)
        return {"op": "clip", "tensors": tensors, "shortest": min(longest, _spread(rng, 1, 1 << 13)), "longest": longest,
                "type": rng.choice(("f16", "bf16", "f32", "mixed")), "share": rng.choice((0.1, 0.3, 2.0))}
    way = rng.choice(("fwd", "fwd", "bwd"))
    m, n, k = _spread(rng, 1, 8192), _width(rng, 256, 16384), _width(rng, 256, 8192)
    most = 3.0e11 if way == "fwd" else 1.5e11
    while m * n * k * (2 if op == "glu" else 1) > most:
        m = max(1, m // 2)
    kind = rng.choice(("f16", "bf16"))
    if op == "glu":
        return {"op": "glu", "way": way, "m": m, "n": n, "k": k, "type": kind, "act": rng.choice(("silu", "gelu", "gelu_tanh", "relu", "sigmoid")),
                "bias": rng.random() < 0.5, "save": way == "fwd" and rng.random() < 0.5}
    act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
    fwd = way == "fwd"
    return {"op": "linear", "way": way, "m": m, "n": n, "k": k, "type": kind, "act": act, "bias": rng.random() < 0.5,
            "residual": fwd and rng.random() < 0.5, "save": fwd and rng.random() < 0.3,
            "y": "f32" if fwd and rng.random() < 0.2 else kind}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _inputs(case, seed):
    """The tensors that a pass reads, from the seed alone."""
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed) * 1000003 + 17)

    def normal(*shape, std=1.0, kind):
        return (torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32) * std).to(TYPES[kind])

    if case["op"] == "clip":
        return {"grads": [normal(c, std=10.0 ** -(1 + i % 3), kind=t) for i, (c, t) in enumerate(_clip_sizes(case))]}
    m, n, k, kind = case["m"], case["n"], case["k"], case["type"]
    # activations of unit size (they follow a norm), weights that keep it
    v = {"X": normal(m, k, kind=kind)}
    if case["op"] == "linear":
        v["W"] = normal(n, k, std=k ** -0.5, kind=kind)
        if case["way"] == "fwd":
            if case["bias"]:
                v["b"] = normal(n, std=0.1, kind="f32")
            if case["residual"]:
                v["R"] = normal(m, n, kind=case["y"])
        else:
            v["dY"] = normal(m, n, std=1e-2, kind=kind)
            if case["act"] != "none":
                v["Z"] = normal(m, n, kind=kind)
    else:
        v["Wg"] = normal(n, k, std=k ** -0.5, kind=kind)
        v["Wu"] = normal(n, k, std=k ** -0.5, kind=kind)
        if case["way"] == "fwd":
            if case["bias"]:
                v["bg"] = normal(n, std=0.1, kind="f32")
                v["bu"] = normal(n, std=0.1, kind="f32")
        else:
            v["dH"] = normal(m, n, std=1e-2, kind=kind)
            v["G"] = normal(m, n, kind=kind)
            v["U"] = normal(m, n, kind=kind)
    return v


def _clip_sizes(case):
    """(count, type) of each gradient: lengths spread from the shortest to the longest, one of each four a whole longest."""
    n, low, high = case["tensors"], case["shortest"], case["longest"]
    sizes = []
    for i in range(n):
        c = high if i % 4 == 0 else int(round(low * (high / low) ** (i / max(1, n - 1))))
        kind = ("bf16", "f32", "f16")[i % 3] if case["type"] == "mixed" else case["type"]
        sizes.append((max(1, c), kind))
    return sizes


def _expected_norm(case):
    """The norm that gradients of these sizes and deviations have, near enough to set a limit by."""
    return math.sqrt(sum(c * 10.0 ** (-2 * (1 + i % 3)) for i, (c, _) in enumerate(_clip_sizes(case))))


def prepare(case, seed):
    v = _inputs(case, seed)
    new = lambda *shape, kind: torch.empty(*shape, dtype=TYPES[kind], device=DEVICE)  # noqa: E731
    out = {}
    if case["op"] == "clip":
        out["grads"] = [torch.empty_like(g) for g in v["grads"]]
        out["norm"] = new(1, kind="f32")
    else:
        m, n, k, kind = case["m"], case["n"], case["k"], case["type"]
        if case["op"] == "linear" and case["way"] == "fwd":
            out["Y"] = new(m, n, kind=case["y"])
            if case["save"]:
                out["Z"] = new(m, n, kind=kind)
        elif case["op"] == "linear":
            out["dX"], out["dW"] = new(m, k, kind=kind), new(n, k, kind=kind)
            if case["bias"]:
                out["db"] = new(n, kind="f32")
        elif case["way"] == "fwd":
            out["H"] = new(m, n, kind=kind)
            if case["save"]:
                out["G"], out["U"] = new(m, n, kind=kind), new(m, n, kind=kind)
        else:
            out["dX"], out["dWg"], out["dWu"] = new(m, k, kind=kind), new(n, k, kind=kind), new(n, k, kind=kind)
            if case["bias"]:
                out["dbg"], out["dbu"] = new(n, kind="f32"), new(n, kind="f32")
    state = {"case": case, "in": v, "out": out}
    if own:  # scratch memory that a program allocates once, of the size that the library asks for
        size = _call(case, v, out, None)
        state["workspace"] = torch.zeros(max(size, 16), dtype=torch.uint8, device=DEVICE)
    return state


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(state):
    case, v, out = state["case"], state["in"], state["out"]
    if own:
        _call(case, v, out, state["workspace"])
        return out
    if case["op"] == "clip":
        return _plain_clip(case, v)
    if case["op"] == "linear":
        return _plain_linear(case, v) if case["way"] == "fwd" else _plain_linear_back(case, v)
    return _plain_glu(case, v) if case["way"] == "fwd" else _plain_glu_back(case, v)


def _call(case, v, out, workspace):
    """The library's call for a case; without a workspace, the bytes of workspace that it needs."""
    import implicit_gemm_convolution_amd as igc

    size = workspace is None
    more = {} if size else {"workspace": workspace}
    if case["op"] == "clip":
        f = igc.grad_clip_workspace_size if size else igc.grad_clip
        return f(v["grads"], case["share"] * _expected_norm(case), out["norm"], out=out["grads"], **more)
    m, n, k = case["m"], case["n"], case["k"]
    kind = {"f16": igc.IGC_F16, "bf16": igc.IGC_BF16, "f32": igc.IGC_F32}
    act = {"none": igc.IGC_ACT_NONE, "relu": igc.IGC_ACT_RELU, "gelu": igc.IGC_ACT_GELU, "gelu_tanh": igc.IGC_ACT_GELU_TANH,
           "silu": igc.IGC_ACT_SILU, "sigmoid": igc.IGC_ACT_SIGMOID}[case["act"]]
    more.update(type=kind[case["type"]], act=act)
    if case["op"] == "linear" and case["way"] == "fwd":
        f = igc.linear_forward_workspace_size if size else igc.linear_forward
        return f(m, n, k, v["X"], k, v["W"], k, out["Y"], n, y_type=kind[case["y"]], bias=v.get("b"),
                 R=v.get("R"), ldr=n, Z=out.get("Z"), ldz=n, **more)
    if case["op"] == "linear":
        f = igc.linear_backward_workspace_size if size else igc.linear_backward
        return f(m, n, k, v["dY"], n, Z=v.get("Z"), ldz=n, X=v["X"], ldx=k, W=v["W"], ldw=k,
                 dX=out["dX"], lddx=k, dW=out["dW"], lddw=k, dbias=out.get("db"), **more)
    if case["way"] == "fwd":
        f = igc.glu_forward_workspace_size if size else igc.glu_forward
        return f(m, n, k, v["X"], k, v["Wg"], k, v["Wu"], k, out["H"], n, bias_g=v.get("bg"), bias_u=v.get("bu"),
                 G=out.get("G"), ldg=n, U=out.get("U"), ldu=n, **more)
    f = igc.glu_backward_workspace_size if size else igc.glu_backward
    return f(m, n, k, v["dH"], n, v["G"], n, v["U"], n, X=v["X"], ldx=k, Wg=v["Wg"], ldwg=k, Wu=v["Wu"], ldwu=k,
             dX=out["dX"], lddx=k, dWg=out["dWg"], lddwg=k, dWu=out["dWu"], lddwu=k, dbias_g=out.get("dbg"), dbias_u=out.get("dbu"), **more)


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    s = 1 / (1 + torch.exp(-z))
    return z * s if name == "silu" else s


def _slope(name, z):
    """The activation's derivative."""
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s)) if name == "silu" else s * (1 - s)


def _plain_linear(case, v):
    z = torch.matmul(v["X"].float(), v["W"].float().t())
    if case["bias"]:
        z = z + v["b"]
    y = _act(case["act"], z)
    if case["residual"]:
        y = y + v["R"].float()
    out = {"Y": y.to(TYPES[case["y"]])}
    if case["save"]:
        out["Z"] = z.to(TYPES[case["type"]])
    return out


def _plain_linear_back(case, v):
    t = TYPES[case["type"]]
    g = v["dY"].float()
    if case["act"] != "none":
        g = g * _slope(case["act"], v["Z"].float())
    out = {"dX": torch.matmul(g, v["W"].float()).to(t), "dW": torch.matmul(g.t(), v["X"].float()).to(t)}
    if case["bias"]:
        out["db"] = g.sum(0)
    return out


def _plain_glu(case, v):
    t, x = TYPES[case["type"]], v["X"].float()
    g, u = torch.matmul(x, v["Wg"].float().t()), torch.matmul(x, v["Wu"].float().t())
    if case["bias"]:
        g, u = g + v["bg"], u + v["bu"]
    out = {"H": (_act(case["act"], g) * u).to(t)}
    if case["save"]:
        out["G"], out["U"] = g.to(t), u.to(t)
    return out


def _plain_glu_back(case, v):
    t, x, dh, g, u = TYPES[case["type"]], v["X"].float(), v["dH"].float(), v["G"].float(), v["U"].float()
    du = dh * _act(case["act"], g)
    dg = dh * u * _slope(case["act"], g)
    out = {"dX": (torch.matmul(dg, v["Wg"].float()) + torch.matmul(du, v["Wu"].float())).to(t),
           "dWg": torch.matmul(dg.t(), x).to(t), "dWu": torch.matmul(du.t(), x).to(t)}
    if case["bias"]:
        out["dbg"], out["dbu"] = dg.sum(0), du.sum(0)
    return out


def _plain_clip(case, v):
    # squares are summed in 64 bits: the sum runs over up to 10^8 values
    norm = torch.stack([g.double().square().sum() for g in v["grads"]]).sum().sqrt()
    scale = torch.clamp(case["share"] * _expected_norm(case) / (norm + EPS), max=1.0).float()
    return {"grads": [(g.float() * scale).to(g.dtype) for g in v["grads"]], "norm": norm.float().reshape(1)}


# ----------------------------------------------------------------------------
# What a pass cannot do without, and its exact outputs
# ----------------------------------------------------------------------------
def work(case):
    if case["op"] == "clip":
        sizes = _clip_sizes(case)
        return {"bytes": sum(2 * c * (4 if t == "f32" else 2) for c, t in sizes) + 4, "flops": 3 * sum(c for c, _ in sizes)}
    m, n, k, fwd = case["m"], case["n"], case["k"], case["way"] == "fwd"
    bias = 4 * n if case["bias"] else 0
    if case["op"] == "linear" and fwd:
        y = 4 if case["y"] == "f32" else 2
        return {"bytes": 2 * (m * k + n * k) + bias + m * n * (y * (2 if case["residual"] else 1) + (2 if case["save"] else 0)), "flops": 2 * m * n * k}
    if case["op"] == "linear":
        return {"bytes": 4 * (m * k + n * k) + bias + 2 * m * n * (1 if case["act"] == "none" else 2), "flops": 4 * m * n * k}
    if fwd:
        return {"bytes": 2 * (m * k + 2 * n * k) + 2 * bias + 2 * m * n * (3 if case["save"] else 1), "flops": 4 * m * n * k}
    return {"bytes": 4 * (m * k + 2 * n * k) + 2 * bias + 6 * m * n, "flops": 8 * m * n * k}


def exact(case, seed):
    """The outputs from the definitions, in 64 bits."""
    v = {name: [g.double() for g in x] if isinstance(x, list) else x.double() for name, x in _inputs(case, seed).items()}
    if case["op"] == "clip":
        total = sum(float(torch.dot(g, g)) for g in v["grads"])
        factor = min(1.0, case["share"] * _expected_norm(case) / (math.sqrt(total) + EPS))
        return {"grads": [g * factor for g in v["grads"]], "norm": torch.tensor([math.sqrt(total)], dtype=torch.float64)}

    name = case["act"]

    def phi(z):  # the activation and its derivative, by its own formula
        if name == "none":
            return z, torch.ones_like(z)
        if name == "relu":
            on = torch.where(z > 0, 1.0, 0.0).double()
            return z * on, on
        if name == "gelu":
            cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
            return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        if name == "gelu_tanh":  # (1 + tanh a) / 2 = 1 / (1 + exp(-2a))
            a = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
            s = torch.sigmoid(2 * a)
            return z * s, s + z * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
        s = torch.sigmoid(z)
        return (z * s, s + z * s * (1 - s)) if name == "silu" else (s, s * (1 - s))

    if case["op"] == "linear":
        if case["way"] == "fwd":
            z = v["X"] @ v["W"].T + v.get("b", 0.0)
            y = phi(z)[0] + v.get("R", 0.0)
            return {"Y": y, "Z": z} if case["save"] else {"Y": y}
        g = v["dY"] * phi(v["Z"])[1] if name != "none" else v["dY"]
        r = {"dX": g @ v["W"], "dW": (v["X"].T @ g).T}
        if case["bias"]:
            r["db"] = torch.einsum("mn->n", g)
        return r
    if case["way"] == "fwd":
        g, u = v["X"] @ v["Wg"].T + v.get("bg", 0.0), v["X"] @ v["Wu"].T + v.get("bu", 0.0)
        r = {"H": phi(g)[0] * u}
        if case["save"]:
            r["G"], r["U"] = g, u
        return r
    a, slope = phi(v["G"])
    du, dg = v["dH"] * a, v["dH"] * v["U"] * slope
    r = {"dX": torch.cat([dg, du], 1) @ torch.cat([v["Wg"], v["Wu"]], 0), "dWg": (v["X"].T @ dg).T, "dWu": (v["X"].T @ du).T}
    if case["bias"]:
        r["dbg"], r["dbu"] = torch.einsum("mn->n", dg), torch.einsum("mn->n", du)
    return r
