"""Performance cases of the operators around the feed-forward products.

What stands before and after the products of a feed-forward block when it is
trained, and its products in 8 bits when it is served:

  norm   mean, rstd over each row;  y = (x - mean) rstd gamma + beta
         back: dx = rstd (g - mean(g) - xh mean(g xh)) + r, g = dy gamma, xh = (x - mean) rstd;
               dgamma = sum dy xh;  dbeta = sum dy (over the rows)
  drop   y = (word < T ? 0 : x 2^32 / (2^32 - T)) + r, T = round(p 2^32), the words from a counter-based
         generator (Philox4x32-10 of Salmon, Moraes, Dror and Shaw, 2011): key = seed, counter = (column / 4, row, offset + step)
  i8     each row in 8 bits, s = max|x| / 127, q = round(127 x / max|x|) with ties to even, of x or of a norm's outputs;
         linear: y = act(sum q w * sw * s + b) + r;  glu: the same for two weights, h = act(g) u

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
EPS = 1e-5  # added to the variance


def listed():
    return [
        # one token's norm before a projection, while serving
        case_norm("token", "fwd", 1, 4096, "bf16"),
        # a training batch's norm, its statistics kept for the backward pass
        case_norm("train", "fwd", 8192, 4096, "bf16", save=True),
        # rows of odd length out of a residual stream that is kept in fp32
        case_norm("ragged", "fwd", 1000, 5001, "f16", x="f32", save=True),
        # the backward pass of the training batch, the residual's gradient added
        case_norm("train", "bwd", 8192, 4096, "bf16", residual=True),
        # a small batch with rows of odd length
        case_norm("ragged", "bwd", 777, 1001, "f16"),
        # the end of a block in training: dropout of the block's output, added to the residual stream
        case_drop("train", 8192, 8192, "bf16", "bf16", 0.1, residual=True),
        # the same for a small batch, an odd width and a stream in fp32
        case_drop("ragged", 333, 1001, "f16", "f32", 0.25, residual=True),
        # one token: norm to 8 bits, then a square projection with the residual
        case_i8("token", "linear", "norm", 1, 4096, 4096, "bf16", "none", bias=True, residual=True),
        # a ragged handful of rows, odd lengths, scores in fp32
        case_i8("ragged", "linear", "rows", 131, 5003, 2049, "f16", "none", y="f32"),
        # a long prompt through the widening projection
        case_i8("prompt", "linear", "rows", 8192, 16384, 4096, "bf16", "gelu_tanh", bias=True),
        # a small serving batch through the gated block's two projections
        case_i8("batch", "glu", "norm", 24, 10944, 4096, "bf16", "silu"),
        # a prompt through them
        case_i8("prompt", "glu", "norm", 4096, 10944, 4096, "f16", "silu", bias=True),
    ]


def case_norm(name, way, m, n, kind, x=None, save=False, residual=False):
    return {"name": "norm_%s_%s" % (way, name), "op": "norm", "way": way, "m": m, "n": n, "type": kind, "x": x or kind, "save": save,
            "residual": residual}


def case_drop(name, m, n, x, y, p, residual=False):
    return {"name": "drop_%s" % name, "op": "drop", "m": m, "n": n, "x": x, "y": y, "p": p, "residual": residual}


def case_i8(name, form, start, m, n, k, kind, act, bias=False, residual=False, y=None):
    return {"name": "i8_%s_%s" % (form, name), "op": "i8", "form": form, "start": start, "m": m, "n": n, "k": k, "type": kind, "act": act,
            "bias": bias, "residual": residual, "y": y or kind}


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A row length: most are multiples of 64 or 16, some are odd."""
    v = _spread(rng, low, high)
    step = rng.choice((64, 64, 16, 1))
    return max(low, v // step * step)


def draw(rng):
    op = rng.choice(("norm", "norm", "drop", "i8", "i8", "i8"))
    kind = rng.choice(("f16", "bf16"))
    m = _spread(rng, 1, 8192)
    if op == "norm":
        way, n = rng.choice(("fwd", "bwd")), _width(rng, 64, 20000)
        while m * n > 1 << 25:
            m = max(1, m // 2)
        return {"op": "norm", "way": way, "m": m, "n": n, "type": kind, "x": rng.choice((kind, kind, "f32")),
                "save": way == "fwd" and rng.random() < 0.5, "residual": way == "bwd" and rng.random() < 0.5}
    if op == "drop":
        n = _width(rng, 64, 20000)
        while m * n > 1 << 26:
            m = max(1, m // 2)
        return {"op": "drop", "m": m, "n": n, "x": rng.choice((kind, kind, "f32")), "y": rng.choice((kind, kind, "f32")),
                "p": rng.choice((0.05, 0.1, 0.25, 0.5)), "residual": rng.random() < 0.6}
    form, n, k = rng.choice(("linear", "glu")), _width(rng, 256, 16384), _width(rng, 256, 8192)
    while m * n * k * (2 if form == "glu" else 1) > 5.0e11:
        m = max(1, m // 2)
    linear = form == "linear"
    return {"op": "i8", "form": form, "start": rng.choice(("norm", "rows")), "m": m, "n": n, "k": k, "type": kind,
            "act": rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")) if linear else rng.choice(("silu", "gelu_tanh", "sigmoid")),
            "bias": rng.random() < 0.5, "residual": linear and rng.random() < 0.5, "y": kind}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _inputs(case, seed):
    """The tensors that a pass reads, from the seed alone."""
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed) * 1000003 + 29)

    def normal(*shape, std=1.0, kind):
        return (torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32) * std).to(TYPES[kind])

    def stream(m, n, kind):
        """Rows of a residual stream: a size of their own for every row, columns with means of their own."""
        x = torch.randn(m, n, generator=gen, device=DEVICE, dtype=torch.float32)
        x = x * torch.exp(0.3 * torch.randn(m, 1, generator=gen, device=DEVICE)) + 0.3 + 0.2 * torch.randn(1, n, generator=gen, device=DEVICE)
        return x.to(TYPES[kind])

    def affine(v, n):
        v["gamma"], v["beta"] = 1 + normal(n, std=0.1, kind="f32"), normal(n, std=0.1, kind="f32")

    def weights(v, name, n, k):
        """Normal weights that keep the size of activations, in 8 bits with a scale for each channel."""
        w = normal(n, k, std=k ** -0.5, kind="f32")
        v["s" + name] = w.abs().amax(1) / 127
        v[name] = torch.round(w / v["s" + name][:, None]).to(torch.int8)

    m, n, v = case["m"], case["n"], {}
    if case["op"] == "norm":
        v["x"] = stream(m, n, case["x"])
        affine(v, n)
        if case["way"] == "bwd":
            v["dy"] = normal(m, n, std=1e-2, kind=case["type"])
            x = v["x"].double()  # what the forward pass left
            v["mean"] = x.mean(1).float()
            v["rstd"] = (1 / torch.sqrt(x.var(1, unbiased=False) + EPS)).float()
            if case["residual"]:
                v["r"] = normal(m, n, std=1e-2, kind=case["x"])
    elif case["op"] == "drop":
        v["x"] = normal(m, n, kind=case["x"])
        if case["residual"]:
            v["r"] = stream(m, n, case["y"])
        v["step"] = torch.full((1,), 1000 * (int(seed) % 1000) + 7, dtype=torch.int64, device=DEVICE)  # the program's count of passes
    else:
        k = case["k"]
        if case["start"] == "norm":
            v["x"] = stream(m, k, case["type"])
            affine(v, k)
        else:
            v["x"] = normal(m, k, kind=case["type"])
        for name in ("w",) if case["form"] == "linear" else ("wg", "wu"):
            weights(v, name, n, k)
            if case["bias"]:
                v["b" + name] = normal(n, std=0.1, kind="f32")
        if case["residual"]:
            v["r"] = normal(m, n, kind=case["y"])
    return v


SEED = 0x5DEECE66D1234567  # of the generator: a program has one
OFFSET = 3                 # and a number for each place that drops


def prepare(case, seed):
    v = _inputs(case, seed)
    m, n = case["m"], case["n"]
    new = lambda *shape, kind: torch.empty(*shape, dtype=TYPES[kind], device=DEVICE)  # noqa: E731
    out = {}
    if case["op"] == "norm" and case["way"] == "fwd":
        out["y"] = new(m, n, kind=case["type"])
        if case["save"]:
            out["mean"], out["rstd"] = new(m, kind="f32"), new(m, kind="f32")
    elif case["op"] == "norm":
        out["dx"], out["dgamma"], out["dbeta"] = new(m, n, kind=case["x"]), new(n, kind="f32"), new(n, kind="f32")
    else:
        out["y"] = new(m, n, kind=case["y"])
    state = {"case": case, "in": v, "out": out}
    if own:  # scratch memory that a program allocates once, of the size that the library asks for
        if case["op"] == "i8":
            state["q"] = torch.empty(m, case["k"], dtype=torch.int8, device=DEVICE)
            state["s"] = new(m, kind="f32")
        size = _call(state, None)
        state["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEVICE)
    return state


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(state):
    case, v = state["case"], state["in"]
    if own:
        _call(state, state["workspace"])
        return state["out"]
    if case["op"] == "norm":
        return _plain_norm(case, v) if case["way"] == "fwd" else _plain_norm_back(case, v)
    return _plain_drop(case, v) if case["op"] == "drop" else _plain_i8(case, v)


def _call(state, workspace):
    """The library's calls for a case; without a workspace, the bytes of workspace that they need."""
    import implicit_gemm_convolution_amd as igc

    case, v, out = state["case"], state["in"], state["out"]
    kind = {"f16": igc.IGC_F16, "bf16": igc.IGC_BF16, "f32": igc.IGC_F32}
    size = workspace is None
    more = {} if size else {"workspace": workspace}
    m, n = case["m"], case["n"]
    if case["op"] == "drop":
        if not size:
            igc.dropout(m, n, v["x"], n, out["y"], n, case["p"], SEED, OFFSET, step=v["step"], R=v.get("r"), ldr=n,
                        type=kind[case["x"]], y_type=kind[case["y"]])
        return 0
    if case["op"] == "norm" and case["way"] == "fwd":
        if not size:
            igc.layer_norm_forward(m, n, v["x"], n, out["y"], n, gamma=v["gamma"], beta=v["beta"], eps=EPS, mean=out.get("mean"),
                                   rstd=out.get("rstd"), type=kind[case["type"]], x_type=kind[case["x"]])
        return 0
    if case["op"] == "norm":
        f = igc.layer_norm_backward_workspace_size if size else igc.layer_norm_backward
        return f(m, n, v["dy"], n, v["x"], n, v["mean"], v["rstd"], gamma=v["gamma"], R=v.get("r"), ldr=n, dX=out["dx"], lddx=n,
                 dgamma=out["dgamma"], dbeta=out["dbeta"], type=kind[case["type"]], x_type=kind[case["x"]], **more)
    k, q, s = case["k"], state["q"], state["s"]
    if not size and case["start"] == "norm":
        igc.layer_norm_forward(m, k, v["x"], k, None, k, gamma=v["gamma"], beta=v["beta"], eps=EPS, Q=q, ldq=k, scale=s, type=kind[case["type"]])
    elif not size:
        igc.quantize_rows(m, k, v["x"], k, q, k, s, type=kind[case["type"]])
    act = {"none": igc.IGC_ACT_NONE, "relu": igc.IGC_ACT_RELU, "gelu": igc.IGC_ACT_GELU, "gelu_tanh": igc.IGC_ACT_GELU_TANH,
           "silu": igc.IGC_ACT_SILU, "sigmoid": igc.IGC_ACT_SIGMOID}[case["act"]]
    if case["form"] == "linear":
        f = igc.linear_i8_workspace_size if size else igc.linear_i8
        return f(m, n, k, q, k, s, v["w"], k, v["sw"], out["y"], n, bias=v.get("bw"), R=v.get("r"), ldr=n, act=act, y_type=kind[case["y"]], **more)
    f = igc.glu_i8_workspace_size if size else igc.glu_i8
    return f(m, n, k, q, k, s, v["wg"], k, v["swg"], v["wu"], k, v["swu"], out["y"], n, bias_g=v.get("bwg"), bias_u=v.get("bwu"), act=act,
             type=kind[case["type"]], **more)


def _norm(x):
    """Mean and 1 / deviation of each row, and the rows by them."""
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    return mean, rstd, d * rstd


def _plain_norm(case, v):
    mean, rstd, xh = _norm(v["x"].float())
    out = {"y": (xh * v["gamma"] + v["beta"]).to(TYPES[case["type"]])}
    if case["save"]:
        out["mean"], out["rstd"] = mean[:, 0], rstd[:, 0]
    return out


def _plain_norm_back(case, v):
    dy, rstd = v["dy"].float(), v["rstd"][:, None]
    xh = (v["x"].float() - v["mean"][:, None]) * rstd
    g = dy * v["gamma"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if case["residual"]:
        dx = dx + v["r"].float()
    return {"dx": dx.to(TYPES[case["x"]]), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


def _wide(a, b):
    """High and low word of the products of 32-bit words (held in 64-bit integers) with the word b."""
    t = a * (b & 0xFFFF)
    u = a * (b >> 16) + (t >> 16)
    return u >> 16, ((u & 0xFFFF) << 16) | (t & 0xFFFF)


def _words(m, n, step):
    """The generator's words for m x n elements."""
    low, high = SEED & 0xFFFFFFFF, SEED >> 32
    at = step + OFFSET  # (on the GPU)
    c0 = torch.arange((n + 3) // 4, device=DEVICE).expand(m, -1)
    c1 = torch.arange(m, device=DEVICE)[:, None].expand_as(c0)
    c2, c3 = (at & 0xFFFFFFFF).expand_as(c0), (at >> 32 & 0xFFFFFFFF).expand_as(c0)
    for _ in range(10):
        h0, l0 = _wide(c0, 0xD2511F53)
        h1, l1 = _wide(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ low, l1, h0 ^ c3 ^ high, l0
        low, high = (low + 0x9E3779B9) & 0xFFFFFFFF, (high + 0xBB67AE85) & 0xFFFFFFFF
    return torch.stack((c0, c1, c2, c3), 2).reshape(m, -1)[:, :n]


def _plain_drop(case, v):
    border = round(case["p"] * 2 ** 32)
    y = torch.where(_words(case["m"], case["n"], v["step"]) < border, 0.0, v["x"].float() * (2.0 ** 32 / (2 ** 32 - border)))
    if case["residual"]:
        y = y + v["r"].float()
    return {"y": y.to(TYPES[case["y"]])}


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


def _plain_rows(x):
    """Rows in 8 bits (as whole fp32 numbers) and their scales.  127 x is exact, and of 16-bit values no quotient but a tie
    lies within 2^-19 of its size of a tie: rounded once to fp32 it goes where the exact one goes."""
    top = x.float().abs().amax(1, keepdim=True)
    return torch.round(127 * x.float() / top), top / 127


def _plain_i8(case, v):
    x = v["x"]
    if case["start"] == "norm":
        x = (_norm(x.float())[2] * v["gamma"] + v["beta"]).to(x.dtype)
    q, s = _plain_rows(x)
    # (sums of whole numbers: exact in fp32 as far as 2^24, which sums of this many random terms stay below)
    z = [torch.matmul(q, v[w].float().t()) * v["s" + w] * s for w in (("w",) if case["form"] == "linear" else ("wg", "wu"))]
    if case["bias"]:
        z = [a + v[b] for a, b in zip(z, ("bw",) if case["form"] == "linear" else ("bwg", "bwu"))]
    y = _act(case["act"], z[0])
    if case["form"] == "glu":
        y = y * z[1]
    if case["residual"]:
        y = y + v["r"].float()
    return {"y": y.to(TYPES[case["y"]])}


# ----------------------------------------------------------------------------
# What a pass cannot do without, and its exact outputs
# ----------------------------------------------------------------------------
def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4}
    m, n = case["m"], case["n"]
    if case["op"] == "norm" and case["way"] == "fwd":
        return {"bytes": m * n * (size[case["x"]] + size[case["type"]]) + 8 * n + (8 * m if case["save"] else 0), "flops": 8 * m * n}
    if case["op"] == "norm":
        return {"bytes": m * n * (size[case["type"]] + size[case["x"]] * (3 if case["residual"] else 2)) + 8 * m + 12 * n, "flops": 14 * m * n}
    if case["op"] == "drop":  # 10 rounds of 2 wide products and 6 operations for each 4 elements
        return {"bytes": m * n * (size[case["x"]] + size[case["y"]] * (2 if case["residual"] else 1)), "flops": 23 * m * n}
    k, products = case["k"], 2 if case["form"] == "glu" else 1
    return {"bytes": 2 * m * k + products * n * (k + (8 if case["bias"] else 4)) + (8 * k if case["start"] == "norm" else 0)
            + m * n * size[case["y"]] * (2 if case["residual"] else 1), "flops": 2 * products * m * n * k}


def exact(case, seed):
    """The outputs from the definitions, in 64 bits."""
    raw = _inputs(case, seed)
    v = {name: t.double() for name, t in raw.items()}

    def normed(x):
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        return mean, (var + EPS) ** -0.5

    if case["op"] == "norm" and case["way"] == "fwd":
        mean, rstd = normed(v["x"])
        r = {"y": torch.addcmul(v["beta"], (v["x"] - mean) * rstd, v["gamma"])}
        if case["save"]:
            r["mean"], r["rstd"] = mean.squeeze(1), rstd.squeeze(1)
        return r
    if case["op"] == "norm":
        n = case["n"]
        xh = torch.addcmul(-(v["mean"] * v["rstd"]).unsqueeze(1), v["x"], v["rstd"].unsqueeze(1))
        g = v["dy"] * v["gamma"]
        # the row's gradient is n g less its parts along the ones and along xh
        along = torch.einsum("mn,mn->m", g, xh).unsqueeze(1)
        dx = (n * g - torch.einsum("mn->m", g).unsqueeze(1) - xh * along) * v["rstd"].unsqueeze(1) / n
        return {"dx": dx + v.get("r", 0.0), "dgamma": torch.einsum("mn,mn->n", v["dy"], xh), "dbeta": torch.einsum("mn->n", v["dy"])}
    if case["op"] == "drop":
        import numpy as np

        m, n = case["m"], case["n"]
        if m * n > 1 << 27:
            return None
        at = int(raw["step"][0]) + OFFSET
        a = np.tile(np.arange((n + 3) // 4, dtype=np.uint64), (m, 1))
        b = np.broadcast_to(np.arange(m, dtype=np.uint64)[:, None], a.shape)
        c, d = np.full(a.shape, at % 2 ** 32, dtype=np.uint64), np.full(a.shape, at // 2 ** 32, dtype=np.uint64)
        word, half = np.uint64(0xFFFFFFFF), np.uint64(32)
        for i in range(10):
            p, q = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)  # (of 32-bit words: 64 bits hold them)
            x, y = (SEED + i * 0x9E3779B9) % 2 ** 32, ((SEED >> 32) + i * 0xBB67AE85) % 2 ** 32
            a, b, c, d = (q >> half) ^ b ^ np.uint64(x), q & word, (p >> half) ^ d ^ np.uint64(y), p & word
        words = np.empty((m, a.shape[1] * 4), dtype=np.int64)
        words[:, 0::4], words[:, 1::4], words[:, 2::4], words[:, 3::4] = a, b, c, d
        border = math.floor(case["p"] * 2 ** 32 + 0.5)
        kept = torch.from_numpy(words[:, :n] >= border).to(DEVICE)
        return {"y": v["x"] * kept * (2 ** 32 / (2 ** 32 - border)) + v.get("r", 0.0)}
    x = v["x"]
    if case["start"] == "norm":
        mean, rstd = normed(x)
        x = torch.addcmul(v["beta"], (x - mean) * rstd, v["gamma"]).to(raw["x"].dtype).double()  # (what is put into 8 bits is of the 16-bit type)
    top = torch.linalg.vector_norm(x, ord=math.inf, dim=1)
    q, s = (x * 127 / top.unsqueeze(1)).round(), top / 127

    def product(w):
        z = q @ v[w].T * torch.outer(s, v["s" + w])
        return z + v["b" + w] if case["bias"] else z

    def phi(z):  # the activation, by its own formula
        name = case["act"]
        if name == "none":
            return z
        if name == "relu":
            return torch.where(z > 0, z, torch.zeros_like(z))
        if name == "gelu":
            return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
        if name == "gelu_tanh":  # (1 + tanh a) / 2 = 1 / (1 + exp(-2a))
            return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return z * torch.sigmoid(z) if name == "silu" else torch.sigmoid(z)

    if case["form"] == "glu":
        return {"y": phi(product("wg")) * product("wu")}
    return {"y": phi(product("w")) + v.get("r", 0.0)}
