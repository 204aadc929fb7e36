"""The 8-bit linear layers of this library, as cases to measure.

A linear layer in 8 bits for serving, and what a training step keeps of one in
8 bits for its backward pass.  Both hold a matrix row by row as integers of
-127 .. 127 times a binary32 scale:

  quantize_rows, dequantize_rows   a matrix into that form and back (a scale
                                   for each row, or for each group of columns)
  linear_i8                        a linear layer whose weight is kept so, a
                                   scale for each output channel; its input is
                                   brought into that form token by token within
                                   the call, or is in it already
  linear_q8_backward               through a layer's activation and its weight
                                   and bias, from an input and a pre-activation
                                   that were kept in 8 bits

scale = max(largest |x| / 127, 2^-126) in binary32, integer = x / scale to the
nearest, ties to even.  `own` False computes them in plain torch in 32 bits,
`own` True calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, M, N, K, **more):
    c = {"name": name, "op": op, "M": M, "N": N, "K": K, "type": "bf16", "out": "bf16", "group": 0, "act": "none",
         "bias": False, "ready": False}
    c.update(more)
    return c


def listed():
    return [
        # one token's features stored and read back: two launches
        _case("store_1_token", "store", 1, 0, 4096),
        # a short batch of an odd width in 32 bits, a scale for each 64 columns
        _case("store_509_tokens_odd", "store", 509, 0, 770, type="f32", group=64),
        # a training step's widest activation
        _case("store_8192_tokens_wide", "store", 8192, 0, 11008, group=128),
        # one decode step of an attention projection
        _case("linear_1_token", "linear", 1, 4096, 4096),
        # a decode batch through a wide layer
        _case("linear_24_tokens_wide", "linear", 24, 11008, 4096, act="silu"),
        # many features into few, as a classifier's neck has it
        _case("linear_105_tokens_deep", "linear", 105, 1024, 12544, type="f32", out="f32", act="relu", bias=True),
        # an odd batch of an encoder
        _case("linear_509_tokens", "linear", 509, 2304, 768, act="gelu", bias=True),
        # one of several projections of an input that was quantised for all of them
        _case("linear_4096_tokens_ready", "linear", 4096, 4096, 4096, ready=True, out="f32"),
        # a long prompt through a wide layer
        _case("linear_8192_tokens_wide", "linear", 8192, 11008, 4096),
        # the backward pass of a short fine-tuning batch
        _case("backward_333_tokens", "backward", 333, 768, 768, act="gelu", bias=True, group=64),
        # an encoder's projection without an activation, gradients coming in 32 bits
        _case("backward_8192_tokens_plain", "backward", 8192, 2304, 768, type="f32", bias=True),
        # the largest: a wide layer with its activation
        _case("backward_8192_tokens_wide", "backward", 8192, 11008, 4096, act="silu", group=128),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    n = _between(rng, lo, hi)
    how = rng.random()
    return max(64, n // 64 * 64) if how < 0.6 else max(16, n // 16 * 16) if how < 0.85 else n


def draw(rng):
    op = rng.choice(["store", "linear", "linear", "backward"])
    K = _width(rng, 128, 12544)
    N = 0 if op == "store" else _width(rng, 128, 12544)
    M = _between(rng, 32 if op == "backward" else 1, 8192)
    # no more work than the largest listed case
    if op != "store":
        M = max(1, min(M, 8192 * 11008 * 4096 // (N * K)))
    c = _case("", op, M, N, K, type=rng.choice(["bf16", "bf16", "f32"]))
    del c["name"]
    if op != "linear":
        c["group"] = rng.choice([0, 32, 64, 128, 256])
    if op != "store":
        c["act"] = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        c["bias"] = rng.random() < 0.5
    if op == "linear":
        c["ready"] = rng.random() < 0.25
        c["out"] = rng.choice(["bf16", "f32"])
    return c


def _quantize(x, group):
    """(integers as int8, scales (rows, groups)); rows in whole 16-byte units, as the library lays them out."""
    M, K = x.shape
    g = group or K
    G = -(-K // g)
    wide = torch.zeros((M, G * g), dtype=torch.float32, device=x.device)
    wide[:, :K] = x
    top = wide.view(M, G, g).abs().amax(2)
    scale = (top.double() / 127.0).clamp_(min=2.0 ** -126).float()
    # (64 bits: quotients next to a half)
    q = torch.round(wide.view(M, G, g).double() / scale.double()[:, :, None]).view(M, G * g)[:, :K]
    out = torch.zeros((M, -(-K // 16) * 16), dtype=torch.int8, device=x.device)[:, :K]
    out.copy_(q)
    return out, scale if group else scale[:, 0]


def _values(q, scale, group):
    """The numbers that 8-bit integers and their scales stand for."""
    if scale.dim() == 1:
        return q.float() * scale[:, None]
    return q.float() * scale.repeat_interleave(group, 1)[:, :q.shape[1]]


def prepare(case, seed):
    M, N, K = case["M"], case["N"], case["K"]
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def features(n):
        # a few channels of a layer's input are far larger than the others
        gain = torch.exp(0.5 * normal(n))
        gain[torch.rand(n, generator=g, device=DEV) < 0.01] *= 12.0
        return normal(M, n) * gain

    t = TYPES[case["type"]]
    s = {"case": case}
    if case["op"] == "store":
        s["x"] = features(K).to(t)
        return s
    s["bias"] = 0.5 * normal(N) if case["bias"] and case["op"] == "linear" else None
    if case["op"] == "linear":
        s["w"], s["w_scale"] = _quantize(normal(N, K) * (1.0 / math.sqrt(K)), 0)
        x = features(K)
        if case["ready"]:
            s["x"], s["x_scale"] = _quantize(x, 0)
        else:
            s["x"], s["x_scale"] = x.to(t), None
        return s
    s["dy"] = (normal(M, N) * (1.0 / M)).to(t)
    s["x"], s["x_scale"] = _quantize(features(K), 0)
    s["z"], s["z_scale"] = _quantize(1.5 * normal(M, N), case["group"]) if case["act"] != "none" else (None, None)
    return s


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    p = 1.0 / (1.0 + torch.exp(-z))
    return p * (1.0 + z * (1.0 - p))


def _store(s, c):
    q, scale = _quantize(s["x"], c["group"])
    return {"scale": scale, "values": _values(q, scale, c["group"]).to(torch.bfloat16)}


def _linear(s, c):
    x, xs = (s["x"], s["x_scale"]) if c["ready"] else _quantize(s["x"], 0)
    y = (x.float() @ s["w"].float().t()) * s["w_scale"] * xs[:, None]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": _act(y, c["act"]).to(TYPES[c["out"]])}


def _backward(s, c):
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _slope(_values(s["z"], s["z_scale"], c["group"]), c["act"])
    dw = dz.t() @ _values(s["x"], s["x_scale"], 0)
    out = {"dz": dz.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}
    if c["bias"]:
        out["dbias"] = dz.sum(0)
    return out


def _with_library(s, c):
    import dynamic_shape_gemm_amd as mkp

    if c["op"] == "store":
        q, scale = mkp.quantize_rows(s["x"], group=c["group"])
        return {"scale": scale, "values": mkp.dequantize_rows(q, scale, group=c["group"])}
    if c["op"] == "linear":
        return {"y": mkp.linear_i8(s["x"], s["w"], s["w_scale"], s["bias"], act=c["act"], x_scale=s["x_scale"],
                                   dtype=TYPES[c["out"]])}
    dz, dw, dbias = mkp.linear_q8_backward(s["dy"], s["x"], s["x_scale"], s["z"], s["z_scale"], z_group=c["group"],
                                           act=c["act"], need_dbias=c["bias"])
    out = {"dz": dz, "dw": dw}
    if c["bias"]:
        out["dbias"] = dbias
    return out


def run(state):
    c = state["case"]
    if own:
        return _with_library(state, c)
    return _store(state, c) if c["op"] == "store" else _linear(state, c) if c["op"] == "linear" else _backward(state, c)


def work(case):
    M, N, K = case["M"], case["N"], case["K"]
    size = {"bf16": 2.0, "f32": 4.0}
    e = size[case["type"]]
    if case["op"] == "store":
        scales = 4.0 * M * (-(-K // case["group"]) if case["group"] else 1)
        # the input; integers and scales written and read; the values
        return {"bytes": (e + 1.0 + 1.0 + 2.0) * M * K + 2.0 * scales, "flops": 4.0 * M * K}
    vectors = 4.0 * N if case["bias"] else 0.0
    if case["op"] == "linear":
        x = M * K + 4.0 * M if case["ready"] else e * M * K
        return {"bytes": x + N * K + 4.0 * N + vectors + size[case["out"]] * M * N, "flops": 2.0 * M * N * K}
    z = 0.0
    if case["act"] != "none":
        z = M * N + 4.0 * M * (-(-N // case["group"]) if case["group"] else 1)
    # incoming gradient, kept pre-activation and input; gradients by the pre-activation, weight and bias
    return {"bytes": e * M * N + z + M * K + 4.0 * M + 2.0 * M * N + 2.0 * N * K + vectors, "flops": 2.0 * M * N * K}


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    act = case["act"]

    def nearest(x, scale):
        t = x / scale
        low = torch.floor(t)
        rest = t - low
        up = (rest > 0.5) | ((rest == 0.5) & (torch.remainder(low, 2.0) == 1.0))
        return low + up.double()

    def columns(scale, group, n):
        # each column's scale
        if scale.dim() == 1:
            return scale.double()[:, None].expand(-1, n)
        return scale.double()[:, torch.arange(n, device=DEV) // group]

    def scales(x, group):
        n = x.shape[1]
        parts = torch.split(x.abs(), group or n, dim=1)
        top = torch.stack([p.max(1).values for p in parts], 1)
        return torch.maximum(top / 127.0, torch.full_like(top, 2.0 ** -126))

    if case["op"] == "store":
        x, group = s["x"].double(), case["group"]
        wide = scales(x, group)
        at = columns(wide.float() if group else wide.float()[:, 0], group, x.shape[1])
        return {"scale": wide if group else wide[:, 0], "values": nearest(x, at) * at}
    if case["op"] == "linear":
        if case["ready"]:
            q, xs = s["x"].double(), s["x_scale"].double()[:, None]
        else:
            x = s["x"].double()
            xs = scales(x, 0).float().double()
            q = nearest(x, xs)
        y = torch.einsum("mk,nk->mn", q * xs, s["w"].double() * s["w_scale"].double()[:, None])
        if s["bias"] is not None:
            y = y + s["bias"].double()
        if act == "relu":
            y = torch.clamp(y, min=0.0)
        elif act == "gelu":
            y = y * torch.special.ndtr(y)
        elif act == "gelu_tanh":
            y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
        elif act == "silu":
            y = y * torch.sigmoid(y)
        return {"y": y}
    dz = s["dy"].double()
    if act != "none":
        z = s["z"].double() * columns(s["z_scale"], case["group"], s["z"].shape[1])
        if act == "relu":
            slope = torch.where(z > 0, 1.0, 0.0).double()
        elif act == "gelu":
            slope = torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        elif act == "gelu_tanh":
            c = 2.0 * math.sqrt(2.0 / math.pi)
            p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
            slope = p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z ** 2)
        else:
            p = torch.sigmoid(z)
            slope = p + z * p * (1 - p)
        dz = dz * slope
    x = s["x"].double() * s["x_scale"].double()[:, None]
    out = {"dz": dz, "dw": torch.matmul(dz.t(), x)}
    if case["bias"]:
        out["dbias"] = dz.sum(0)
    return out
