"""The operators of a quantized feed-forward network and their gradients, as a user's program calls them.

  linear        Y  = act(X . W^T + bias) + residual            W^ in 4 bits: (q - z) * scale * s
  linear_grad   dZ = dY * act'(Z);  dX = dZ . W^;  dbias = sum of dZ over the tokens
  gated         H  = act(X . Wg^T + bg) * (X . Wu^T + bu)      W^ = [Wg; Wu], one packed matrix of 2F rows
  gated_grad    dG = dH * U * act'(G), dU = dH * act(G);  dX = [dG dU] . W^;  dbias as above

The weights are frozen: gradients go to the activations and to the bias.  Z = [G U] are the pre-activations that a
training step saves in the activations' type.  Layers are 8B and 70B feed-forward and attention projections.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _case(name, op, M, N, K, dtype="bf16", group=128, awq=False, bias=False, residual=False, act="none", save=False):
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "dtype": dtype, "group": group, "awq": awq, "bias": bias,
            "residual": residual, "act": act, "save": save}


def listed():
    return [
        # decoding one token: the attention output projection, added to the residual stream
        _case("linear_o_proj_1", "linear", 1, 4096, 4096, residual=True),
        # checking drafted tokens: the down projection with AWQ scales, added to the residual stream
        _case("linear_down_16_awq", "linear", 16, 4096, 14336, awq=True, residual=True),
        # an encoder-style layer of odd width over a short ragged batch, fp16, groups of 64
        _case("linear_odd_77_f16", "linear", 77, 1001, 1088, dtype="f16", group=64, bias=True, act="gelu_tanh"),
        # a prompt of a large model: the attention output projection into the residual stream
        _case("linear_o_proj_2048", "linear", 2048, 8192, 8192, residual=True),
        # a training step of adapters on a frozen layer: gradient of the fused q, k, v projection with bias
        _case("linear_grad_qkv_512", "linear_grad", 512, 6144, 4096, bias=True),
        # the same of an activated layer of odd width, fp16
        _case("linear_grad_odd_301_f16", "linear_grad", 301, 1001, 1088, dtype="f16", group=64, bias=True, act="gelu_tanh"),
        # decoding one token: gate and up projections and their product
        _case("gated_1", "gated", 1, 28672, 4096, act="silu"),
        # a small batch of drafted tokens with AWQ scales
        _case("gated_48_awq", "gated", 48, 28672, 4096, awq=True, act="silu"),
        # a long prompt of a large model
        _case("gated_8192", "gated", 8192, 57344, 8192, act="silu"),
        # forward of a training step: the pre-activations are kept
        _case("gated_train_2048", "gated", 2048, 28672, 4096, act="silu", save=True),
        # backward of that step
        _case("gated_grad_2048", "gated_grad", 2048, 28672, 4096, act="silu"),
        # backward of a small odd block with AWQ scales, groups of 32 and biases
        _case("gated_grad_odd_203", "gated_grad", 203, 2 * 1003, 640, group=32, awq=True, bias=True, act="gelu_tanh"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "gated", "linear_grad", "gated_grad"])
    group = rng.choice([128, 128, 128, 64, 32])
    unit = max(group, 64)
    K = unit * max(1, _log(rng, 256, 28672) // unit)
    N = _log(rng, 64, 57344)
    M = _log(rng, 1, 8192)
    if rng.random() < 0.5:
        N = max(8, N // 8 * 8)  # widths of models; the others are odd
    N = min(N, 57344 * 8192 // K)  # the largest layer's weights
    M = max(1, min(M, (1 << 40) // (N * K)))
    gated = op.startswith("gated")
    if gated:
        N = 2 * max(1, N // 2)
    act = rng.choice(["silu", "gelu_tanh", "relu"]) if gated else rng.choice(["none", "none", "gelu_tanh", "silu", "relu"])
    c = _case("", op, M, N, K, dtype=rng.choice(["bf16", "bf16", "f16"]), group=group, awq=rng.random() < 0.3,
              bias=rng.random() < 0.4, residual=op == "linear" and rng.random() < 0.5, act=act,
              save=op in ("linear", "gated") and act != "none" and rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    M, N, K, group = case["M"], case["N"], case["K"], case["group"]
    gated, grad = case["op"].startswith("gated"), case["op"].endswith("_grad")
    dt = _DT[case["dtype"]]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    st = {"case": case}
    # a layer's channels differ in size: 1 % of them carry activations 5 times as large
    gain = torch.where(torch.rand(K, generator=gen, device="cuda") < 0.01, 5.0, 1.0)
    s = (0.8 * gain).sqrt() if case["awq"] else None
    st["packed"], st["scales"], st["zeros"] = _quantize(normal(N, K) * (1.28 / math.sqrt(K)), s, group)
    st["awq_s"] = s
    st["bias"] = normal(N) * 0.2 if case["bias"] and not grad else None
    if not grad:
        st["X"] = (normal(M, K) * gain).to(dt)
        st["residual"] = (normal(M, N) * 3).to(dt) if case["residual"] else None
    else:
        out = N // 2 if gated else N
        # gradients are small, and their size differs from token to token
        size = torch.exp(normal(M, 1) - (4.0 if case["dtype"] == "f16" else 9.0))
        st["dY"] = (normal(M, out) * size).to(dt)
        st["Z"] = (normal(M, N) * 1.4).to(dt) if gated or case["act"] != "none" else None
    return st


def _quantize(W, s, group):
    """Round to nearest, asymmetric, 4 bits: codes two to a byte (low nibble: even k), fp16 scales and zero points."""
    N, K = W.shape
    if s is not None:
        W = W / s
    w = W.view(N, K // group, group)
    mn, mx = w.amin(2, keepdim=True), w.amax(2, keepdim=True)
    scale = ((mx - mn) / 15).to(torch.float16)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    z = torch.round(-mn / scale.float()).clamp_(0, 15)
    q = (torch.round(w / scale.float()) + z).clamp_(0, 15).to(torch.uint8).view(N, K)
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), scale.view(N, -1).contiguous(), z.view(N, -1).to(torch.float16).contiguous()


# ------------------------------------------------------------------ one pass
_w4 = None


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    W = _weights(st)
    if c["op"] == "linear":
        Z = st["X"].float() @ W.t()
        if st["bias"] is not None:
            Z += st["bias"]
        Y = _act(Z, c["act"])
        if st["residual"] is not None:
            Y = Y + st["residual"].float()
        return _out(st, Y, Z)
    if c["op"] == "gated":
        Z = st["X"].float() @ W.t()
        if st["bias"] is not None:
            Z += st["bias"]
        G, U = Z[:, : c["N"] // 2], Z[:, c["N"] // 2:]
        return _out(st, _act(G, c["act"]) * U, Z)
    dY = st["dY"].float()
    if c["op"] == "linear_grad":
        dZ = dY if st["Z"] is None else dY * _dact(st["Z"].float(), c["act"])
    else:
        G, U = st["Z"][:, : c["N"] // 2].float(), st["Z"][:, c["N"] // 2:].float()
        dZ = torch.cat([dY * U * _dact(G, c["act"]), dY * _act(G, c["act"])], 1)
    dX = (dZ @ W).to(st["dY"].dtype)
    return {"dX": dX, "dbias": dZ.sum(0)} if c["bias"] else {"dX": dX}


def _out(st, Y, Z):
    dt = st["X"].dtype
    return {"Y": Y.to(dt), "Z": Z.to(dt)} if st["case"]["save"] else {"Y": Y.to(dt)}


def _weights(st):
    """W^ [N, K] in 32 bits."""
    p, g = st["packed"], st["case"]["group"]
    N, K = p.shape[0], p.shape[1] * 2
    q = torch.stack([p & 15, p >> 4], 2).view(N, K // g, g).float()
    W = ((q - st["zeros"].float()[:, :, None]) * st["scales"].float()[:, :, None]).view(N, K)
    return W if st["awq_s"] is None else W * st["awq_s"]


_C = math.sqrt(2 / math.pi)


def _act(x, act):
    if act == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(_C * (x + 0.044715 * x * x * x)))
    return x


def _dact(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if act == "gelu_tanh":
        t = torch.tanh(_C * (x + 0.044715 * x * x * x))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * _C * (1 + 3 * 0.044715 * x * x)
    return torch.ones_like(x)


def _run_own(st):
    global _w4
    if _w4 is None:
        from weight_only_int4_w4_b200 import w4 as _w4
    c = st["case"]
    w = (st["packed"], st["scales"], st["zeros"])
    if c["op"] == "linear":
        r = _w4.w4a16_linear(st["X"], *w, awq_s=st["awq_s"], bias=st["bias"], act=c["act"], residual=st["residual"],
                             save_preact=c["save"], group=c["group"])
    elif c["op"] == "gated":
        r = _w4.w4a16_gated(st["X"], *w, awq_s=st["awq_s"], bias=st["bias"], act=c["act"], save_preact=c["save"],
                            group=c["group"])
    elif c["op"] == "linear_grad":
        r = _w4.w4a16_linear_grad(st["dY"], *w, awq_s=st["awq_s"], preact=st["Z"], act=c["act"], dbias=c["bias"],
                                  group=c["group"])
    else:
        r = _w4.w4a16_gated_grad(st["dY"], st["Z"], *w, awq_s=st["awq_s"], act=c["act"], dbias=c["bias"],
                                 group=c["group"])
    names = ("dX", "dbias") if c["op"].endswith("_grad") else ("Y", "Z")
    return dict(zip(names, r if isinstance(r, tuple) else (r,)))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    M, N, K = case["M"], case["N"], case["K"]
    gated, grad = case["op"].startswith("gated"), case["op"].endswith("_grad")
    out = N // 2 if gated else N
    b = N * K // 2 + 4 * N * (K // case["group"]) + 2 * M * K + 2 * M * out  # weights, X or dX, Y or dY
    b += 4 * K if case["awq"] else 0
    b += 4 * N if case["bias"] else 0
    b += 2 * M * N if case["residual"] or case["save"] else 0
    b += 2 * M * N if case["residual"] and case["save"] else 0
    b += 2 * M * N if grad and (gated or case["act"] != "none") else 0
    return {"bytes": b, "flops": 2 * M * N * K}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definition in 64 bits, one weight group after another: sum over the groups of scale * (x s) . (q - z)."""
    st = prepare(case, seed)
    N, K, g = case["N"], case["K"], case["group"]
    act, gated = case["act"], case["op"].startswith("gated")
    scales, zeros, packed = st["scales"].double(), st["zeros"].double(), st["packed"]
    s = st["awq_s"].double() if st["awq_s"] is not None else torch.ones(K, device="cuda", dtype=torch.float64)

    def block(k):  # columns k*g .. of W^, without s
        b = packed[:, k * g // 2:(k + 1) * g // 2].to(torch.int32)
        q = torch.empty((N, g), device="cuda", dtype=torch.float64)
        q[:, 0::2] = (b % 16).double()
        q[:, 1::2] = torch.div(b, 16, rounding_mode="floor").double()
        return (q - zeros[:, k:k + 1]) * scales[:, k:k + 1]

    if not case["op"].endswith("_grad"):
        X = st["X"].double() * s
        Z = torch.zeros((case["M"], N), device="cuda", dtype=torch.float64)
        if st["bias"] is not None:
            Z += st["bias"].double()
        for k in range(K // g):
            Z.addmm_(X[:, k * g:(k + 1) * g], block(k).t())
        Y = _f64(Z[:, : N // 2], act) * Z[:, N // 2:] if gated else _f64(Z, act)
        if case["residual"]:
            Y = Y + st["residual"].double()
        return {"Y": Y, "Z": Z} if case["save"] else {"Y": Y}
    dY = st["dY"].double()
    if gated:
        G, U = st["Z"][:, : N // 2].double(), st["Z"][:, N // 2:].double()
        dZ = torch.empty((case["M"], N), device="cuda", dtype=torch.float64)
        dZ[:, : N // 2] = dY * U * _slope64(G, act)
        dZ[:, N // 2:] = dY * _f64(G, act)
    else:
        dZ = dY if st["Z"] is None else dY * _slope64(st["Z"].double(), act)
    dX = torch.empty((case["M"], K), device="cuda", dtype=torch.float64)
    for k in range(K // g):
        dX[:, k * g:(k + 1) * g] = (dZ @ block(k)) * s[k * g:(k + 1) * g]
    return {"dX": dX, "dbias": dZ.sum(0)} if case["bias"] else {"dX": dX}


def _f64(x, act):
    """tanh-GELU is x times the logistic function of 2u, u = sqrt(2/pi) (x + 0.044715 x^3); SiLU has u = x / 2."""
    if act == "none":
        return x
    if act == "relu":
        return x.clamp(min=0)
    u = x / 2 if act == "silu" else math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    return x * torch.sigmoid(2 * u)


def _slope64(x, act):
    if act == "none":
        return torch.ones_like(x)
    if act == "relu":
        return torch.heaviside(x, torch.zeros_like(x))
    u = x / 2 if act == "silu" else math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    du = 0.5 if act == "silu" else math.sqrt(2 / math.pi) * (1 + 0.134145 * x ** 2)
    p = torch.sigmoid(2 * u)
    return p + 2 * x * p * (1 - p) * du
