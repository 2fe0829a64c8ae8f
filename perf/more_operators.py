"""The measured cases of the feed-forward operators that stand around the private
update step:

  gated    the gated feed-forward block y = (act(x W_gate) * (x W_up)) W_down with
           its gradients; for the backward pass it keeps its input alone, or its
           input and both projections in 8 bits
  pack     writing an activation in 8 bits (blocks of 32 channels that share a
           power of two) and reading it back
  project  a layer's input written in 8 bits, and the layer's projected per-sample
           gradients from it

`run` computes a case in elementary torch operations in 32 bits, or, where `own`
is true, through dp_grape_projection_amd. B samples of T tokens; the last tokens
of a sample may be padding, whose activations and gradients are zero.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    def gated(name, B, T, d, f, dtype, act, keep, dx, dw):
        return {"name": name, "op": "gated", "B": B, "T": T, "d": d, "f": f, "dtype": dtype,
                "act": act, "keep": keep, "dx": dx, "dw": dw}

    def pack(name, B, T, d, dtype):
        return {"name": name, "op": "pack", "B": B, "T": T, "d": d, "dtype": dtype}

    def project(name, B, T, d, d_out, r):
        return {"name": name, "op": "project", "B": B, "T": T, "d": d, "d_out": d_out, "r": r,
                "dtype": "fp32"}

    return [
        # the next token of 4 sequences being answered: the weights are read for 4 rows
        gated("gated_one_token", 4, 1, 2048, 8192, "bf16", "silu", "input", False, False),
        # the smallest training step (the 64-wide fp32 workload's B and T)
        gated("gated_tiny", 8, 16, 64, 256, "fp32", "silu", "input", True, True),
        # an ordinary training step of a decoder, its activations kept in 8 bits
        gated("gated_step", 16, 512, 2048, 8192, "bf16", "silu", "int8", True, True),
        # an ordinary training step of a small encoder, only its input kept
        gated("gated_encoder", 64, 256, 768, 2048, "bf16", "gelu", "input", True, True),
        # odd sizes, the block's weights frozen
        gated("gated_frozen_odd", 7, 333, 1002, 2675, "bf16", "gelu_tanh", "int8", True, False),
        # a small fp32 model
        gated("gated_fp32", 9, 111, 768, 2050, "fp32", "gelu", "input", True, True),
        # the largest: long samples, a wide model
        gated("gated_large", 4, 4096, 4096, 11008, "bf16", "silu", "input", True, True),
        # the hidden activations of an ordinary step
        pack("pack_step", 16, 512, 8192, "bf16"),
        # rows that are no multiple of a block, fp32
        pack("pack_odd", 7, 333, 1002, "fp32"),
        # the input of a wide layer, long samples
        pack("pack_large", 4, 4096, 11008, "bf16"),
        # the smallest step's layer
        project("project_tiny", 8, 16, 64, 64, 8),
        # an encoder's layer
        project("project_encoder", 32, 128, 768, 2048, 128),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):
        # any, or whole multiples of 64 as trained models have
        n = log(lo, hi)
        return max(64, n // 64 * 64) if rng.random() < 0.6 else n

    op = rng.choice(("gated", "gated", "pack", "project"))
    case = {"op": op, "B": log(1, 64)}
    case["T"] = log(1, 8192 // case["B"])
    case["dtype"] = "fp32" if op == "project" else rng.choice(("bf16", "bf16", "fp32"))
    if op == "project":
        case["d"], case["d_out"] = width(32, 2048), width(32, 2048)
        case["r"] = rng.choice((8, 16, 33, 64, 100, 128, 256))
        return case
    if op == "pack":
        case["d"] = width(32, 11008)
        return case
    fp32 = case["dtype"] == "fp32"
    case["d"] = width(32, 1024 if fp32 else 4096)
    case["f"] = width(32, 2730 if fp32 else 11008)
    case["act"] = rng.choice(("silu", "gelu", "gelu_tanh"))
    case["dx"] = rng.random() < 0.8
    case["dw"] = case["dx"] and rng.random() < 0.6
    # (a code of fp32 projections hangs on the last bits of their sums)
    case["keep"] = "input" if fp32 else rng.choice(("input", "int8"))
    return case


def _lengths(case):
    """Tokens of each sample that count; the rest of its T are padding. Up to
    a quarter of a sample, by a fixed rule on its index."""
    return [case["T"] - (i * 7919 + 13) % (case["T"] // 4 + 1) for i in range(case["B"])]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    B, T, d = case["B"], case["T"], case["d"]
    dt = DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    n_tok = torch.tensor(_lengths(case), device=dev)
    there = (torch.arange(T, device=dev)[None, :] < n_tok[:, None])[..., None]
    # normalised activations with a few wide channels, as trained models have
    wide = torch.exp(1.5 * (torch.rand(d, generator=g, device=dev) < 0.02) *
                     torch.rand(d, generator=g, device=dev))
    X = torch.where(there, randn(B, T, d) * wide, 0.0).to(dt)
    state = {"case": case, "X": X}
    if case["op"] == "gated":
        f = case["f"]
        state["W_in"] = (randn(d, 2 * f) / math.sqrt(d)).to(dt)
        state["W_out"] = (randn(f, d) / math.sqrt(f)).to(dt)
        if case["dx"]:
            state["dY"] = torch.where(there, randn(B, T, d) / math.sqrt(T * d), 0.0).to(dt)
    elif case["op"] == "project":
        d_out = case["d_out"]
        state["dY"] = torch.where(there, randn(B, T, d_out) / math.sqrt(T * d_out), 0.0).to(dt)
        state["key"] = 0x1234567 + 1000003 * int(seed)  # of the projection's random stream
    return state


def run(state):
    return (_run_own if own else _run_plain)(state)


# ------------------------------------------------------------- framework --

def _run_own(state):
    import dp_grape_projection_amd as dpg
    case, X = state["case"], state["X"]
    if case["op"] == "pack":
        return {"X": dpg.dpg_unpack_act(dpg.dpg_pack_act(X))}
    if case["op"] == "project":
        norm_sq = torch.zeros(case["B"], device="cuda")
        G_hat = dpg.dpg_project_layer_packed(dpg.dpg_pack_act(X), state["dY"], case["r"],
                                             state["key"], 3, 5, norm_sq)
        return {"G_hat": G_hat, "norm_sq": norm_sq}
    W_in, W_out, act = state["W_in"], state["W_out"], case["act"]
    int8 = case["keep"] == "int8" and case["dx"]
    Y, Z = dpg.dpg_gated(X, W_in, W_out, act=act, keep=int8)
    out = {"Y": Y}
    if case["dx"]:
        kept = dpg.dpg_pack_act(X) if int8 and case["dw"] else X
        g = dpg.dpg_gated_grad(state["dY"], kept, W_in, W_out, act=act, Z=Z,
                               need_dW=case["dw"])
        out["dX"] = g.dX
        if case["dw"]:
            out["dW_in"], out["dW_out"] = g.dW_in, g.dW_out
    return out


# ------------------------------------------------------------ plain form --

def _run_plain(state):
    op = state["case"]["op"]
    return (_plain_gated if op == "gated" else _plain_pack if op == "pack" else
            _plain_project)(state)


def _eight_bits(x):
    """The values that 8 bits keep of x [..., d] (32 bits): blocks of 32 channels
    share the step 2^(e - 6), 2^e the power of two at or below the block's largest
    magnitude (2^-120 at least); a value is the nearest multiple of the step, ties to
    even, of at most 127 steps."""
    d = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -d % 32)).unflatten(-1, (-1, 32))
    e = torch.frexp(b.abs().amax(-1, keepdim=True)).exponent - 1
    e = e.clamp(min=-120)
    q = torch.round(torch.ldexp(b, 6 - e)).clamp(-127, 127)
    return torch.ldexp(q, e - 6).flatten(-2)[..., :d]


def _plain_pack(state):
    X = state["X"]
    return {"X": _eight_bits(X.float()).to(X.dtype)}


def _act(x, kind):
    """act(x) and its derivative."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return x * s, s * (1.0 + x * (1.0 - s))
    if kind == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
        return x * cdf, cdf + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (
        1.0 + 3 * 0.044715 * x * x)


def _plain_gated(state):
    case = state["case"]
    f, dt = case["f"], DT[case["dtype"]]
    x, w_in, w_out = state["X"].float().flatten(0, 1), state["W_in"].float(), state["W_out"].float()
    g, u = (x @ w_in).split(f, dim=-1)
    shape = state["X"].shape
    out = {"Y": ((_act(g, case["act"])[0] * u) @ w_out).to(dt).view(shape)}
    if case["dx"]:
        if case["keep"] == "int8":
            g, u, x = _eight_bits(g), _eight_bits(u), _eight_bits(x)
        a, da = _act(g, case["act"])
        dy = state["dY"].float().flatten(0, 1)
        dh = dy @ w_out.t()
        dz = torch.cat([dh * u * da, dh * a], dim=-1)
        out["dX"] = (dz @ w_in.t()).to(dt).view(shape)
        if case["dw"]:
            out["dW_in"] = (x.t() @ dz).to(dt)
            out["dW_out"] = ((a * u).t() @ dy).to(dt)
    return out


def _normals(key, layer, step, n):
    """The framework's stream of n standard normals for the projection: Philox4x32-10
    (counter: element / 4, layer, step, 0) and Box-Muller, in 64 bits."""
    low = 0xFFFFFFFF

    def product(a, m):  # high and low word of a m, both below 2^32
        return (a * (m >> 16) + ((a * (m & 0xFFFF)) >> 16)) >> 16, (a * m) & low

    c0 = torch.arange((n + 3) // 4, device="cuda")
    c1, c2, c3 = torch.full_like(c0, layer), torch.full_like(c0, step), torch.zeros_like(c0)
    k0, k1 = key & low, key >> 32
    for _ in range(10):
        h0, l0 = product(c0, 0xD2511F53)
        h1, l1 = product(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    u = (torch.stack([c0, c1, c2, c3], 1) >> 9).double().mul_(2).add_(1).mul_(2.0 ** -24)
    radius = torch.sqrt(-2.0 * torch.log(u[:, 0::2]))
    angle = 2.0 * math.pi * u[:, 1::2]
    z = torch.stack([radius * torch.cos(angle), radius * torch.sin(angle)], -1)
    return z.flatten()[:n]


def _plain_project(state):
    case = state["case"]
    r, d = case["r"], case["d"]
    P = (_normals(state["key"], 5, 3, r * d) / math.sqrt(r)).float().view(r, d)
    Q = _eight_bits(state["X"]) @ P.t()                                  # [B, T, r]
    G_hat = torch.bmm(Q.transpose(1, 2).contiguous(), state["dY"])       # [B, r, d_out]
    return {"G_hat": G_hat, "norm_sq": G_hat.square().sum((1, 2))}


# ----------------------------------------------------------------- 64 bits --

def _kept_in_8_bits(x):
    rows, d = x.shape
    n = -(-d // 32)
    full = x.new_zeros((rows, n * 32))
    full[:, :d] = x
    blocks = full.view(rows, n, 32)
    top = blocks.abs().max(dim=2, keepdim=True).values.clamp(min=2.0 ** -120)
    step = torch.exp2(torch.floor(torch.log2(top)) - 6)
    return (torch.clamp(torch.round(blocks / step), -127, 127) * step).view(rows, -1)[:, :d]


def _stream64(key, layer, step, n):
    u64, low = np.uint64, np.uint64(0xFFFFFFFF)
    x = [np.arange((n + 3) // 4, dtype=u64)] + [
        np.full((n + 3) // 4, v, dtype=u64) for v in (layer, step, 0)]
    k = [key & 0xFFFFFFFF, key >> 32]
    for _ in range(10):
        p, q = x[0] * u64(0xD2511F53), x[2] * u64(0xCD9E8D57)
        x = [(q >> u64(32)) ^ x[1] ^ u64(k[0]), q & low, (p >> u64(32)) ^ x[3] ^ u64(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    u = [(2.0 * (w >> u64(9)).astype(np.float64) + 1.0) / 2.0 ** 24 for w in x]
    out = np.empty((u[0].size, 4))
    for i in (0, 2):
        size = np.sqrt(-2.0 * np.log(u[i]))
        out[:, i] = size * np.cos(2.0 * np.pi * u[i + 1])
        out[:, i + 1] = size * np.sin(2.0 * np.pi * u[i + 1])
    return out.ravel()[:n]


def exact(case, seed):
    st = prepare(case, seed)
    B, T, d = case["B"], case["T"], case["d"]
    x = st["X"].double().reshape(B * T, d)
    if case["op"] == "pack":
        return {"X": _kept_in_8_bits(x).reshape(B, T, d)}
    if case["op"] == "project":
        r = case["r"]
        P = torch.from_numpy(_stream64(st["key"], 5, 3, r * d)).cuda().reshape(r, d) / math.sqrt(r)
        A = _kept_in_8_bits(x).reshape(B, T, d)
        G = torch.stack([torch.mm(torch.mm(P, A[i].t()), st["dY"][i].double()) for i in range(B)])
        return {"G_hat": G, "norm_sq": torch.linalg.vector_norm(G, dim=(1, 2)) ** 2}
    f, kind = case["f"], case["act"]
    w_gate, w_up = st["W_in"][:, :f].double(), st["W_in"][:, f:].double()
    w_out = st["W_out"].double()

    def value(v):
        if kind == "silu":
            return v * torch.sigmoid(v)
        if kind == "gelu":
            return v * torch.special.ndtr(v)
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))

    def slope(v):
        if kind == "silu":
            s = torch.sigmoid(v)
            return s + v * s * torch.sigmoid(-v)
        if kind == "gelu":
            return torch.special.ndtr(v) + v * torch.exp(-v ** 2 / 2) / math.sqrt(2 * math.pi)
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = torch.sigmoid(c * (v + 0.044715 * v ** 3))
        return s + v * s * (1.0 - s) * c * (1.0 + 3 * 0.044715 * v ** 2)

    gate, up = torch.mm(x, w_gate), torch.mm(x, w_up)
    out = {"Y": torch.mm(value(gate) * up, w_out).reshape(B, T, d)}
    if not case["dx"]:
        return out
    if case["keep"] == "int8":
        gate, up, x = (_kept_in_8_bits(v) for v in (gate, up, x))
    dy = st["dY"].double().reshape(B * T, d)
    dh = torch.mm(dy, w_out.t())
    dgate, dup = dh * up * slope(gate), dh * value(gate)
    del dh
    out["dX"] = (torch.mm(dgate, w_gate.t()) + torch.mm(dup, w_up.t())).reshape(B, T, d)
    if case["dw"]:
        out["dW_in"] = torch.cat([torch.mm(x.t(), dgate), torch.mm(x.t(), dup)], dim=1)
        out["dW_out"] = torch.mm((value(gate) * up).t(), dy)
    return out


def work(case):
    """Every input read once, every output written once, and the 8-bit form written and
    read where it is what the calls pass on. The block's products: three of [N][d][f]
    forwards, three for dX, three for the weights' gradients."""
    B, T, d = case["B"], case["T"], case["d"]
    N, size = B * T, SIZE[case["dtype"]]
    packed = N * (32 * -(-d // 32) + -(-d // 32))
    if case["op"] == "pack":
        return {"bytes": 2 * N * d * size + 2 * packed, "flops": 3 * N * d}
    if case["op"] == "project":
        r, d_out = case["r"], case["d_out"]
        return {"bytes": N * (d + d_out) * size + 2 * packed + 4 * B * r * d_out + 4 * B,
                "flops": 2 * N * r * (d + d_out) + 2 * B * r * d_out}
    f = case["f"]
    products = 3 + 3 * int(case["dx"]) + 3 * int(case["dw"])
    nbytes = (2 * N * d + 3 * d * f) * size
    nbytes += 2 * N * d * size if case["dx"] else 0
    nbytes += 3 * d * f * size if case["dw"] else 0
    return {"bytes": nbytes, "flops": 2 * products * N * d * f}
