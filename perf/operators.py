"""The measured cases of the token operators that stand at the two ends of a
language model around the private update step:

  embed    token lookup with scaling, each sample's squared gradient norm of
           the table, and the table's gradient with per-sample clip factors
  vocab    softmax cross entropy of hidden states against a [V][d] table, in
           pieces of the vocabulary, with the gradients of both
  distill  the same product against a teacher's top-k logits per row

`run` computes a case in elementary torch operations in 32 bits, or, where
`own` is true, through dp_grape_projection_amd. B samples of T tokens; the
last tokens of a sample may be padding (id or target -1).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    def embed(name, B, T, d, V, table, act, grad):
        return {"name": name, "op": "embed", "B": B, "T": T, "d": d, "V": V,
                "table": table, "act": act, "grad": grad, "scale": math.sqrt(d)}

    def vocab(name, B, T, d, V, act, dx, de):
        return {"name": name, "op": "vocab", "B": B, "T": T, "d": d, "V": V,
                "act": act, "dx": dx, "de": de, "scale": 1.0}

    def distill(name, B, T, d, V, k, act, dx, de, temperature):
        return {"name": name, "op": "distill", "B": B, "T": T, "d": d, "V": V, "k": k,
                "act": act, "dx": dx, "de": de, "scale": 1.0, "temperature": temperature}

    return [
        # the next token of 16 sequences being answered: latency only
        embed("lookup_one_token", 16, 1, 2048, 50304, "bf16", "bf16", False),
        # the smallest training step (the 64-wide fp32 workload's B and T)
        embed("embed_tiny", 8, 16, 64, 1000, "fp32", "fp32", True),
        # an ordinary training step: fp32 master table, bf16 activations
        embed("embed_step", 16, 512, 2048, 50304, "fp32", "bf16", True),
        # odd width (rows not 16-byte aligned), odd batch and vocabulary
        embed("embed_odd", 7, 333, 1002, 32003, "bf16", "bf16", True),
        # scoring one token of 4 sequences: the table is read once for 4 rows
        vocab("loss_one_token", 4, 1, 2048, 50304, "bf16", False, False),
        # the smallest training step, fp32
        vocab("loss_tiny", 8, 16, 64, 1000, "fp32", True, True),
        # an ordinary training step, both gradients (a trained head)
        vocab("loss_step", 16, 512, 2048, 50304, "bf16", True, True),
        # an ordinary fp32 step at odd sizes, the head frozen
        vocab("loss_frozen_fp32", 9, 111, 768, 32003, "fp32", True, False),
        # the largest: long samples, a wide model, a large vocabulary
        vocab("loss_large", 4, 2048, 4096, 128000, "bf16", True, True),
        # a small fp32 student at odd sizes
        distill("distill_odd", 5, 37, 200, 5003, 7, "fp32", True, True, 2.0),
        # an ordinary distillation step, both gradients
        distill("distill_step", 32, 128, 2048, 50304, 64, "bf16", True, True, 2.0),
        # long samples, a wide model with its head frozen
        distill("distill_frozen", 4, 1024, 4096, 128000, 32, "bf16", True, False, 1.0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("embed", "vocab", "distill"))
    case = {"op": op, "B": log(1, 32)}
    case["T"] = log(1, 8192 // case["B"])
    # widths: any, or whole multiples of 64 as trained models have
    case["d"] = log(32, 4096)
    if rng.random() < 0.6:
        case["d"] = max(64, case["d"] // 64 * 64)
    case["V"] = log(500, 128000)
    case["act"] = rng.choice(("bf16", "bf16", "fp32"))
    if op == "embed":
        case["table"] = rng.choice(("bf16", "fp32")) if case["act"] == "bf16" else "fp32"
        case["grad"] = rng.random() < 0.75
        case["scale"] = math.sqrt(case["d"]) if rng.random() < 0.5 else 1.0
        return case
    step = rng.random() < 0.8
    if case["act"] == "fp32":  # fp32 products cost several bf16 ones
        case["d"] = min(case["d"], 1024)
    case["dx"] = step
    case["de"] = step and rng.random() < 0.6
    case["scale"] = rng.choice((1.0, 1.0, 0.5))
    if op == "distill":
        case["k"] = log(1, 100)
        case["temperature"] = rng.choice((1.0, 2.0, 4.0))
    return case


def _lengths(case):
    """Tokens of each sample that count; the rest of its T are padding. Up to
    a quarter of a sample, by a fixed rule on its index."""
    return [case["T"] - (i * 7919 + 13) % (case["T"] // 4 + 1) for i in range(case["B"])]


def _zipf(shape, V, g, dev):
    """Token ids whose frequency falls as 1 / rank, as in text."""
    u = torch.rand(shape, generator=g, device=dev, dtype=torch.float64)
    return (torch.exp(u * math.log(V + 1.0)).long() - 1).clamp_(0, V - 1)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    B, T, d, V = case["B"], case["T"], case["d"], case["V"]
    act = DT[case["act"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    n_tok = torch.tensor(_lengths(case), device=dev)
    pad = torch.arange(T, device=dev)[None, :] >= n_tok[:, None]
    ids = _zipf((B, T), V, g, dev).masked_fill_(pad, -1)
    state = {"case": case, "ids": ids}
    if case["op"] == "embed":
        state["E"] = (randn(V, d) / math.sqrt(d)).to(DT[case["table"]])
        if case["grad"]:
            state["dY"] = (randn(B, T, d) / math.sqrt(T * d)).to(act)
            # clip factors min(1, C / n_i): some samples clipped, some not
            state["clip"] = (0.3 + torch.rand(B, generator=g, device=dev)).clamp_(max=1.0)
        return state
    # logits with a standard deviation near 2, the target's raised by 4
    E = randn(V, d) * (2.0 / math.sqrt(d))
    X = randn(B, T, d) + E[ids.clamp(min=0)]
    state["E"], state["X"] = E.to(act), X.to(act)
    # each sample's mean loss, some samples clipped
    clip = (0.3 + torch.rand(B, generator=g, device=dev)).clamp_(max=1.0)
    state["dloss"] = (clip / n_tok)[:, None].expand(B, T).contiguous()
    if case["op"] == "distill":
        k = min(case["k"], V)
        stride = torch.randint(1, max(2, V // k), (B, T, 1), generator=g, device=dev)
        top = (ids[..., None] + stride * torch.arange(k, device=dev)) % V
        # one row in five keeps fewer than k entries of its teacher
        keep = torch.randint(1, k + 1, (B, T, 1), generator=g, device=dev)
        short = torch.rand((B, T, 1), generator=g, device=dev) < 0.2
        drop = short & (torch.arange(k, device=dev) >= keep)
        state["top_ids"] = top.masked_fill_(drop | pad[..., None], -1)
        t = randn(B, T, k) * 2.0 + 4.0
        state["top_logits"] = torch.sort(t, dim=-1, descending=True).values.contiguous()
    return state


def run(state):
    return (_run_own if own else _run_plain)(state)


# ------------------------------------------------------------- framework --

def _run_own(state):
    import dp_grape_projection_amd as dpg
    case = state["case"]
    if case["op"] == "embed":
        out = {"Y": dpg.dpg_embed(state["ids"], state["E"], scale=case["scale"],
                                  dtype=DT[case["act"]])}
        if case["grad"]:
            norm_sq = torch.zeros(case["B"], device="cuda")
            out["norm_sq"] = dpg.dpg_embed_norms(state["ids"], state["dY"], case["V"],
                                                 norm_sq, scale=case["scale"])
            out["dE"] = dpg.dpg_embed_grad(state["ids"], state["dY"], case["V"],
                                           scale=case["scale"], sample_scales=state["clip"],
                                           table_dtype=DT[case["table"]])
        return out
    X, E = state["X"], state["E"]
    out = {}
    if case["op"] == "vocab":
        out["loss"], out["lse"] = dpg.dpg_vocab_loss(X, E, state["ids"], scale=case["scale"])
        if case["dx"]:
            out["dX"], dE = dpg.dpg_vocab_loss_grad(
                X, E, state["ids"], out["lse"], state["dloss"], scale=case["scale"],
                need_dE=case["de"])
    else:
        out["loss"], out["lse"] = dpg.dpg_distill_loss(
            X, E, state["top_ids"], state["top_logits"], temperature=case["temperature"],
            scale=case["scale"])
        if case["dx"]:
            out["dX"], dE = dpg.dpg_distill_loss_grad(
                X, E, state["top_ids"], state["top_logits"], out["lse"], state["dloss"],
                temperature=case["temperature"], scale=case["scale"], need_dE=case["de"])
    if case["de"]:
        out["dE"] = dE
    return out


# ------------------------------------------------------------ plain form --

def _run_plain(state):
    return _plain_embed(state) if state["case"]["op"] == "embed" else _plain_loss(state)


def _plain_embed(state):
    case, E = state["case"], state["E"]
    B, T, d, V = case["B"], case["T"], case["d"], case["V"]
    ids = state["ids"].reshape(-1)
    ok = ids >= 0
    at = ids.clamp(min=0)
    rows = E[at].float() * case["scale"]
    out = {"Y": torch.where(ok[:, None], rows, 0.0).to(DT[case["act"]]).view(B, T, d)}
    if not case["grad"]:
        return out
    f = torch.where(ok[:, None], state["dY"].reshape(-1, d).float() * case["scale"], 0.0)
    sample = torch.arange(B, device=ids.device).repeat_interleave(T)
    # squared norm per sample: the rows of one token of one sample are added
    # first; sorted (sample, token) keys, one group per change of key
    key, order = torch.sort(sample * (V + 1) + ids + 1, stable=True)
    new = torch.ones_like(key)
    new[1:] = (key[1:] != key[:-1]).long()
    group = torch.cumsum(new, 0) - 1
    sums = torch.zeros_like(f).index_add_(0, group, f[order])
    owner = torch.zeros_like(ids).index_put_((group,), sample[order])
    out["norm_sq"] = torch.zeros(B, device=ids.device).index_add_(
        0, owner, (sums * sums).sum(1))
    dE = torch.zeros((V, d), device=ids.device)
    dE.index_add_(0, at, f * state["clip"][sample][:, None])
    out["dE"] = dE.to(DT[case["table"]])
    return out


def _plain_loss(state):
    case = state["case"]
    B, T, d = case["B"], case["T"], case["d"]
    X = state["X"].reshape(-1, d).float()
    E = state["E"].float()
    tau = case.get("temperature", 1.0)
    z = (X @ E.t()) * (case["scale"] / tau)
    m = z.amax(1, keepdim=True)
    p = torch.exp(z - m)
    s = p.sum(1, keepdim=True)
    lse = m + torch.log(s)
    if case["op"] == "vocab":
        at = state["ids"].reshape(-1, 1)
        q = (at >= 0).float()
        teacher = torch.zeros_like(q)
    else:
        at = state["top_ids"].flatten(0, 1)
        t = (state["top_logits"].flatten(0, 1) / tau).masked_fill(at < 0, -math.inf)
        t = t - t.amax(1, keepdim=True).clamp(min=-1e30)
        e = torch.exp(t)
        total = e.sum(1, keepdim=True).clamp(min=1e-30)
        q = e / total
        teacher = torch.where(q > 0, t - torch.log(total), 0.0)
    on = q.sum(1) > 0
    at = at.clamp(min=0)
    loss = (tau * tau) * (q * (teacher - z.gather(1, at) + lse)).sum(1)
    out = {"loss": torch.where(on, loss, 0.0).view(B, T),
           "lse": torch.where(on, lse[:, 0], 0.0).view(B, T)}
    if case["dx"]:
        del z
        c = torch.where(on, state["dloss"].reshape(-1) * (tau * case["scale"]), 0.0)[:, None]
        p.mul_(c / s).scatter_add_(1, at, -c * q)
        out["dX"] = (p @ E).to(DT[case["act"]]).view(B, T, d)
        if case["de"]:
            out["dE"] = (p.t() @ X).to(DT[case["act"]])
    return out


# ----------------------------------------------------------------- 64 bits --

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    B, T, d, V = case["B"], case["T"], case["d"], case["V"]
    E = st["E"].to(f64)
    if case["op"] == "embed":
        Y = torch.zeros((B, T, d), dtype=f64, device="cuda")
        norm_sq = torch.zeros(B, dtype=f64, device="cuda")
        dE = torch.zeros((V, d), dtype=f64, device="cuda") if case["grad"] else None
        for b in range(B):
            there = torch.nonzero(st["ids"][b] >= 0)[:, 0]
            tok = st["ids"][b, there]
            Y[b, there] = case["scale"] * E[tok]
            if case["grad"]:
                kinds, which = torch.unique(tok, return_inverse=True)
                hot = torch.zeros((kinds.numel(), tok.numel()), dtype=f64, device="cuda")
                hot[which, torch.arange(tok.numel(), device="cuda")] = 1.0
                own_rows = hot @ (case["scale"] * st["dY"][b, there].to(f64))
                norm_sq[b] = own_rows.square().sum()
                dE[kinds] += st["clip"][b].to(f64) * own_rows
        return {"Y": Y, "norm_sq": norm_sq, "dE": dE} if case["grad"] else {"Y": Y}
    tau = case.get("temperature", 1.0)
    X = st["X"].reshape(-1, d).to(f64)
    N = B * T
    if case["op"] == "vocab":
        top = st["ids"].reshape(N, 1)
        t = torch.zeros((N, 1), dtype=f64, device="cuda")
    else:
        top = st["top_ids"].reshape(N, -1)
        t = st["top_logits"].reshape(N, -1).to(f64)
    g = st["dloss"].reshape(N).to(f64)
    loss = torch.zeros(N, dtype=f64, device="cuda")
    lse = torch.zeros(N, dtype=f64, device="cuda")
    dX = torch.zeros((N, d), dtype=f64, device="cuda")
    dE = torch.zeros((V, d), dtype=f64, device="cuda") if case["de"] else None
    for n0 in range(0, N, 1024):
        rows = torch.nonzero((top[n0:n0 + 1024] >= 0).any(1))[:, 0] + n0
        if not rows.numel():
            continue
        z = torch.mm(X[rows], E.t()) * case["scale"]
        logp = torch.log_softmax(z / tau, dim=1)
        valid = top[rows] >= 0
        logq = torch.log_softmax(torch.where(valid, t[rows] / tau, -math.inf), dim=1)
        q = torch.exp(logq)
        dist = torch.zeros_like(z).scatter_add_(1, top[rows].clamp(min=0), q)
        entropy = torch.where(valid, q * logq, 0.0).sum(1)
        loss[rows] = tau ** 2 * (entropy - (dist * logp).sum(1))
        lse[rows] = torch.logsumexp(z / tau, dim=1)
        if case["dx"]:
            D = (torch.exp(logp) - dist) * (g[rows] * tau * case["scale"])[:, None]
            dX[rows] = torch.mm(D, E)
            if case["de"]:
                dE += torch.mm(D.t(), X[rows])
    out = {"loss": loss.view(B, T), "lse": lse.view(B, T)}
    if case["dx"]:
        out["dX"] = dX.view(B, T, d)
        if case["de"]:
            out["dE"] = dE
    return out


def work(case):
    """Every input read once, every output written once. The losses: one
    product for the logits and one for each gradient, over the rows that
    have a target."""
    B, T, d, V = case["B"], case["T"], case["d"], case["V"]
    N, used = B * T, sum(_lengths(case))
    act = SIZE[case["act"]]
    if case["op"] == "embed":
        table = SIZE[case["table"]]
        nbytes = 8 * N + min(used, V) * d * table + N * d * act
        flops = used * d
        if case["grad"]:
            nbytes += used * d * act + V * d * table + 12 * B
            flops += 4 * used * d
        return {"bytes": nbytes, "flops": flops}
    k = min(case.get("k", 1), V)
    nbytes = (used + V) * d * act + N * k * (8 if case["op"] == "vocab" else 12) + 8 * N
    products = 1 + int(case["dx"]) + int(case["de"])
    nbytes += (N * d * act + 4 * N if case["dx"] else 0) + (V * d * act if case["de"] else 0)
    return {"bytes": nbytes, "flops": 2 * products * used * d * V}
