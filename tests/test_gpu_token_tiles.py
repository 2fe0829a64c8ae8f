"""The losses and their gradients at shapes that reach every tile size, in each
operand type and with teacher ids, for several steps of every product's sum, and that
carry their state from one piece of the vocabulary to the next. Against float64.

Bars: those of the other loss tests for the largest piece of a row (fp32 1e-5, bf16
2^-7) and for loss and lse; and for a bf16 gradient as a whole the roundings that it
passes, of D, of X times its factor and of the result, 1.65e-3 of its norm each if
independent: 3e-3."""
import math

import pytest

pytestmark = pytest.mark.gpu

TOL = {"fp32": 1e-5, "bf16": 2.0 ** -7}
WHOLE = {"fp32": 1e-5, "bf16": 3e-3}


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dp_grape_projection_amd as dpg
    dpg.load_library()     # fails loudly when libdpg.so is missing


def _off_by_one(t):
    """t one element off an aligned start."""
    import torch
    return torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape).copy_(t)


def _errors(got, want, width=256):
    """The largest relative error of a row's pieces of `width` columns, and that of the
    whole (as tests/_helpers.rel_err, on the GPU)."""
    import torch
    got, worst = got.double(), 0.0
    n = want.shape[1]
    for c0 in range(0, n, width):
        c0 = min(c0, max(n - width, 0))
        w, g = want[:, c0:c0 + width], got[:, c0:c0 + width]
        den, num = w.norm(dim=1), (g - w).norm(dim=1)
        worst = max(worst, float(torch.where(den > 0, num / den, num).max()))
    return worst, float((got - want).norm() / want.norm())


# Columns after which a piece ends, at one of the shapes below or another.
ENDS = [10752, 32768, 65536, 174592, 262144, 349184, 349440]


def _case(N, d, V, k, act, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    X = torch.randn(N, d, generator=g, device="cuda").to(dt)
    E = (torch.randn(V, d, generator=g, device="cuda") * 2 / math.sqrt(d)).to(dt)
    ids = torch.randint(-V // 8, V, (N, max(k, 1)), generator=g, device="cuda")
    ends = [e for e in ENDS if e < V]
    for n in range(min(N, 4 * len(ends))):   # on both sides of a piece's end
        e = ends[n // 4]
        if k < 5:
            ids[n, 0] = min(e - 2 + n % 4, V - 1)
        else:                                # one of them twice
            ids[n, :5] = torch.tensor([e, e - 1, 1, min(e + 1, V - 1), e], device="cuda")
            ids[n] = ids[n].roll(n)
    ids[N // 2] = -1
    X[N // 2] = float("nan")                 # a row without target
    t = torch.randn(N, max(k, 1), generator=g, device="cuda") * 2
    w = torch.rand(N, generator=g, device="cuda") / 7
    return X, E, ids, t, w


def _reference(X, E, ids, t, w, k, scale, tau):
    import torch
    valid = ids >= 0
    on = valid.any(1)
    Xd, Ed = torch.where(on[:, None], X, 0.0).double(), E.double()
    z = Xd @ Ed.t() * (scale / tau)
    q = valid.double() if k == 0 else torch.where(
        valid, t.double() / tau, -math.inf).softmax(1).nan_to_num(0.0)
    at = ids.clamp(min=0)
    lse = torch.logsumexp(z, 1)
    loss = tau ** 2 * (torch.xlogy(q, q).sum(1) - (q * z.gather(1, at)).sum(1) + lse) * on
    D = z.sub_(lse[:, None]).exp_().scatter_add_(1, at, -q)
    D *= (w.double() * scale * tau * on)[:, None]
    return loss, lse * on, D @ Ed, D.t() @ Xd


def _check(N, d, V, k, act):
    import torch
    import dp_grape_projection_amd as dpg
    X, E, ids, t, w = _case(N, d, V, k, act, 51)
    scale, tau = (0.9, 1.0) if k == 0 else (1.1, 2.0)
    want = _reference(X, E, ids, t, w, k, scale, tau)
    bar = 2e-5 * max(1.0, float(want[1].abs().max())) * max(1.0, tau * tau)
    for e in (E, _off_by_one(E)):
        if k == 0:
            y = ids[:, 0].contiguous()
            loss, lse = dpg.dpg_vocab_loss(X, e, y, scale=scale)
            dX, dE = dpg.dpg_vocab_loss_grad(X, e, y, lse, w, scale=scale)
        else:
            args = dict(temperature=tau, scale=scale)
            loss, lse = dpg.dpg_distill_loss(X, e, ids, t, **args)
            dX, dE = dpg.dpg_distill_loss_grad(X, e, ids, t, lse, w, **args)
        for got, ref in ((loss, want[0]), (lse, want[1])):
            assert float((got.double() - ref).abs().max()) <= bar
        for got, ref in ((dX, want[2]), (dE, want[3])):
            assert torch.isfinite(got).all()
            piece, whole = _errors(got, ref)
            print(f"[tiles] {N} x {d} x {V} k {k} {act}: {piece:.2e} {whole:.2e}", flush=True)
            assert piece <= TOL[act] and whole <= WHOLE[act]


# N, d, V, k (0: cross entropy), act
TILES = [
    # logits in 128 x 128 tiles, four steps of 64
    (200, 200, 17003, 0, "bf16"), (200, 200, 17003, 9, "bf16"), (200, 202, 17003, 9, "bf16"),
    (200, 200, 17003, 9, "fp32"), (4, 328, 40003, 0, "bf16"),
    # logits in 256 x 256 tiles, five
    (1100, 264, 10003, 0, "bf16"), (1100, 264, 10003, 37, "bf16"), (1100, 264, 10003, 37, "fp32"),
    # dX and dE in 256 x 256 tiles as well
    (3000, 2100, 7000, 0, "bf16"), (2100, 1200, 9000, 9, "bf16"), (1030, 520, 24000, 5, "fp32"),
]


@pytest.mark.parametrize("N,d,V,k,act", TILES)
def test_every_tile(N, d, V, k, act):
    _check(N, d, V, k, act)


# The table one element off is packed 64 MiB at a time; the last shapes' own table is
# read as it is, and D (gradient) or the teacher's bits (both) bound the piece.
PIECES = [
    (10, 1000, 70000, 0, "bf16"), (10, 1000, 70000, 9, "bf16"), (1500, 1000, 40003, 9, "bf16"),
    (10, 1000, 30000, 9, "fp32"), (9, 24, 400003, 0, "fp32"), (9, 24, 400003, 5, "fp32"),
    (200, 64, 400003, 5, "bf16"),
]


@pytest.mark.parametrize("N,d,V,k,act", PIECES)
def test_pieces_of_the_vocabulary(N, d, V, k, act):
    _check(N, d, V, k, act)


# Either side of what few fp32 rows need for their table to be read as it is.
@pytest.mark.parametrize("N,d,V", [(128, 1024, 8192), (128, 1024, 8191), (129, 1024, 8192),
                                   (128, 1026, 8192)])
def test_where_few_fp32_rows_end(N, d, V):
    _check(N, d, V, 0, "fp32")
    _check(N, d, V, 6, "fp32")
