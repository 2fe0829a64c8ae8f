"""How exact the token operators are where a row's own factor, or a long sum,
decides: the gradients of bf16 losses under per-sample factors, against float64.

A bf16 value is off by at most 2^-8 of itself, values of spread size by 1.6e-3 of
their norm. dX carries that once for its own rounding. D = p - q is rounded too: a
row's target entry, -(1 - p) with p of some 1 / V here, by at most p, the entries p
by 1.6e-3 of a part that is small where p is spread thin. So dX is within 2.0e-3 of
its norm, and its size along the exact gradient, where independent roundings average
to nothing, within 2^-10 (p, 3e-4 on average, is the rest). A factor of the row
that is rounded with D shows at up to 2^-8 in both. dE takes the factor with the rows
of X, whose roundings are nearly independent of each other: its size along the exact
gradient is held to 2^-10 as well."""
import math

import numpy as np
import pytest

from oracle import tokens as ot

pytestmark = pytest.mark.gpu

V, D, T = 3001, 192, 64
SIZE_BAR, DX_BAR = 2.0 ** -10, 2.0e-3


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dp_grape_projection_amd as dpg
    dpg.load_library()     # fails loudly when libdpg.so is missing


def _bf16(a):
    import torch
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().cuda()


def _size(got, want):
    """How large `got` is along `want`, minus one."""
    return float((got * want).sum() / (want * want).sum()) - 1.0


# factors of a whole sample: half a bf16 step off a bf16 value, on either side, and
# others as a mean over a sample's tokens with a clip factor gives them
FACTORS = [1.0 + 0.98 * 2.0 ** -8, 1.4140625 + 0.98 * 2.0 ** -8, 0.37 / 61, 1.0 / 57,
           1.0 / 511, 0.0, -3.0 / 4, 1.0 / 128]


@pytest.mark.parametrize("which", ["vocab", "distill k 1", "distill k 9"])
def test_a_samples_factor_is_no_common_error(which):
    import torch
    import dp_grape_projection_amd as dpg
    r = np.random.default_rng(31)
    N = T * len(FACTORS)
    x = _bf16(r.standard_normal((N, D)))
    e = _bf16(r.standard_normal((V, D)) / math.sqrt(D))
    X, E = (a.double().cpu().numpy() for a in (x, e))
    k = 9 if which.endswith("9") else 1
    ids = np.stack([r.permutation(V)[:k] for _ in range(N)])
    t = (r.standard_normal((N, k)) * 2.0).astype(np.float32)
    g = np.repeat(np.float32(FACTORS), T)
    q = ot.teacher_weights(ids, t, V, 1.0) if k > 1 else np.ones((N, 1))
    args = (torch.from_numpy(ids[:, 0]).cuda(),) if which == "vocab" else (
        torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda())
    fn, grad = ((dpg.dpg_vocab_loss, dpg.dpg_vocab_loss_grad) if which == "vocab" else
                (dpg.dpg_distill_loss, dpg.dpg_distill_loss_grad))
    lse = fn(x, e, *args)[1]
    for i, f in enumerate(FACTORS):
        rows = slice(i * T, (i + 1) * T)
        # the other samples have no factor: their part of dE is nothing
        w = np.zeros(N, np.float32)
        w[rows] = g[rows]
        dX, dE = (a.double().cpu().numpy() for a in grad(x, e, *args, lse, torch.from_numpy(w).cuda()))
        _, _, want_dX, want_dE = ot.target_loss(X[rows], E, ids[rows], q[rows], 1.0, 1.0, g[rows])
        if f == 0.0:
            assert not dX.any() and not dE.any()
            continue
        rel = np.linalg.norm(dX[rows] - want_dX) / np.linalg.norm(want_dX)
        sizes = _size(dX[rows], want_dX), _size(dE, want_dE)
        print(f"[precision] {which} factor {f:.6f}: dX {rel:.2e}, sizes {sizes[0]:+.1e} {sizes[1]:+.1e}",
              flush=True)
        assert abs(sizes[0]) <= SIZE_BAR, (f, sizes)
        assert abs(sizes[1]) <= SIZE_BAR, (f, sizes)
        if k == 1:
            assert rel <= DX_BAR, (f, rel)


# T, d, act: one token all along a sample (padding that is a token, say); rows of up to
# and of more than a block's 2048 columns, sorted samples and short ones
RUNS = [(2 ** 17, 1032, "bf16"), (2 ** 16, 2061, "fp32"), (2 ** 20, 24, "bf16"), (2 ** 20, 5, "fp32"),
        (1000, 2061, "bf16"), (700, 4104, "fp32"), (3000, 2056, "bf16")]


@pytest.mark.parametrize("T,d,act", RUNS)
def test_norms_of_a_token_repeated_all_along(T, d, act):
    """The sum of T equal rows of like sign, whose terms fall below the sum's last
    bits one by one. The bar is that of the other fp32 results, 1e-5: sums of at most
    64 terms in fp32, 64 * 2^-24, and what follows them in 64 bits."""
    import torch
    import dp_grape_projection_amd as dpg
    g = torch.Generator(device="cuda").manual_seed(41)
    x = torch.rand(d, generator=g, device="cuda") + 0.1
    x = x.bfloat16() if act == "bf16" else x
    B = 1 if T > 4096 else 2
    dY = x.expand(B, T, d).contiguous()
    ids = torch.full((B, T), 3, device="cuda")
    ids[-1, T // 3] = -1                           # two rows less
    ids[-1, T // 2] = 9
    norm_sq = torch.full((B,), 0.5, device="cuda")
    dpg.dpg_embed_norms(ids, dY, 9, norm_sq, scale=0.25)
    unit = float(x.double().square().sum()) * 0.0625
    for b in range(B):
        n = T - 2 if b == B - 1 else T
        want = 0.5 + unit * n * n
        err = abs(float(norm_sq[b]) / want - 1.0)
        print(f"[precision] norm of {n} rows of {d} {act}: {err:.1e}", flush=True)
        assert err <= 1e-5


def test_norms_of_many_tokens_of_equal_size():
    """A sample of 2^22 different tokens, whose squares are added up."""
    import torch
    import dp_grape_projection_amd as dpg
    T, d = 2 ** 22, 4
    x = torch.tensor([0.3, -0.7, 0.11, 0.9], device="cuda")
    ids = torch.arange(T, device="cuda").flip(0).view(1, T)
    norm_sq = torch.zeros(1, device="cuda")
    dpg.dpg_embed_norms(ids, x.expand(1, T, d).contiguous(), T, norm_sq)
    want = float(x.double().square().sum()) * T
    err = abs(float(norm_sq[0]) / want - 1.0)
    print(f"[precision] norms of {T} tokens: {err:.1e}", flush=True)
    assert err <= 1e-5


@pytest.mark.parametrize("which", ["vocab", "distill k 1", "distill k 5"])
@pytest.mark.parametrize("N", [1, 3, 12, 300])
def test_rows_whose_target_is_no_longer_unlikely(N, which):
    """Rows of which the model gives the target some percent to a half, so that -(1 - p) is
    no bf16 value, few enough that nothing averages out; the teacher is sure of its token.
    dX carries its own rounding, 1.65e-3, and D's of the part that p spreads: 1.8e-3. dE
    carries its own and that of X times the factor: 2.33e-3, and 2.5e-3 with that part."""
    import torch
    import dp_grape_projection_amd as dpg
    r = np.random.default_rng([61, N])
    V, d, k = 1000, 512, 5 if which.endswith("5") else 1
    E = r.standard_normal((V, d)) * 2 / math.sqrt(d)
    ids = np.stack([r.permutation(V)[:k] for _ in range(N)])
    x, e = _bf16(r.standard_normal((N, d)) + 1.5 * E[ids[:, 0]]), _bf16(E)
    X, E = (a.double().cpu().numpy() for a in (x, e))
    t = r.standard_normal((N, k)).astype(np.float32)
    t[:, 0] += 9.0
    g = (0.3 + r.random(N)).astype(np.float32) / 57
    y, tt, w = torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda(), torch.from_numpy(g).cuda()
    if which == "vocab":
        _, lse = dpg.dpg_vocab_loss(x, e, y[:, 0].contiguous())
        got = dpg.dpg_vocab_loss_grad(x, e, y[:, 0].contiguous(), lse, w)
    else:
        _, lse = dpg.dpg_distill_loss(x, e, y, tt)
        got = dpg.dpg_distill_loss_grad(x, e, y, tt, lse, w)
    q = ot.teacher_weights(ids, t, V, 1.0) if k > 1 else np.ones((N, 1))
    want = ot.target_loss(X, E, ids, q, 1.0, 1.0, g)[2:]
    rel = [np.linalg.norm(a.double().cpu().numpy() - b) / np.linalg.norm(b) for a, b in zip(got, want)]
    print(f"[precision] likely targets {which} N {N}: dX {rel[0]:.2e} dE {rel[1]:.2e}", flush=True)
    assert rel[0] <= 1.8e-3 and rel[1] <= 2.5e-3
