"""The feed-forward operators' calls that the documentation allows, or refuses, beside the
ordinary ones."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dp_grape_projection_amd as dpg
    dpg.load_library()     # fails loudly when libdpg.so is missing


def test_projections_of_another_type_are_not_overwritten():
    """What is returned says which type its values had: an earlier result of fp32 rows is
    refused for bf16 ones, as dpg_pack_act refuses it, and stays as it was."""
    import torch
    import dp_grape_projection_amd as dpg
    X, W_in, W_out = (torch.randn(s, device="cuda") for s in ((6, 16), (16, 48), (24, 16)))
    _, Z = dpg.dpg_gated(X, W_in, W_out, keep=True)
    codes = Z.codes.clone()
    half = [t.bfloat16() for t in (X, W_in, W_out)]
    with pytest.raises(TypeError, match="Z is of"):
        dpg.dpg_gated(*half, keep=True, Z=Z)
    assert torch.equal(Z.codes, codes)
    _, again = dpg.dpg_gated(X, W_in, W_out, keep=True, Z=Z)
    assert again is Z and torch.equal(Z.codes, codes)


def test_projection_of_more_rows_than_the_16_bit_products_index():
    """fp32, 107 million tokens: A is read back and taken as dpg_project_layer takes it.
    Every sample against the formula; products and sums in fp32, the step's fp32 bar."""
    import torch
    import oracle
    import dp_grape_projection_amd as dpg
    from _helpers import TOL, rel_err
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GiB")
    B, T, d = 105000, 1024, 8
    assert B * T * (d // 8 + 9) >= 1 << 30     # (below, the other path)
    print(f"[edges] {B} x {T} x {d}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(6)
    codes = torch.randint(-127, 128, (B, T, 32), generator=g, device="cuda", dtype=torch.int8)
    exps = torch.randint(125, 129, (B, T, 1), generator=g, device="cuda", dtype=torch.uint8)
    dY = torch.randn(B, T, 1, generator=g, device="cuda") / T ** 0.5
    p = dpg.PackedActivations(codes, exps, d, torch.float32)
    n = torch.ones(B, device="cuda")
    G = dpg.dpg_project_layer_packed(p, dY, 1, 8, 2, 3, n)
    P = torch.from_numpy(oracle.projection_matrix(8, 3, 2, 1, d)).cuda()[0]
    want = torch.empty(B, dtype=torch.float64, device="cuda")
    scale = torch.empty_like(want)
    for i in range(0, B, 5000):
        s = slice(i, i + 5000)
        A = codes[s, :, :d].double() * torch.exp2(exps[s].double() - 133)
        terms = (A @ P) * dY[s, :, 0].double()
        want[s], scale[s] = terms.sum(1), terms.square().sum(1).sqrt()
    # (a sample's one sum may cancel: its error is that of its terms)
    assert float(((G[:, 0, 0].double() - want).abs() / scale).max()) <= TOL["fp32"]
    assert rel_err(n.double().cpu().numpy(), (1 + want.square()).cpu().numpy()) <= TOL["fp32"]


def test_a_gradient_that_needs_no_workspace_takes_none():
    """dZ, H and dX where no operand is copied and no sum is split: the query says 0 bytes,
    and the call takes a null pointer for them."""
    import ctypes
    import torch
    import dp_grape_projection_amd as dpg
    from dp_grape_projection_amd import binding as b
    N, d, f = 16384, 64, 512
    X, W_in, W_out, dY = (torch.randn(s, device="cuda").bfloat16()
                          for s in ((N, d), (d, 2 * f), (f, d), (N, d)))
    assert b._gated_grad_workspace_size(N, d, f, b.DPG_BF16, 1, 0, 1) == 0
    _, Z = dpg.dpg_gated(X, W_in, W_out, keep=True)
    want = dpg.dpg_gated_grad(dY, None, W_in, W_out, Z=Z, need_dW=False, need_layers=True)
    dX, dZ, H = (torch.full_like(t, float("nan")) for t in (want.dX, want.dZ, want.H))
    lib = dpg.load_library()
    status = lib.dpg_gated_grad(
        None, None, None, W_in.data_ptr(), W_out.data_ptr(), Z.codes.data_ptr(),
        Z.exps.data_ptr(), dY.data_ptr(), N, d, f, b.DPG_BF16, 0, dX.data_ptr(), None, None,
        dZ.data_ptr(), H.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    assert status == b.DPG_OK, lib.dpg_last_error()
    torch.cuda.synchronize()
    for got, ref in zip((dX, dZ, H), (want.dX, want.dZ, want.H)):
        assert torch.equal(got, ref)


def _products(a, b, rows=1 << 18):
    """a^T b in 64 bits, by pieces of their rows."""
    import torch
    out = torch.zeros(a.shape[1], b.shape[1], dtype=torch.float64, device="cuda")
    for i in range(0, a.shape[0], rows):
        out += a[i:i + rows].double().t().contiguous() @ b[i:i + rows].double()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,d,f", [(1 << 22, 64, 40), (20, 1 << 16, 64), (20, 64, 1 << 16),
                                   (3, 1 << 16, 96), (3, 96, 1 << 16)])
def test_block_at_its_limits(N, d, f, dtype):
    """The most rows, and the widest rows. bf16: two roundings of 2^-8 at most, independent, at
    most 0.82 of 2^-8 in the mean square. fp32: the fp32 bar, or what K terms of random
    signs summed one after the other may lose: six additions for every 32 of them, each off
    by one last place, 2^-23, of a partial sum, which is 2 / 3 sqrt(K) terms in the mean where
    the whole is sqrt(K): K / 8 2^-23. In S parts, should all be off the same way, each part's
    K / S terms lose (K / 8 S) 2^-23 sqrt(K / S), S of them together K / 8 2^-23 / sqrt(S) of
    the whole; the 2^22 rows are summed in 200 parts and more."""
    import torch
    import dp_grape_projection_amd as dpg
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    parts = 200 if N > 1 << 20 else 1
    bar = {"bf16": 2.0 ** -8, "fp32": max(1e-5, max(N, d, f) / 8 * 2.0 ** -23 / parts ** 0.5)}[dtype]
    print(f"[edges] block {N} x {d} x {f} {dtype}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(9)
    X, W_in, W_out, dY = (torch.randn(s, generator=g, device="cuda").div_(n ** 0.5).to(dt)
                          for s, n in (((N, d), 1), ((d, 2 * f), d), ((f, d), f), ((N, d), d)))
    Y, none = dpg.dpg_gated(X, W_in, W_out)
    out = dpg.dpg_gated_grad(dY, X, W_in, W_out, need_layers=True)
    wi, wo = W_in.double(), W_out.double()
    worst = {}

    def check(name, got, want):
        off = float((got.double() - want).norm() / want.norm())
        worst[name] = max(worst.get(name, 0.0), off)

    H, dZ = torch.empty(N, f, device="cuda"), torch.empty(N, 2 * f, device="cuda")
    for i in range(0, N, 1 << 18):
        r = slice(i, i + (1 << 18))
        G, U = (X[r].double() @ wi).chunk(2, 1)
        s = torch.sigmoid(G)
        h, dh = G * s * U, dY[r].double() @ wo.t().contiguous()
        dz = torch.cat([dh * U * s * (1 + G * (1 - s)), dh * G * s], 1)
        check("Y", Y[r], h @ wo)
        check("H", out.H[r], h)
        check("dZ", out.dZ[r], dz)
        check("dX", out.dX[r], dz @ wi.t().contiguous())
        H[r], dZ[r] = h.float(), dz.float()
    check("dW_in", out.dW_in, _products(X, dZ))
    check("dW_out", out.dW_out, _products(H, dY))
    assert max(worst.values()) <= bar, worst


@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_autograd_on_another_stream_and_captured(checkpoint):
    """Forward and backward pass of the torch function on a stream of their own, and in a
    graph that is replayed on new data between eager work. (Captured while no eager graph
    of the same leaves lives, as torch needs it.)"""
    import torch
    import dp_grape_projection_amd as dpg
    g = torch.Generator(device="cuda").manual_seed(12)
    X, W_in, W_out, dY = (torch.randn(s, generator=g, device="cuda").div_(8).bfloat16()
                          for s in ((5, 20, 64), (64, 192), (96, 64), (5, 20, 64)))
    leaves = [t.requires_grad_() for t in (X, W_in, W_out)]

    def step():
        Y = dpg.gated_feed_forward(*leaves, act="gelu", checkpoint=checkpoint)
        return [Y.detach(), *torch.autograd.grad(Y, leaves, dY)]

    want = step()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        other = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    del other
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    data = torch.randn(3, *X.shape, generator=g, device="cuda").bfloat16()
    for k in (0, 1, 2, 0):
        with torch.no_grad():
            X.copy_(data[k])
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), k
