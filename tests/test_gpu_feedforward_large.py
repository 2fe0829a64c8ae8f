"""Feed-forward operators where offsets pass 32 bits: rows at the end against calls of those
rows alone."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GiB")
    import dp_grape_projection_amd as dpg
    dpg.load_library()     # fails loudly when libdpg.so is missing
    yield
    torch.cuda.empty_cache()


def _fro(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_pack_and_unpack():
    """5 GB of rows, and 2^31 pieces of eight channels, which take a second launch."""
    import torch
    import dp_grape_projection_amd as dpg
    for N, d in ((300001, 8200), ((1 << 24) + 5, 1020)):
        print(f"[large] pack {N} x {d}", flush=True)
        X = torch.empty(N, d, dtype=torch.bfloat16, device="cuda")
        tail = torch.randn(1000, d, device="cuda").bfloat16()
        X[:1000] = tail.flip(0)
        X[1000:-1000] = 1.5
        X[-1000:] = tail
        p = dpg.dpg_pack_act(X)
        want = dpg.dpg_pack_act(tail)
        assert torch.equal(p.codes[-1000:], want.codes) and torch.equal(p.exps[-1000:], want.exps)
        back = dpg.dpg_unpack_act(p, X=X)
        assert torch.equal(back[-1000:], dpg.dpg_unpack_act(want))
        assert torch.equal(back[:1000], dpg.dpg_unpack_act(want).flip(0))
        assert torch.equal(back[N // 2], torch.full_like(back[0], 1.5))
        del X, p, back


@pytest.mark.parametrize("keep", [False, True])
def test_block(keep):
    """17 GB of dZ, 9 of H. Up to the rows' own sums everything is the same to the bit; Y
    and dX may be split over f differently, one rounding of the result apart."""
    import torch
    import dp_grape_projection_amd as dpg
    N, d, f, n = (1 << 18) + 3, 64, 16384, 300
    print(f"[large] block {N} x {d} x {f}, keep {keep}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    X, dY = (torch.randn(N, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    W_in = (torch.randn(d, 2 * f, generator=g, device="cuda") / 8).bfloat16()
    W_out = (torch.randn(f, d, generator=g, device="cuda") / 128).bfloat16()
    Y, Z = dpg.dpg_gated(X, W_in, W_out, keep=keep)
    out = dpg.dpg_gated_grad(dY, X, W_in, W_out, Z=Z, need_layers=True)
    end, dend = X[-n:].contiguous(), dY[-n:].contiguous()
    y, z = dpg.dpg_gated(end, W_in, W_out, keep=keep)
    small = dpg.dpg_gated_grad(dend, end, W_in, W_out, Z=z, need_layers=True)
    if keep:
        assert torch.equal(Z.codes[-n:], z.codes) and torch.equal(Z.exps[-n:], z.exps)
    assert torch.equal(out.dZ[-n:], small.dZ) and torch.equal(out.H[-n:], small.H)
    assert _fro(Y[-n:], y) <= 2 ** -8 and _fro(out.dX[-n:], small.dX) <= 2 ** -8
    # the sums over all rows, from dZ and H as they were rounded, 2^14 rows at a time
    dW_in = torch.zeros(d, 2 * f, device="cuda")
    dW_out = torch.zeros(f, d, device="cuda")
    for i in range(0, N, 1 << 14):
        rows = slice(i, i + (1 << 14))
        dW_in += X[rows].float().t() @ out.dZ[rows].float()
        dW_out += out.H[rows].float().t() @ dY[rows].float()
    # (one rounding of the result, and two sums of 2^18 fp32 terms)
    assert _fro(out.dW_in, dW_in) <= 2 ** -8 and _fro(out.dW_out, dW_out) <= 2 ** -8


def test_projection():
    """Samples of 300000 tokens, 4.6 GB read back: the last one against itself alone. Either
    is within the fp32 bar of 1e-5 of the formula."""
    import torch
    import dp_grape_projection_amd as dpg
    B, T, d_in, d_out, r = 3, 300001, 2560, 24, 8
    print(f"[large] projection {B} x {T} x {d_in} x {d_out}, r {r}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    A = torch.randn(B, T, d_in, generator=g, device="cuda", dtype=torch.bfloat16)
    p = dpg.dpg_pack_act(A)
    del A
    dY = torch.randn(B, T, d_out, generator=g, device="cuda") / (T * d_out) ** 0.5
    n3, n1 = torch.zeros(B, device="cuda"), torch.zeros(1, device="cuda")
    G = dpg.dpg_project_layer_packed(p, dY, r, 1, 1, 1, n3)
    last = p._replace(codes=p.codes[2:].contiguous(), exps=p.exps[2:].contiguous())
    own = dpg.dpg_project_layer_packed(last, dY[2:].contiguous(), r, 1, 1, 1, n1)
    assert _fro(G[2:], own) <= 2e-5 and _fro(n3[2:], n1) <= 4e-5
