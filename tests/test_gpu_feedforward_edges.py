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
