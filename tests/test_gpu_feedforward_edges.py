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
