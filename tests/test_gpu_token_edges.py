"""Edges of the token operators' arguments: widths and batches of zero."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dp_grape_projection_amd as dpg
    dpg.load_library()     # fails loudly when libdpg.so is missing


def test_losses_of_width_zero_are_refused():
    """Rows without columns have a loss (ln V) that no call computes: an error, not
    outputs that nothing was written to."""
    import torch
    import dp_grape_projection_amd as dpg
    X, E = torch.empty((4, 0), device="cuda"), torch.empty((9, 0), device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.zeros(4, device="cuda")
    with pytest.raises(dpg.DpgError):
        dpg.dpg_vocab_loss(X, E, ids)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_vocab_loss_grad(X, E, ids, f, f)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_distill_loss(X, E, ids.view(4, 1), f.view(4, 1))
    with pytest.raises(dpg.DpgError):
        dpg.dpg_distill_loss_grad(X, E, ids.view(4, 1), f.view(4, 1), f, f)
    loss, lse = dpg.dpg_vocab_loss(X[:0], E, ids[:0])
    assert loss.shape == lse.shape == (0,)


@pytest.mark.parametrize("B,T", [(0, 4), (3, 0), (0, 0)])
def test_an_empty_batch_adds_nothing(B, T):
    """As the lookup and the losses do, the norms and the gradient take a batch of no
    samples or of no tokens."""
    import torch
    import dp_grape_projection_amd as dpg
    ids = torch.empty((B, T), dtype=torch.int64, device="cuda")
    dY = torch.empty((B, T, 12), device="cuda")
    norm_sq = torch.arange(1.0, B + 1.0, device="cuda")
    assert dpg.dpg_embed_norms(ids, dY, 9, norm_sq) is norm_sq
    assert torch.equal(norm_sq, torch.arange(1.0, B + 1.0, device="cuda"))
    s = torch.ones(B, device="cuda")
    dE = dpg.dpg_embed_grad(ids, dY, 9, sample_scales=s,
                            dE=torch.full((9, 12), float("nan"), device="cuda"))
    assert not dE.any()
    old = torch.randn(9, 12, device="cuda")
    kept = dpg.dpg_embed_grad(ids, dY, 9, dE=old.clone(), accumulate=True)
    assert torch.equal(kept, old)
    with pytest.raises(ValueError):
        dpg.dpg_embed_grad(ids, dY, 9, dE=old[:, :8].contiguous())
