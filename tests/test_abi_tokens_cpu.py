"""The token operators of the C ABI on the host (no GPU): invalid arguments
are refused before HIP is touched, and workspace queries are sane."""
import ctypes
import os

import pytest

import dp_grape_projection_amd as dpg

INVALID, WORKSPACE = dpg.binding.DPG_ERR_INVALID_ARG, dpg.binding.DPG_ERR_WORKSPACE
P = 0x10000                                  # a 256-byte aligned stand-in pointer


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dpg.library_path()):
        pytest.skip("libdpg.so not built")
    return dpg.load_library()


def _call(fn, names, defaults, kw):
    args = dict(defaults, **kw)
    return fn(*[args[n] for n in names])


EMBED_NAMES = "ids n E V d table scale dtype Y stream".split()
EMBED = dict(ids=P, n=4, E=P, V=9, d=8, table=0, scale=1.0, dtype=0, Y=P, stream=None)
BAD_EMBED = [dict(n=0), dict(n=2 ** 23 + 1), dict(V=0), dict(V=2 ** 23 + 1), dict(d=0),
             dict(d=2 ** 20 + 1), dict(table=5), dict(dtype=-1), dict(table=1, dtype=0),
             dict(scale=float("nan")), dict(scale=float("inf")), dict(ids=None), dict(E=None),
             dict(Y=None)]


@pytest.mark.parametrize("kw", BAD_EMBED, ids=str)
def test_embed_refuses(lib, kw):
    assert _call(lib.dpg_embed, EMBED_NAMES, EMBED, kw) == INVALID
    assert lib.dpg_last_error() != b""


NORM_NAMES = "ids dY B T V d dtype scale norm_sq ws n stream".split()
GRAD_NAMES = "ids dY B T V d dtype scale s table acc dE ws n stream".split()
BATCH = dict(ids=P, dY=P, B=2, T=3, V=9, d=8, dtype=0, scale=1.0, norm_sq=P, s=None, table=0,
             acc=0, dE=P, ws=P, n=1 << 30, stream=None)
BAD_BATCH = [dict(B=0), dict(T=0), dict(B=2 ** 22, T=3), dict(V=0), dict(d=0), dict(dtype=2),
             dict(scale=float("inf")), dict(ids=None), dict(dY=None)]


@pytest.mark.parametrize("kw", BAD_BATCH + [dict(norm_sq=None)], ids=str)
def test_embed_norms_refuses(lib, kw):
    assert _call(lib.dpg_embed_norms, NORM_NAMES, BATCH, kw) == INVALID


@pytest.mark.parametrize("kw", BAD_BATCH + [dict(dE=None), dict(table=3), dict(table=1, dtype=0)],
                         ids=str)
def test_embed_grad_refuses(lib, kw):
    assert _call(lib.dpg_embed_grad, GRAD_NAMES, BATCH, kw) == INVALID


def test_embed_workspace(lib):
    need = ctypes.c_size_t(0)
    assert lib.dpg_embed_workspace_size(2, 3, 9, 8, ctypes.byref(need)) == 0
    assert need.value > 0 and need.value % 256 == 0
    assert lib.dpg_embed_workspace_size(2, 3, 9, 8, None) == INVALID
    for fn, names in ((lib.dpg_embed_norms, NORM_NAMES), (lib.dpg_embed_grad, GRAD_NAMES)):
        assert _call(fn, names, BATCH, dict(n=need.value - 1)) == WORKSPACE
        assert _call(fn, names, BATCH, dict(ws=None)) == WORKSPACE
        assert _call(fn, names, BATCH, dict(ws=P + 16)) == WORKSPACE
        assert b"workspace" in lib.dpg_last_error()


LOSS_NAMES = "X E ids N d V dtype scale loss lse ws n stream".split()
LGRAD_NAMES = "X E ids lse dloss N d V dtype scale dX dE ws n stream".split()
DLOSS_NAMES = "X E ids t N d V k dtype scale tau loss lse ws n stream".split()
DGRAD_NAMES = "X E ids t lse dloss N d V k dtype scale tau dX dE ws n stream".split()
LOSS = dict(X=P, E=P, ids=P, t=P, N=4, d=8, V=9, k=3, dtype=1, scale=1.0, tau=1.0, loss=P, lse=P,
            dloss=P, dX=P, dE=P, ws=P, n=1 << 40, stream=None)
BAD_LOSS = [dict(N=0), dict(N=2 ** 22 + 1), dict(d=0), dict(d=2 ** 16 + 1), dict(V=0),
            dict(V=2 ** 22 + 1), dict(dtype=2), dict(scale=float("nan")), dict(X=None),
            dict(E=None), dict(ids=None), dict(lse=None)]
BAD_TOP = [dict(k=0), dict(k=1025), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("inf")),
           dict(t=None)]


@pytest.mark.parametrize("kw", BAD_LOSS + [dict(loss=None)], ids=str)
def test_losses_refuse(lib, kw):
    assert _call(lib.dpg_vocab_loss, LOSS_NAMES, LOSS, kw) == INVALID
    assert _call(lib.dpg_distill_loss, DLOSS_NAMES, LOSS, kw) == INVALID


@pytest.mark.parametrize("kw", BAD_LOSS + [dict(dloss=None), dict(dX=None, dE=None)], ids=str)
def test_loss_gradients_refuse(lib, kw):
    assert _call(lib.dpg_vocab_loss_grad, LGRAD_NAMES, LOSS, kw) == INVALID
    assert _call(lib.dpg_distill_loss_grad, DGRAD_NAMES, LOSS, kw) == INVALID


@pytest.mark.parametrize("kw", BAD_TOP, ids=str)
def test_distillation_refuses(lib, kw):
    assert _call(lib.dpg_distill_loss, DLOSS_NAMES, LOSS, kw) == INVALID
    assert _call(lib.dpg_distill_loss_grad, DGRAD_NAMES, LOSS, kw) == INVALID


def test_loss_workspace(lib):
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert lib.dpg_vocab_loss_workspace_size(4, 8, 9, 1, 0, ctypes.byref(a)) == 0
    assert lib.dpg_vocab_loss_workspace_size(4, 8, 9, 1, 1, ctypes.byref(b)) == 0
    assert 0 < a.value < b.value and b.value % 256 == 0
    assert _call(lib.dpg_vocab_loss, LOSS_NAMES, LOSS, dict(n=a.value - 1)) == WORKSPACE
    assert _call(lib.dpg_vocab_loss_grad, LGRAD_NAMES, LOSS, dict(n=b.value - 1)) == WORKSPACE
    assert _call(lib.dpg_vocab_loss, LOSS_NAMES, LOSS, dict(ws=P + 16)) == WORKSPACE
    assert lib.dpg_distill_loss_workspace_size(4, 8, 9, 3, 1, 1, ctypes.byref(b)) == 0
    assert _call(lib.dpg_distill_loss_grad, DGRAD_NAMES, LOSS, dict(n=b.value - 1)) == WORKSPACE
    assert lib.dpg_vocab_loss_workspace_size(4, 8, 9, 1, 0, None) == INVALID
    assert lib.dpg_distill_loss_workspace_size(4, 8, 9, 3, 1, 1, None) == INVALID


def test_a_piece_of_the_gradient_bounds_the_workspace(lib):
    """The gradient keeps one piece of [N][V], not all of it: N = 65536 rows
    against 128000 columns would be 16.8 GB in bf16."""
    need = ctypes.c_size_t(0)
    assert lib.dpg_vocab_loss_workspace_size(65536, 64, 128000, 1, 1, ctypes.byref(need)) == 0
    assert need.value < 1 << 30
