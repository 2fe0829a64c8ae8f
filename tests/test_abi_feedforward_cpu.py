"""The feed-forward operators of the C ABI on the host (no GPU): invalid arguments are
refused before HIP is touched, and workspace queries are sane."""
import ctypes
import os

import pytest
import torch

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
    return fn(*[args[n] for n in names.split()])


PACK = "X N d dtype codes exps stream"
UNPACK = "codes exps N d dtype X stream"
ACT = dict(X=P, N=4, d=8, dtype=1, codes=P, exps=P, stream=None)


@pytest.mark.parametrize("kw", [dict(N=0), dict(N=2 ** 30 + 1), dict(d=0), dict(d=2 ** 20 + 1),
                                dict(dtype=2), dict(X=None), dict(codes=None), dict(exps=None)],
                         ids=str)
def test_activations_refuse(lib, kw):
    assert _call(lib.dpg_pack_act, PACK, ACT, kw) == INVALID
    assert lib.dpg_last_error() != b""
    assert _call(lib.dpg_unpack_act, UNPACK, ACT, kw) == INVALID


GATED = "X W_in W_out N d f dtype act Y zc ze ws n stream"
GRAD = "X xc xe W_in W_out zc ze dY N d f dtype act dX dW_in dW_out dZ H ws n stream"
BLOCK = dict(X=P, W_in=P, W_out=P, N=4, d=8, f=16, dtype=1, act=0, Y=P, zc=P, ze=P, ws=P, n=1 << 40,
             stream=None, xc=None, xe=None, dY=P, dX=P, dW_in=P, dW_out=P, dZ=P, H=P)
BAD_BLOCK = [dict(N=0), dict(N=2 ** 22 + 1), dict(d=0), dict(d=2 ** 16 + 1), dict(f=0),
             dict(f=2 ** 16 + 1), dict(dtype=2), dict(act=3), dict(act=-1), dict(W_in=None),
             dict(W_out=None), dict(zc=None), dict(ze=None)]


@pytest.mark.parametrize("kw", BAD_BLOCK + [dict(X=None), dict(Y=None)], ids=str)
def test_block_refuses(lib, kw):
    assert _call(lib.dpg_gated, GATED, BLOCK, kw) == INVALID


@pytest.mark.parametrize("kw", BAD_BLOCK + [
    dict(dY=None), dict(xc=P), dict(xe=P), dict(xc=P, xe=P), dict(X=None),
    dict(zc=None, ze=None, X=None, dW_in=None),
    dict(dX=None, dW_in=None, dW_out=None, dZ=None, H=None)], ids=str)
def test_block_gradient_refuses(lib, kw):
    assert _call(lib.dpg_gated_grad, GRAD, BLOCK, kw) == INVALID


def test_block_workspace(lib):
    a, b, c, e = (ctypes.c_size_t(0) for _ in range(4))
    assert lib.dpg_gated_workspace_size(4, 8, 16, 1, 0, ctypes.byref(a)) == 0
    assert lib.dpg_gated_grad_workspace_size(4, 8, 16, 1, 1, 0, 1, 0, ctypes.byref(b)) == 0
    assert lib.dpg_gated_grad_workspace_size(4, 8, 16, 1, 1, 1, 1, 0, ctypes.byref(c)) == 0
    assert lib.dpg_gated_grad_workspace_size(4, 8, 16, 1, 0, 1, 1, 0, ctypes.byref(e)) == 0
    assert 0 < a.value and b.value < c.value < e.value
    assert all(x.value % 256 == 0 for x in (a, b, c, e))
    for kw in (dict(n=a.value - 1), dict(ws=None), dict(ws=P + 16)):
        assert _call(lib.dpg_gated, GATED, BLOCK, kw) == WORKSPACE
    for kw in (dict(n=c.value - 1), dict(zc=None, ze=None, n=e.value - 1), dict(ws=P + 16),
               dict(dW_in=None, dW_out=None, n=b.value - 1)):
        assert _call(lib.dpg_gated_grad, GRAD, BLOCK, kw) == WORKSPACE
    assert lib.dpg_gated_workspace_size(4, 8, 16, 1, 0, None) == INVALID
    assert lib.dpg_gated_workspace_size(4, 8, 16, 7, 0, ctypes.byref(a)) == INVALID
    assert lib.dpg_gated_grad_workspace_size(4, 8, 16, 1, 1, 1, 0, 0, None) == INVALID


def test_workspace_holds_copies_only_where_they_are_needed(lib):
    """Aligned bf16 operands of whole K steps are read where they are, and the private
    step's dZ and H are written where the caller has them."""
    def size(name, *args):
        need = ctypes.c_size_t(0)
        assert getattr(lib, name)(*args, ctypes.byref(need)) == 0
        return need.value
    N, d, f = 4096, 1024, 4096
    operands = 2 * (N * d + 3 * d * f)
    forward = size("dpg_gated_workspace_size", N, d, f, 1, 0)
    assert 2 * N * f <= forward < 2 * N * f + (1 << 20)
    assert size("dpg_gated_workspace_size", N, d, f, 1, 1) >= forward + operands
    assert size("dpg_gated_workspace_size", N, d, f, 0, 0) >= 3 * operands
    args = (N, d, f, 1, 1, 0)
    made = size("dpg_gated_grad_workspace_size", *args, 0, 0)
    assert made >= 6 * N * f
    assert size("dpg_gated_grad_workspace_size", *args, 1, 0) <= made - 6 * N * f
    assert size("dpg_gated_grad_workspace_size", *args, 1, 1) >= made + operands


@pytest.mark.parametrize("N", [128, 192, 320])
def test_rows_are_padded_to_whole_steps_alone(lib, N):
    """dZ and H of the workspace, which the caller's own take the place of: tiles of rows
    beyond them would be computed like any other."""
    d, f, need = 64, 8192, []
    for layers in (0, 1):
        n = ctypes.c_size_t(0)
        assert lib.dpg_gated_grad_workspace_size(N, d, f, 1, 1, 0, layers, 0, ctypes.byref(n)) == 0
        need.append(n.value)
    assert need[0] - need[1] == 2 * N * 3 * f


@pytest.mark.parametrize("dtype", [0, 1])
def test_no_room_for_8_bits_of_what_cannot_be_in_8_bits(lib, dtype):
    """Projections computed again need X as it is: nothing of it is read back, and with
    tiles enough not to split a sum the weights' gradients need no workspace."""
    need = []
    for weights in (0, 1):
        n = ctypes.c_size_t(0)
        assert lib.dpg_gated_grad_workspace_size(16384, 4096, 11008, dtype, 0, weights, 0, 0,
                                                 ctypes.byref(n)) == 0
        need.append(n.value)
    assert need[0] == need[1]


def test_projections_computed_again_take_a_bounded_workspace(lib):
    """G and U in fp32 would be 2^20 x 2 x 4096 x 4 bytes, 34 GB, at once."""
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert lib.dpg_gated_grad_workspace_size(2 ** 20, 64, 4096, 1, 1, 0, 0, 0, ctypes.byref(a)) == 0
    assert lib.dpg_gated_grad_workspace_size(2 ** 20, 64, 4096, 1, 0, 0, 0, 0, ctypes.byref(b)) == 0
    assert b.value - a.value <= 1 << 30


PROJ = "layer codes exps B T r dtype seed proj_step G norm_sq ws n stream"


def _layer(**kw):
    arr = (dpg.LayerGrad * 1)()
    arr[0].d_in, arr[0].d_out, arr[0].layer_id, arr[0].dY = 8, 12, 3, P
    for k, v in kw.items():
        setattr(arr[0], k, v)
    return arr


PACKED = dict(layer=_layer(), codes=P, exps=P, B=2, T=5, r=4, dtype=0, seed=1, proj_step=1, G=P,
              norm_sq=P, ws=P, n=1 << 30, stream=None)


@pytest.mark.parametrize("kw", [dict(layer=None), dict(codes=None), dict(exps=None), dict(B=0),
                                dict(T=0), dict(r=0), dict(dtype=3), dict(proj_step=2 ** 32),
                                dict(G=None), dict(norm_sq=None), dict(layer=_layer(dY=None)),
                                dict(layer=_layer(d_in=0)), dict(layer=_layer(reserved=1))],
                         ids=lambda kw: next(iter(kw)))
def test_packed_projection_refuses(lib, kw):
    assert _call(lib.dpg_project_layer_packed, PROJ, PACKED, kw) == INVALID


def test_packed_projection_workspace(lib):
    plain, packed = ctypes.c_size_t(0), ctypes.c_size_t(0)
    size = (_layer(), 2, 5, 4, 0)
    assert lib.dpg_project_layer_workspace_size(*size, ctypes.byref(plain)) == 0
    assert lib.dpg_project_layer_packed_workspace_size(*size, ctypes.byref(packed)) == 0
    assert plain.value <= packed.value
    for kw in (dict(n=packed.value - 1), dict(ws=None), dict(ws=P + 16)):
        assert _call(lib.dpg_project_layer_packed, PROJ, PACKED, kw) == WORKSPACE
    assert lib.dpg_project_layer_packed_workspace_size(*size, None) == INVALID


def test_wrappers_refuse_on_the_host():
    """What the Python layer refuses before it needs a GPU."""
    X, W_in, W_out = torch.zeros(2, 4), torch.zeros(4, 12), torch.zeros(6, 4)
    with pytest.raises(ValueError, match="on the GPU"):
        dpg.dpg_gated(X, W_in, W_out)
    with pytest.raises(ValueError, match="on the GPU"):
        dpg.dpg_pack_act(X)
    with pytest.raises(TypeError, match="PackedActivations"):
        dpg.dpg_unpack_act(X)
    with pytest.raises(ValueError, match="checkpoint"):
        dpg.gated_feed_forward(X, W_in, W_out, checkpoint="fp8")
    with pytest.raises(ValueError, match="checkpoint"):
        dpg.GatedFeedForward(4, 6, (0, 1), checkpoint="int4", device="cpu")
    with pytest.raises(ValueError, match="act"):
        dpg.GatedFeedForward(4, 6, (0, 1), act="relu", device="cpu")
    layer = dpg.ProjectedLinear(4, 6, 0, device="cpu")
    with pytest.raises(ValueError, match="checkpoint"):
        dpg.GrapeOptimizer([layer], r=2, clip_C=1.0, sigma=0.0, seed=0, lr=0.1, checkpoint="int4")
    block = dpg.GatedFeedForward(4, 6, (0, 1), device="cpu")
    dpg.GrapeOptimizer([block.up], r=2, clip_C=1.0, sigma=0.0, seed=0, lr=0.1)
    with pytest.raises(RuntimeError, match="both"):
        block(torch.zeros(1, 2, 4))


def test_packed_shapes():
    p = dpg.PackedActivations(torch.zeros(3, 5, 64, dtype=torch.int8),
                              torch.zeros(3, 5, 2, dtype=torch.uint8), 40, torch.bfloat16)
    assert tuple(p.shape) == (3, 5, 40) and p.nbytes == 3 * 5 * 66
