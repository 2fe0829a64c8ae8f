"""GPU parity of activations in 8 bits (dpg_pack_act, dpg_unpack_act) and of the
projection from them (dpg_project_layer_packed). Codes are whole numbers and what they
stand for is exact in either type: everything is compared for equality."""
import numpy as np
import pytest

from oracle import feedforward as of
import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dp_grape_projection_amd as dpg
    dpg.load_library()     # fails loudly when libdpg.so is missing


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _dev(a, dtype, offset=0):
    """A contiguous device copy; offset elements off an aligned start."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    flat = torch.empty(t.numel() + offset, dtype=_dtype(dtype), device="cuda")
    out = flat[offset:].view(t.shape)
    out.copy_(t)
    return out


def _rows(N, d, dtype, seed=0):
    """Rows of every scale, with zeros, subnormals, largest values, ties, infinities and
    NaN, as the values a tensor of `dtype` holds."""
    import torch
    r = np.random.default_rng([N, d, seed])
    x = r.standard_normal((N, d)) * np.exp(r.uniform(-80, 80, (N, 1)))
    x[r.random((N, d)) < 0.1] = 0.0
    if N > 8:
        x[1] = 0.0
        x[2] = 2.0 ** -133 * r.integers(-3, 4, d)
        x[3] = 3.3895314e38 * r.choice([-1, 1], d)
        x[4] = 0.25 * r.integers(-300, 300, d)
        x[5, ::37] = np.inf
        x[6, d // 2] = np.nan
        x[7, d - 1] = -np.inf
        x[8] = 1.0 + 2.0 ** -7 * r.integers(0, 128, d)   # the last half step below 2
    t = torch.from_numpy(x.astype(np.float32))
    return t.to(_dtype(dtype)).float().numpy()


SHAPES = [(1, 1), (1, 8), (3, 31), (9, 32), (17, 33), (64, 64), (33, 100), (300, 1002), (2, 8191),
          (11, 11008), (5000, 24)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,d", SHAPES)
def test_pack_and_unpack(N, d, dtype):
    import torch
    import dp_grape_projection_amd as dpg
    print(f"[act8] {N} x {d} {dtype}", flush=True)
    x = _rows(N, d, dtype)
    codes, exps = of.pack8(x)
    want = of.unpack8(codes, exps, d)
    for offset in (0, 1):
        p = dpg.dpg_pack_act(_dev(x, dtype, offset))
        np.testing.assert_array_equal(p.exps.cpu().numpy(), exps)
        np.testing.assert_array_equal(p.codes.cpu().numpy(), codes)
        assert p.dtype == _dtype(dtype) and tuple(p.shape) == (N, d)
        for out in ("bf16", "fp32"):
            X = _dev(np.zeros((N, d), np.float32), out, offset)
            assert dpg.dpg_unpack_act(p, X=X) is X
            np.testing.assert_array_equal(X.double().cpu().numpy(), want)
        back = dpg.dpg_unpack_act(p)
        assert back.dtype == _dtype(dtype)
        again = dpg.dpg_pack_act(_dev(x, dtype), out=p)
        assert again is p
        np.testing.assert_array_equal(p.codes.cpu().numpy(), codes)
        # what was read back is kept as it is
        fine = torch.from_numpy(np.isfinite(want).all(1)).cuda()
        twice = dpg.dpg_unpack_act(dpg.dpg_pack_act(back))
        assert torch.equal(twice[fine], back[fine])


def test_codes_at_unaligned_addresses_and_padding_left_out():
    """Codes and exponents anywhere; what pads the last block stands for nothing."""
    import torch
    import dp_grape_projection_amd as dpg
    x = _rows(20, 70, "bf16", 1)
    codes, exps = of.pack8(x)
    flat_c = torch.zeros(20 * 96 + 3, dtype=torch.int8, device="cuda")
    flat_e = torch.zeros(20 * 3 + 1, dtype=torch.uint8, device="cuda")
    p = dpg.PackedActivations(flat_c[3:].view(20, 96), flat_e[1:].view(20, 3), 70, torch.bfloat16)
    dpg.dpg_pack_act(_dev(x, "bf16"), out=p)
    np.testing.assert_array_equal(p.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(p.exps.cpu().numpy(), exps)
    p.codes[:, 70:] = 77
    np.testing.assert_array_equal(dpg.dpg_unpack_act(p).double().cpu().numpy(),
                                  of.unpack8(codes, exps, 70))


def test_leading_shapes_and_empty():
    import torch
    import dp_grape_projection_amd as dpg
    x = torch.randn(2, 3, 4, 40, device="cuda")
    p = dpg.dpg_pack_act(x)
    assert tuple(p.codes.shape) == (2, 3, 4, 64) and tuple(p.shape) == (2, 3, 4, 40)
    flat = dpg.dpg_pack_act(x.view(24, 40))
    assert torch.equal(p.codes.view(24, 64), flat.codes)
    e = dpg.dpg_pack_act(torch.empty(0, 5, device="cuda"))
    assert tuple(dpg.dpg_unpack_act(e).shape) == (0, 5)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_pack_act(torch.empty(3, 0, device="cuda"))


def test_refusals():
    import torch
    import dp_grape_projection_amd as dpg
    x = torch.randn(4, 64, device="cuda")
    p = dpg.dpg_pack_act(x)
    for bad, kind in ((x.half(), TypeError), (x.t(), ValueError), (x.cpu(), ValueError),
                      (torch.tensor(1.0, device="cuda"), ValueError)):
        with pytest.raises(kind):
            dpg.dpg_pack_act(bad)
    with pytest.raises(TypeError):
        dpg.dpg_pack_act(x.bfloat16(), out=p)
    with pytest.raises(ValueError):
        dpg.dpg_pack_act(x[:3].contiguous(), out=p)
    for bad in (p._replace(codes=p.codes[:, :32].contiguous()), p._replace(d=100),
                p._replace(exps=p.exps[:3].contiguous())):
        with pytest.raises(ValueError):
            dpg.dpg_unpack_act(bad)
    with pytest.raises(TypeError):
        dpg.dpg_unpack_act(p._replace(codes=p.codes.view(torch.uint8)))
    with pytest.raises(TypeError):
        dpg.dpg_unpack_act(p, dtype=torch.float16)


def test_another_stream_and_a_replayed_graph():
    import torch
    import dp_grape_projection_amd as dpg
    s = torch.cuda.Stream()
    a, b = _rows(50, 200, "bf16", 2), _rows(50, 200, "bf16", 3)
    x = _dev(a, "bf16")
    p = dpg.dpg_pack_act(x)
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        dpg.dpg_pack_act(x, out=p)
        dpg.dpg_unpack_act(p, X=y)
    for data in (a, b, a):
        x.copy_(torch.from_numpy(data))
        p.codes.zero_(), p.exps.zero_(), y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(y.double().cpu().numpy(), of.unpack8(*of.pack8(data), 200))
    with torch.cuda.stream(s):
        q = dpg.dpg_pack_act(x, stream=s)
    s.synchronize()
    np.testing.assert_array_equal(q.codes.cpu().numpy(), of.pack8(a)[0])


# B, T, d_in, d_out, r
LAYERS = [(1, 1, 8, 8, 1), (3, 5, 33, 17, 4), (2, 100, 70, 130, 33), (8, 16, 64, 64, 8),
          (4, 128, 256, 192, 128), (2, 256, 192, 320, 256), (5, 64, 1000, 40, 64),
          (1, 1000, 96, 256, 96)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,d_in,d_out,r", LAYERS)
def test_projection_from_8_bits(B, T, d_in, d_out, r, dtype):
    """Per-sample gradients at what the codes stand for, against the float64 formula.
    fp32: sums of fp32 products, 1e-5 (the fp32 bar of the step). bf16: P and A P^T are
    rounded to bf16, two independent roundings of at most 2^-8, which 2e-2 (the step's
    bf16 bar) covers for pieces of few elements too."""
    import torch
    import dp_grape_projection_amd as dpg
    from _helpers import TOL, rel_err
    print(f"[project] {B} {T} {d_in} {d_out} {r} {dtype}", flush=True)
    rng = np.random.default_rng([B, T, d_in, d_out, r])
    A = _dev(rng.standard_normal((B, T, d_in)), dtype)
    dY = _dev(rng.standard_normal((B, T, d_out)) / np.sqrt(T * d_out), dtype)
    p = dpg.dpg_pack_act(A)
    base = torch.linspace(0.5, 2.0, B, device="cuda")
    norm_sq = base.clone()
    G = dpg.dpg_project_layer_packed(p, dY, r, 77, 4, 9, norm_sq,
                                     G_hat=torch.full((B, r, d_out), float("nan"), device="cuda"))
    kept = of.unpack8(*(t.cpu().numpy().reshape(B * T, -1) for t in (p.codes, p.exps)),
                      d_in).reshape(B, T, d_in)
    P = oracle.projection_matrix(77, 9, 4, r, d_in)
    want = np.stack([(P @ kept[i].T) @ dY[i].double().cpu().numpy() for i in range(B)])
    assert rel_err(G.double().cpu().numpy(), want) <= TOL[dtype]
    n = base.double().cpu().numpy() + np.sum(want ** 2, axis=(1, 2))
    assert rel_err(norm_sq.double().cpu().numpy(), n) <= TOL[dtype]
    again = base.clone()
    assert torch.equal(G, dpg.dpg_project_layer_packed(p, dY, r, 77, 4, 9, again))
    assert torch.equal(norm_sq, again)


# more tokens than tiny tiles are for; a d_in that is split, at an odd count of tokens; long
# samples, whose tokens are summed in parts
MORE_LAYERS = [(16, 1024, 100, 33, 321), (3, 37, 1000, 65, 33), (1, 1, 2000, 40, 16), (7, 3, 400, 9, 70),
               (1, 5003, 40, 130, 5), (2, 2501, 64, 7, 3), (5, 65, 33, 257, 129), (1, 2049, 8, 300, 300)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,d_in,d_out,r", MORE_LAYERS)
def test_projection_in_a_used_workspace(B, T, d_in, d_out, r, dtype):
    """Whatever the workspace held, in a graph that is replayed, on another stream: the
    projection of what the codes stand for, within each type's bar (see above)."""
    import torch
    import dp_grape_projection_amd as dpg
    from _helpers import TOL, rel_err
    print(f"[project] {B} {T} {d_in} {d_out} {r} {dtype}", flush=True)
    rng = np.random.default_rng([B, T, d_in, d_out, r, 1])
    A = _dev(rng.standard_normal((B, T, d_in)), dtype)
    dY = _dev(rng.standard_normal((B, T, d_out)) / np.sqrt(T * d_out), dtype)
    p = dpg.dpg_pack_act(A)
    ws = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")     # all NaN
    norm_sq = torch.zeros(B, device="cuda")
    G = dpg.dpg_project_layer_packed(p, dY, r, 5, 2, 3, norm_sq, workspace=ws)
    P = oracle.projection_matrix(5, 3, 2, r, d_in)
    kept = dpg.dpg_unpack_act(p, dtype=torch.float32).double().cpu().numpy()
    want = np.stack([(P @ kept[i].T) @ dY[i].double().cpu().numpy() for i in range(B)])
    assert rel_err(G.double().cpu().numpy(), want) <= TOL[dtype]
    assert rel_err(norm_sq.double().cpu().numpy(), np.sum(want ** 2, axis=(1, 2))) <= TOL[dtype]
    s = torch.cuda.Stream()
    got, n = torch.empty_like(G), torch.zeros_like(norm_sq)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        dpg.dpg_project_layer_packed(p, dY, r, 5, 2, 3, n, G_hat=got, workspace=ws)
    for _ in range(3):
        ws.fill_(0xFF), got.fill_(float("nan")), n.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, G) and torch.equal(n, norm_sq)
    n.zero_()
    torch.cuda.synchronize()
    other = dpg.dpg_project_layer_packed(p, dY, r, 5, 2, 3, n, stream=s)
    s.synchronize()
    assert torch.equal(other, G) and torch.equal(n, norm_sq)


def test_packed_projection_refuses():
    import torch
    import dp_grape_projection_amd as dpg
    p = dpg.dpg_pack_act(torch.randn(2, 3, 8, device="cuda"))
    dY, n = torch.randn(2, 3, 4, device="cuda"), torch.zeros(2, device="cuda")
    with pytest.raises(ValueError):
        dpg.dpg_project_layer_packed(p, dY[:, :2].contiguous(), 4, 0, 1, 0, n)
    with pytest.raises(ValueError):
        dpg.dpg_project_layer_packed(p, dY, 4, 0, 1, 0, n[:1])
    with pytest.raises(TypeError):
        dpg.dpg_project_layer_packed(torch.zeros(2, 3, 8, device="cuda"), dY, 4, 0, 1, 0, n)
    with pytest.raises(TypeError):
        dpg.dpg_project_layer_packed(p, dY.half(), 4, 0, 1, 0, n)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_project_layer_packed(p, dY, 0, 0, 1, 0, n)
