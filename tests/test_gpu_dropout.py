"""GPU dropout against the oracle's generator: every value bit for bit (kept values are one fp32
product rounded once), alone, fused with an index map, and in the layer on every weight form."""
import numpy as np
import pytest

from oracle import poetx_ref as ref

from .gpu_harness import host, tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from orthogonal_reparameterized_cnp_b200 import poetx
    poetx.lib()
    return poetx


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _x(rows, cols, dt, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, cols, generator=g).to(dt).cuda()


def _expect(x, f):
    """x * f as the kernels round it: fp32 product, one rounding; a dropped value is +0."""
    import torch
    f32 = torch.from_numpy(f.astype(np.float32)).cuda()
    return torch.where(f32 > 0, x.float() * f32, torch.zeros_like(f32)).to(x.dtype)


def _same(a, b):
    import torch
    return torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32),
                       b.view(torch.int16 if b.element_size() == 2 else torch.int32))


SHAPES = [(1, 1), (1, 5), (3, 8), (7, 33), (2, 247), (2, 248), (2, 249), (5, 1000), (129, 2048),
          (33, 5003), (1, 65537), (1000, 3), (3, 16384)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dropout_matches_the_generator(P, dt, rows, cols):
    x = _x(rows, cols, _dt(dt), rows + cols)
    for p, seed, site, row0 in [(0.1, 3, 0, 0), (0.5, (7 << 40) | 11, 9, 4000000000)]:
        out = x.clone()
        P.dropout(P.dropout_desc(p, seed, site, row0), x, out)
        assert _same(out, _expect(x, ref.dropout_factor(rows, cols, p, seed, site, row0)))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_dropout_limits_in_place_and_tails(P, dt):
    import torch
    dtype = _dt(dt)
    x = _x(37, 1003, dtype)
    out = torch.empty_like(x)
    P.dropout(P.dropout_desc(0.0, 1), x, out)                    # nothing dropped
    assert _same(out, x)
    P.dropout(P.dropout_desc(65535 / 65536, 1), x, out)          # almost everything
    assert _same(out, _expect(x, ref.dropout_factor(37, 1003, 65535 / 65536, 1)))
    y = x.clone()
    P.dropout(P.dropout_desc(0.3, 5), y, y)                      # in place
    assert _same(y, _expect(x, ref.dropout_factor(37, 1003, 0.3, 5)))
    # infinities and NaN in dropped places become 0; in kept places they stay
    f = ref.dropout_factor(4, 64, 0.5, 8)
    z = torch.full((4, 64), float("inf"), device="cuda", dtype=dtype)
    z[1] = float("nan")
    o = torch.empty_like(z)
    P.dropout(P.dropout_desc(0.5, 8), z, o)
    o = o.float().cpu().numpy()
    assert np.all(o[f == 0] == 0) and np.all(~np.isfinite(o[f > 0]))
    # nothing is written behind the last row
    buf = torch.full((10 * 1003 + 64,), 7.0, device="cuda", dtype=dtype)
    P.dropout(P.dropout_desc(0.3, 5), x[:10].contiguous(), buf[:10 * 1003].view(10, 1003))
    assert torch.all(buf[10 * 1003:] == 7.0)


# narrow rows (interleaved gather), wide rows (row batches), odd widths (row in shared memory),
# rows beyond shared memory (direct)
GATHERS = [("bf16", 9, 256), ("bf16", 21, 2040), ("bf16", 17, 2048), ("bf16", 5, 13824),
           ("bf16", 6, 333), ("bf16", 2, 110000), ("bf16", 1, 8), ("f32", 9, 256),
           ("f32", 6, 5120), ("f32", 7, 1023), ("f32", 2, 60000), ("f32", 3, 20000),
          ("f32", 3, 14000), ("bf16", 3, 16384), ("bf16", 3, 16392), ("bf16", 3, 4101),
          ("f32", 1, 1)]


@pytest.mark.parametrize("dt,rows,cols", GATHERS)
def test_dropout_fused_with_an_index_map(P, dt, rows, cols):
    import torch
    x = _x(rows, cols, _dt(dt), cols)
    perm, inv = P.make_perm(cols, cols)
    pd, idv = tensor(perm, torch.int32), tensor(inv, torch.int32)
    p, seed, site, row0 = 0.2, 99, 2, 12345
    d = P.dropout_desc(p, seed, site, row0)
    f = ref.dropout_factor(rows, cols, p, seed, site, row0)
    out = torch.full_like(x, 3.0)
    P.permute_cols_dropout(d, x, out, pd)
    assert _same(out, _expect(x, f)[:, pd.long()])
    # the same as the two calls one after the other
    tmp, two = torch.empty_like(x), torch.empty_like(x)
    P.dropout(d, x, tmp)
    P.permute_cols(tmp, two, pd)
    assert _same(out, two)
    # the gradient of that map: inverse map, then the mask of the output column
    dx = torch.full_like(x, 3.0)
    P.permute_cols_dropout(d, out, dx, idv, mask_output=True)
    assert _same(dx, _expect(out[:, idv.long()], f))


def test_mask_of_a_shard_is_the_shard_of_the_mask(P):
    import torch
    x = _x(100, 520, torch.float32)
    full = torch.empty_like(x)
    P.dropout(P.dropout_desc(0.4, 21, row0=50), x, full)
    part = torch.empty_like(x[33:])
    P.dropout(P.dropout_desc(0.4, 21, row0=83), x[33:].contiguous(), part)
    assert _same(part, full[33:].contiguous())


def test_step_counter_in_a_replayed_graph_and_on_another_stream(P):
    import torch
    x = _x(64, 2050, torch.float32)
    step = torch.full((1,), (5 << 32) | 40, dtype=torch.int64, device="cuda")
    drop = P.Dropout(0.25, 17, site=1, step=step)
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    P.dropout(drop.desc(), x, out, s)
    torch.cuda.synchronize()
    assert _same(out, _expect(x, ref.dropout_factor(64, 2050, 0.25, 17, 1, 0, 40)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.dropout(drop.desc(), x, out)
        drop.advance()
    for k in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert _same(out, _expect(x, ref.dropout_factor(64, 2050, 0.25, 17, 1, 0, 40 + k)))
    assert int(step) == (5 << 32) | 43


def test_python_refusals_of_shapes_types_and_devices(P):
    import torch
    x = _x(4, 16, torch.float32)
    d = P.dropout_desc(0.1, 1)
    with pytest.raises(ValueError):
        P.dropout(d, x, torch.empty(4, 15, device="cuda"))
    with pytest.raises(ValueError):
        P.dropout(d, x, torch.empty(4, 16, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        P.dropout(d, x, torch.empty(4, 16))
    with pytest.raises(ValueError):
        P.dropout(d, x.t(), torch.empty(16, 4, device="cuda"))     # not contiguous
    with pytest.raises(ValueError):
        P.permute_cols_dropout(d, x, torch.empty_like(x), torch.zeros(16, device="cuda").long())
    with pytest.raises(ValueError):
        P.dropout_desc(0.1, 1, step=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        P.dropout(d, x.half(), torch.empty_like(x).half())


# ------------------------------------------------------------------------ in the layer
def _layer(P, kind, T, n, m, b, drop, save=True, seed=0):
    import torch
    rng = np.random.default_rng(seed + n + m)
    act = torch.float32 if kind == "f32" else torch.bfloat16
    W0 = tensor(rng.standard_normal((m, n)) / np.sqrt(n), act)
    tri = b * (b - 1) // 2
    th = [tensor(rng.standard_normal((k // b, tri)) * 0.01, torch.float32) for k in (n, m)]
    pP, _ = P.make_perm(seed + 1, n)
    pR, _ = P.make_perm(seed + 2, m)
    L = P.PoetxLinear(W0, th[0], th[1], pP, pR, b, 4, T, save_activations=save,
                      int8_weight=kind == "q8", int4_group=64 if kind == "q4" else 0, dropout=drop)
    L.cnp_forward()
    return L, tensor(rng.standard_normal((T, n)), act), tensor(rng.standard_normal((T, m)), act)


def _run(L, x, dy):
    import torch
    y = torch.empty(x.shape[0], L.m, dtype=x.dtype, device="cuda")
    dx = torch.empty_like(x)
    L.forward(x, y)
    L.backward(x, dy, dx)
    return y, dx, L.dG.clone()


@pytest.mark.parametrize("kind,T,n,m,b", [("f32", 70, 128, 96, 32), ("bf16", 300, 512, 256, 128),
                                          ("q8", 300, 512, 512, 256), ("q4", 300, 256, 512, 128),
                                          ("q4", 20, 512, 256, 128), ("bf16", 1, 256, 256, 128),
                                          ("q4", 3, 256, 512, 128)])
def test_layer_with_dropout_is_the_layer_of_dropped_inputs(P, kind, T, n, m, b):
    """y, dG of the layer with dropout are those of the layer without it on dropout(x), and dx is
    the mask applied to its dx, bit for bit; saved and recomputed activations agree."""
    import torch
    drop = P.Dropout(0.2, 5, site=4, row0=1000)
    L, x, dy = _layer(P, kind, T, n, m, b, drop)
    y, dx, dG = _run(L, x, dy)
    xd = torch.empty_like(x)
    P.dropout(drop.desc(), x, xd)
    L.training = False
    if kind == "q4" and T <= 64:  # without dropout few tokens take other kernels: same values
        y0, dx0, dG0 = _run(L, xd, dy)
        assert float((y.float() - y0.float()).abs().max()) <= 2e-2 * float(y0.float().abs().max())
    else:
        y0, dx0, dG0 = _run(L, xd, dy)
        assert _same(y, y0)
        assert torch.equal(dG, dG0)
        masked = torch.empty_like(dx0)
        P.dropout(drop.desc(), dx0, masked)
        assert _same(dx, masked)
    M, _, _ = _layer(P, kind, T, n, m, b, drop, save=False)
    ym, dxm, dGm = _run(M, x, dy)
    assert _same(ym, y) and _same(dxm, dx) and torch.equal(dGm, dG)
    assert P.device_status() == P.POETX_OK


def test_layer_with_dropout_gradients_by_differences(P):
    """fp32 layer: y is linear in x and in each G, so a finite difference along any direction is
    exact up to rounding: <dy, y(x + e) - y(x)> = <dx, e>, and the same for G_P and G_R.  The two
    sides are sums of about 10^4 products of fp32 results; 1e-4 of the sum of their magnitudes
    is above 10^2 roundings (2^-24 each) of every term."""
    import torch
    drop = P.Dropout(0.3, 6)
    T, n, m, b = 48, 128, 160, 32
    L, x, dy = _layer(P, "f32", T, n, m, b, drop)
    y, dx, dG = _run(L, x, dy)
    g = torch.Generator().manual_seed(1)
    for what in ("x", "G"):
        e = torch.randn(x.shape if what == "x" else L.G.shape, generator=g).cuda()
        x2 = x + e if what == "x" else x
        if what == "G":
            L.G += e
        y2 = torch.empty_like(y)
        L.forward(x2, y2)
        if what == "G":  # bilinear in (G_P, G_R): one side at a time
            L.G -= e
            G0 = L.G.clone()
            for side in (slice(0, L.nP), slice(L.nP, None)):
                L.G.copy_(G0)
                L.G[side] += e[side]
                L.forward(x, y2)
                lhs = (dy.double() * (y2.double() - y.double()))
                rhs = (dG[side].double() * e[side].double())
                assert abs(lhs.sum() - rhs.sum()) <= 1e-4 * (lhs.abs().sum() + rhs.abs().sum())
            L.G.copy_(G0)
        else:
            lhs = (dy.double() * (y2.double() - y.double()))
            rhs = (dx.double() * e.double())
            assert abs(lhs.sum() - rhs.sum()) <= 1e-4 * (lhs.abs().sum() + rhs.abs().sum())


def test_step_moves_the_mask_and_evaluation_has_none(P):
    import torch
    drop = P.Dropout(0.5, 6, site=2)
    L, x, dy = _layer(P, "bf16", 64, 256, 256, 128, drop)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    ys = []
    for _ in range(2):
        L.step(x, dy, y, dx)
        ys.append(y.clone())
    assert int(drop.step) == 2 and not _same(ys[0], ys[1])
    L.training = False
    L.step(x, dy, y, dx)
    plain = P.PoetxLinear(L.W0, L.theta[:L.nP], L.theta[L.nP:], L.perm_P.cpu().numpy(),
                          L.perm_R.cpu().numpy(), 128, 4, 64)
    y0, dx0 = torch.empty_like(y), torch.empty_like(dx)
    plain.step(x, dy, y0, dx0)
    assert int(drop.step) == 2 and _same(y, y0) and _same(dx, dx0)


def test_group_gives_each_linear_its_own_site_and_one_counter(P):
    import torch
    rng = np.random.default_rng(0)
    T, n, b = 40, 256, 128
    th = [tensor(rng.standard_normal((2, b * (b - 1) // 2)) * 0.01, torch.float32)
          for _ in range(2)]
    pP, _ = P.make_perm(1, n)
    W0 = tensor(rng.standard_normal((n, n)) / 16, torch.bfloat16)
    drop = P.Dropout(0.5, 3, site=10)
    G = P.PoetxLinearGroup([(W0, th[0], th[1], pP, pP)] * 2, b, 4, T, int4_group=128, dropout=drop)
    x = tensor(rng.standard_normal((T, n)), torch.bfloat16)
    ys = [torch.empty_like(x) for _ in range(2)]
    dxs = [torch.empty_like(x) for _ in range(2)]
    G.step([x, x], [x, x], ys, dxs)
    assert int(drop.step) == 1 and not _same(ys[0], ys[1])
    for i, L in enumerate(G.layers):
        f = ref.dropout_factor(T, n, 0.5, 3, 10 + i, 0, 0)
        assert _same(L.U, _expect(x, f)[:, L.perm_P.long()])
    G.train(False)
    G.step([x, x], [x, x], ys, dxs)
    assert int(drop.step) == 1 and _same(ys[0], ys[1])


def test_step_counter_moved_by_the_launch_just_before(P):
    """The kernels read the counter when they run, behind the launch that moved it."""
    import torch
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    d = P.dropout_desc(0.5, 99, 3, 0, step)
    x = torch.ones(64, 512, dtype=torch.bfloat16, device="cuda")
    idx = torch.arange(512, dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(x) for _ in range(60)]
    for o in outs[:30]:
        P.permute_cols_dropout(d, x, o, idx)
        step.add_(1)
    torch.cuda.synchronize()
    step.zero_()
    for o in outs[30:]:
        P.dropout(d, x, o)
        step.add_(1)
        torch.cuda.synchronize()
    for a, b in zip(outs[:30], outs[30:]):
        assert torch.equal(a, b)
    assert not torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("T,n,m,b", [(1, 256, 512, 128), (3, 256, 512, 128), (20, 512, 256, 128),
                                     (64, 512, 512, 256)])
def test_gradients_of_a_few_tokens_with_dropout(P, T, n, m, b):
    """Few tokens on a 4-bit weight: other kernels run the forward without dropout than with it, but
    dx and dG_P depend on dy, G, the weight, U and the mask alone, so they are those of the layer
    without dropout on dropout(x) bit for bit, dx through the mask.  dG_R = dZ^T W, whose W comes
    from the two forwards: each stores it rounded to bf16, one (above 4 tokens both) from a V
    rounded to bf16."""
    import torch
    drop = P.Dropout(0.2, 5, site=4, row0=1000)
    L, x, dy = _layer(P, "q4", T, n, m, b, drop)
    _, dx, dG = _run(L, x, dy)
    W = L.Wsave.float()
    xd = torch.empty_like(x)
    P.dropout(drop.desc(), x, xd)
    L.training = False
    _, dx0, dG0 = _run(L, xd, dy)
    masked = torch.empty_like(dx0)
    P.dropout(drop.desc(), dx0, masked)
    assert _same(dx, masked) and bool((masked == 0).any())
    assert torch.equal(dG[: L.nP], dG0[: L.nP]) and bool((dG[: L.nP] != 0).any())
    # dG_R from each stored W: exact products, fp32 sums on the tensor cores (one truncation every 16
    # products and as many as 64 in the joins)
    dZ = dy[:, L.perm_R.long()].double().view(T, -1, b)
    for got, Ws in ((dG, W), (dG0, L.Wsave.float())):
        Wb = Ws.double().view(T, -1, b)
        want, mag = (torch.einsum("tji,tjk->jik", u, v) for u, v in ((dZ, Wb),
                                                                     (dZ.abs(), Wb.abs())))
        assert bool(((got[L.nP:].double() - want).abs() <= (T / 16 + 64) * 2.0 ** -23 * mag).all())
    # the two W: up to four bf16 roundings (V and W, twice), 0.0017 of the value each in the root
    # mean square; 2^-7 is more than twice their sum in squares
    assert float((W - L.Wsave.float()).norm()) <= 2.0 ** -7 * float(W.norm())
    assert P.device_status() == P.POETX_OK
