"""GPU parity of the 4-bit merged weight: codes and scales bit for bit with the oracle's
quantiser, the products with it against float64, and the layer on it against the oracle's layer
on the dequantised weight.

Bound of a product: the result is rounded once to bf16 (half a step, 2^-8 of its magnitude), and
the fp32 sums of K products add at most (K / 16 + 64) roundings of 2^-23 (the tensor cores may
truncate) of the sum of the magnitudes: 16 products a matrix instruction, then at most 64 partial
sums."""
import numpy as np
import pytest

from oracle import poetx_ref as ref
from poetx_inputs import LayerShape, layer_inputs, round_to_bf16

from .gpu_harness import host, norm_max_err, tensor

pytestmark = pytest.mark.gpu

BF16_NORM = 2e-2  # the layer's bar (four stored intermediates of half a step each)


@pytest.fixture(scope="module")
def P():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from orthogonal_reparameterized_cnp_b200 import poetx
    poetx.lib()
    return poetx


def _buffers(P, m, n, group, fill=0):
    import torch
    qs, ss = P.q4_shapes(m, n, group)
    return (torch.full(qs, fill, dtype=torch.uint8, device="cuda"),
            torch.full(ss, float(fill), dtype=torch.bfloat16, device="cuda"))


def _same_scales(s, s_ref, group):
    a = s.float().cpu().numpy()
    return np.array_equal(a, ref.pack_scales(s_ref, group), equal_nan=True)


def _weights(m, n, dt, seed):
    rng = np.random.default_rng(seed)
    W = rng.standard_normal((m, n)) * rng.uniform(1e-3, 5.0, (m, 1))
    W[min(2, m - 1), :] = 0.0
    W[0, : n // 2] = 0.0
    return round_to_bf16(W) if dt == "bf16" else W.astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(1, 128), (7, 384), (300, 2176), (65, 13824), (5, 16384),
                                 (3, 16512), (2, 25600)])
def test_merge_and_read_back_bit_exact(P, m, n, dt, group):
    import torch
    act = torch.bfloat16 if dt == "bf16" else torch.float32
    W = _weights(m, n, dt, m * 7 + n)
    Wd = tensor(W, act)
    pR, _ = P.make_perm(m + 1, m)
    pP, _ = P.make_perm(n + 2, n)
    for perms in (False, True):
        q, s = _buffers(P, m, n, group, 255)
        if perms:
            P.merge_perm_q4(Wd, q, s, tensor(pR, torch.int32), tensor(pP, torch.int32), group)
            q_ref, s_ref = ref.quantize_groups_q4(ref.merge_perm(W, pR, pP), group)
        else:
            P.quantize_q4(Wd, q, s, group)
            q_ref, s_ref = ref.quantize_groups_q4(W, group)
        assert np.array_equal(q.cpu().numpy(), ref.pack_q4(q_ref))
        assert _same_scales(s, s_ref, group)
        W_ref = ref.dequantize_groups(q_ref, s_ref)
        for t in (torch.bfloat16, torch.float32):
            out = torch.full((m, n), 9.0, dtype=t, device="cuda")
            P.dequantize_q4(q, s, out, group)
            assert np.array_equal(host(out), W_ref)  # exact in either type


def test_quantiser_edges(P):
    """Ties, tiny (subnormal) and huge groups, infinities and NaN, against the oracle."""
    import torch
    rng = np.random.default_rng(5)
    n, rows = 128, []
    for k in range(-149, 127, 4):  # every scale, subnormal ones among them
        with np.errstate(over="ignore"):
            rows.append(np.clip(rng.standard_normal(n) * 2.0 ** k, -3.3e38, 3.3e38))
    # ties: multiples of half a scale
    for sc in (1.0, 31 / 32, 2.0 ** -120, 17.0 * 2.0 ** 30):
        r = rng.integers(-14, 15, n) * (sc / 2)
        r[:: 32] = 7 * sc
        rows.append(r)
    for bad in (np.inf, -np.inf, np.nan):
        r = rng.standard_normal(n)
        r[rng.integers(0, n)] = bad
        rows.append(r)
    rows.append(np.full(n, -0.0))
    W = np.array(rows).astype(np.float32)
    for dt in (torch.float32, torch.bfloat16):
        Wd = torch.from_numpy(W).cuda().to(dt)
        Wh = Wd.float().cpu().numpy()
        for group in (32, 64, 128):
            q, s = _buffers(P, W.shape[0], n, group)
            P.quantize_q4(Wd, q, s, group)
            q_ref, s_ref = ref.quantize_groups_q4(Wh, group)
            assert np.array_equal(q.cpu().numpy(), ref.pack_q4(q_ref))
            assert _same_scales(s, s_ref, group)
            out = torch.empty(W.shape, dtype=torch.float32, device="cuda")
            P.dequantize_q4(q, s, out, group)
            assert np.array_equal(host(out), ref.dequantize_groups(q_ref, s_ref), equal_nan=True)


def _packed(P, m, n, group, seed, scale_bits=5):
    """Codes over the whole range and scales of `scale_bits` significant bits."""
    import torch
    rng = np.random.default_rng(seed)
    q = rng.integers(-8, 8, (m, n)).astype(np.int8)
    mant = rng.integers(1 << (scale_bits - 1), 1 << scale_bits, (m, n // group))
    s = mant * 2.0 ** rng.integers(-12, -6, (m, n // group))
    qd = torch.from_numpy(ref.pack_q4(q)).cuda()
    sd = torch.from_numpy(ref.pack_scales(s, group)).to(torch.bfloat16).cuda()
    return qd, sd, ref.dequantize_groups(q, s)


def _check_product(y, x, W, transpose, extra=0.0):
    Wt = W if transpose else W.T
    ref_y = x @ Wt
    mag = np.abs(x) @ np.abs(Wt)
    K = x.shape[1]
    bound = 2.0 ** -8 * np.abs(ref_y) + (K / 16 + 64) * 2.0 ** -23 * mag + extra * mag
    assert np.all(np.abs(host(y) - ref_y) <= bound)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n", [(1, 128), (17, 256), (333, 1152), (2048, 640)])
def test_few_token_products(P, m, n, group, transpose):
    import torch
    q, s, W = _packed(P, m, n, group, m + n + group)
    rng = np.random.default_rng(m)
    k, o = (m, n) if transpose else (n, m)
    for T in (1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 65, 130):
        x = round_to_bf16(rng.standard_normal((T, k)))
        xd = tensor(x, torch.bfloat16)
        buf = torch.full((T * o + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
        y = buf[: T * o].view(T, o)
        P.matmul_q4(xd, q, s, y, group, transpose=transpose)
        _check_product(y, x, W, transpose)
        assert torch.all(buf[T * o:] == 5.0)     # nothing behind the last row
        y2 = torch.empty_like(y)
        P.matmul_q4(xd, q, s, y2, group, transpose=transpose)
        assert torch.equal(y, y2)                # same sums in the same order
    assert P.device_status() == P.POETX_OK


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("T,m,n,group,pairs", [(256, 512, 256, 32, True), (300, 256, 512, 128, True),
                                               (777, 768, 1024, 64, True),
                                               (1000, 520, 768, 128, True),
                                               (513, 999, 640, 32, True),
                                               (600, 512, 512, 64, False),
                                               (1030, 2560, 2560, 64, True),
                                               (1100, 2560, 2816, 32, True),
                                               (1300, 2304, 2560, 128, True),
                                               (150, 1001, 384, 64, True)])
def test_many_token_products(P, T, m, n, group, pairs, transpose):
    import torch
    q, s, W = _packed(P, m, n, group, T + m)
    rng = np.random.default_rng(T)
    k, o = (m, n) if transpose else (n, m)
    x = round_to_bf16(rng.standard_normal((T, k)))
    xd = tensor(x, torch.bfloat16)
    buf = torch.full((T * o + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    y = buf[: T * o].view(T, o)
    prev = P.set_gemm_pairs(pairs)
    try:
        P.matmul_q4(xd, q, s, y, group, transpose=transpose)
        torch.cuda.synchronize()
    finally:
        P.set_gemm_pairs(prev)
    _check_product(y, x, W, transpose)
    assert torch.all(buf[T * o:] == 5.0)
    assert P.device_status() == P.POETX_OK


@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("transpose", [False, True])
def test_products_with_a_callers_own_scales(P, T, transpose):
    """Scales of 8 significant bits: s q may be rounded to bf16 (half a step, 2^-8)."""
    import torch
    q, s, W = _packed(P, 512, 512, 64, 4, scale_bits=8)
    x = round_to_bf16(np.random.default_rng(T).standard_normal((T, 512)))
    y = torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")
    P.matmul_q4(tensor(x, torch.bfloat16), q, s, y, 64, transpose=transpose)
    _check_product(y, x, W, transpose, extra=2.0 ** -8)


def test_a_row_of_infinities_stays_in_its_row(P):
    import torch
    q, s, W = _packed(P, 256, 256, 32, 9)
    for T in (5, 40, 300):
        for transpose in (False, True):
            x = round_to_bf16(np.random.default_rng(T).standard_normal((T, 256)))
            xd = tensor(x, torch.bfloat16)
            xd[2] = float("inf")
            xd[3, 7] = float("nan")
            y = torch.empty(T, 256, dtype=torch.bfloat16, device="cuda")
            P.matmul_q4(xd, q, s, y, 32, transpose=transpose)
            rows = [r for r in range(T) if r not in (2, 3)]
            _check_product(y[rows], x[rows], W, transpose)
            assert torch.all(torch.isnan(y[3].float()))


def test_products_on_another_stream_and_in_two_graphs(P):
    """The products keep no workspace: two captured graphs replayed at once do not meet."""
    import torch
    q, s, W = _packed(P, 640, 512, 64, 11)
    rng = np.random.default_rng(1)
    cases = []
    for T, transpose in ((1, False), (3, True), (300, False), (300, True)):
        k, o = (640, 512) if transpose else (512, 640)
        x = round_to_bf16(rng.standard_normal((T, k)))
        y = torch.zeros(T, o, dtype=torch.bfloat16, device="cuda")
        cases.append((x, tensor(x, torch.bfloat16), y, transpose))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for (x, xd, y, tr), st in zip(cases, streams):
        P.matmul_q4(xd, q, s, y, 64, transpose=tr, stream=st)
    torch.cuda.synchronize()
    graphs = []
    for x, xd, y, tr in cases:
        _check_product(y, x, W, tr)
        y.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            P.matmul_q4(xd, q, s, y, 64, transpose=tr)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for x, xd, y, tr in cases:
        _check_product(y, x, W, tr)


def test_python_refusals(P):
    import torch
    q, s, _ = _packed(P, 8, 128, 64, 1)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, y = torch.zeros(2, 128, **bf), torch.zeros(2, 8, **bf)
    for bad in (dict(q=q[:, :4].contiguous()), dict(s=s.float()), dict(group=128),
                dict(x=x.float()), dict(y=torch.zeros(3, 8, **bf)), dict(q=q.cpu()),
                dict(x=torch.zeros(128, 2, **bf).t())):
        a = dict(x=x, q=q, s=s, y=y, group=64)
        a.update(bad)
        with pytest.raises(ValueError):
            P.matmul_q4(a["x"], a["q"], a["s"], a["y"], a["group"])
    with pytest.raises(ValueError):
        P.dequantize_q4(q, s, torch.zeros(8, 256, **bf), 64)
    with pytest.raises(ValueError):
        P.merge_perm_q4(torch.zeros(8, 128, **bf), q, s, torch.zeros(8, device="cuda"),
                        torch.zeros(128, dtype=torch.int32, device="cuda"), 64)
    with pytest.raises(ValueError):
        P.PoetxLinear(torch.zeros(256, 256, device="cuda"), 0, 0, np.arange(256), np.arange(256),
                      128, 4, 8, int4_group=64)


# ------------------------------------------------------------------------ the layer
def _layer(P, T, n, m, b, group, save=True):
    import torch
    sh = LayerShape(f"q4-{n}x{m}", T=T, n=n, m=m, b=b, k=4, dtype="bf16", config_id=21,
                    std_theta=0.01)
    inp = layer_inputs(sh)
    pP, _ = P.make_perm(inp.seed_P, n)
    pR, _ = P.make_perm(inp.seed_R, m)
    L = P.PoetxLinear(tensor(inp.W0, torch.bfloat16), tensor(inp.theta_P, torch.float32),
                      tensor(inp.theta_R, torch.float32), pP, pR, b, 4, T, save_activations=save,
                      int4_group=group)
    return inp, L, pP, pR


@pytest.mark.parametrize("T,n,m,b,group", [(1, 256, 512, 128, 32), (5, 512, 512, 256, 64),
                                           (13, 512, 1024, 512, 128), (50, 768, 256, 128, 64),
                                           (64, 256, 256, 256, 32), (65, 256, 512, 128, 128),
                                           (300, 512, 768, 256, 64), (700, 384, 640, 128, 128)])
def test_layer_step_matches_the_oracle(P, T, n, m, b, group):
    """One step of the layer on the 4-bit weight (merge, CNP, forward, backward) against the
    float64 oracle's layer on the weight that the oracle's quantiser gives."""
    import torch
    inp, L, pP, pR = _layer(P, T, n, m, b, group)
    q_ref, s_ref = ref.quantize_groups_q4(ref.merge_perm(inp.W0, pR, pP), group)
    W_ref = ref.dequantize_groups(q_ref, s_ref)
    x, dy = tensor(inp.x, torch.bfloat16), tensor(inp.dy, torch.bfloat16)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    L.step(x, dy, y, dx)
    torch.cuda.synchronize()
    assert P.device_status() == P.POETX_OK
    G_P = ref.cnp_forward(inp.theta_P, b, 4)
    G_R = ref.cnp_forward(inp.theta_R, b, 4)
    out = ref.layer_forward(inp.x, W_ref, G_P, G_R, pP, pR)
    y_ref, U_ref, W_act = out[0], out[1], out[-1]
    assert norm_max_err(host(y), y_ref) <= BF16_NORM
    back = ref.layer_backward(inp.x, inp.dy, W_ref, G_P, G_R, pP, pR)
    assert norm_max_err(host(dx), back[0]) <= BF16_NORM
    assert norm_max_err(host(L.dG[: L.nP]), back[1]) <= BF16_NORM
    assert norm_max_err(host(L.dG[L.nP:]), back[2]) <= BF16_NORM
    dth_P = ref.cnp_backward(inp.theta_P, back[1], b, 4)
    assert norm_max_err(host(L.dtheta[: L.nP]), dth_P) <= BF16_NORM
    # recomputed activations give the same step
    _, M, _, _ = _layer(P, T, n, m, b, group, save=False)
    ym, dxm = torch.empty_like(y), torch.empty_like(dx)
    M.step(x, dy, ym, dxm)
    assert torch.equal(ym, y) and torch.equal(dxm, dx) and torch.equal(M.dG, L.dG)
    # forward without save buffers (decoding) writes the same y
    yd = torch.full_like(y, 7.0)
    GP, GR = L.G_ops()
    P.linear_fwd_ex(L.desc, L.weight, None, x, GP, GR, yd, None, None, L.ws if L.ws.numel() >=
                    P.linear_ex_workspace(L.desc, L.weight, False, False) else M.ws)
    assert torch.equal(yd, y)


@pytest.mark.parametrize("T,n,m", [(1, 512, 512), (40, 512, 512), (300, 512, 512),
                                   (1300, 2048, 2048)])
def test_layer_equals_the_bf16_layer_on_the_dequantised_weight(P, T, n, m):
    import torch
    b, group = 256, 64
    inp, L, pP, pR = _layer(P, T, n, m, b, group)
    x, dy = tensor(inp.x, torch.bfloat16), tensor(inp.dy, torch.bfloat16)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    L.step(x, dy, y, dx)
    W = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    P.dequantize_q4(L.W0q, L.scales, W, group)
    GP, GR = L.G_ops()
    ws = torch.empty(max(P.linear_fwd_workspace(L.desc), P.linear_bwd_workspace(L.desc)),
                     dtype=torch.uint8, device="cuda")
    y0, dx0 = torch.empty_like(y), torch.empty_like(dx)
    U, Ws = torch.empty_like(L.U), torch.empty_like(L.Wsave)
    dGP, dGR = torch.empty_like(L.dG[: L.nP]), torch.empty_like(L.dG[L.nP:])
    P.linear_fwd(L.desc, x, GP, GR, W, y0, U, Ws, ws)
    P.linear_bwd(L.desc, x, dy, GP, GR, W, U, Ws, dx0, dGP, dGR, 0, ws)
    assert torch.equal(L.U, U)  # gathered bit for bit in either form
    if T >= 1024:  # the same tensor-core kernel on the same operands
        assert torch.equal(y, y0) and torch.equal(dx, dx0)
        assert torch.equal(L.dG[: L.nP], dGP) and torch.equal(L.dG[L.nP:], dGR)
    else:
        for a, r in ((y, y0), (dx, dx0), (L.dG[: L.nP], dGP), (L.dG[L.nP:], dGR)):
            assert norm_max_err(host(a), host(r)) <= BF16_NORM


def test_decoding_in_a_graph_while_a_step_runs(P):
    """A captured decoding pass replayed on one stream while a training step of another layer
    runs on a second stream: both give what they give alone."""
    import torch
    inp, L, _, _ = _layer(P, 1, 512, 512, 256, 128)
    inp2, M, _, _ = _layer(P, 300, 512, 512, 256, 64)
    L.cnp_forward()
    x = tensor(inp.x, torch.bfloat16)
    y = torch.empty(1, 512, dtype=torch.bfloat16, device="cuda")
    L.forward(x, y)
    want = y.clone()
    x2, dy2 = tensor(inp2.x, torch.bfloat16), tensor(inp2.dy, torch.bfloat16)
    y2, dx2 = torch.empty_like(dy2), torch.empty_like(x2)
    M.step(x2, dy2, y2, dx2)
    want2 = (y2.clone(), dx2.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.forward(x, y)
    y.zero_()
    y2.zero_()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            g.replay()
        M.step(x2, dy2, y2, dx2, s2)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(y2, want2[0]) and torch.equal(dx2, want2[1])


@pytest.mark.parametrize("T,n,m,b,group", [(1, 512, 768, 128, 64), (3, 1024, 512, 256, 32),
                                           (4, 2560, 256, 256, 128), (2, 512, 1024, 512, 128),
                                           (7, 512, 2048, 512, 128), (8, 2560, 256, 256, 128),
                                           (11, 512, 768, 128, 32), (16, 768, 512, 256, 64),
                                           (19, 512, 1024, 256, 128), (32, 256, 768, 128, 64)])
def test_roundings_of_the_few_token_layer(P, T, n, m, b, group):
    """y is off by half a step (2^-8) and by what V and W are off by: half a step each, or up to 4
    tokens, where they are sums of two bf16 numbers, 2^-16 (half a step of half a step); the fp32
    sums of b, n and b products by at most 2^-23 for each of their (2 b + n) / 16 + 3 * 64
    roundings."""
    import torch
    _, L, pP, pR = _layer(P, T, n, m, b, group, save=False)
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, n))
    xd = tensor(x, torch.bfloat16)
    GP = tensor(rng.standard_normal((n // b, b, b)) / 16, torch.bfloat16)
    GR = tensor(rng.standard_normal((m // b, b, b)) / 16, torch.bfloat16)
    y = torch.full((T, m), 7.0, dtype=torch.bfloat16, device="cuda")
    U, V = torch.empty_like(xd), torch.empty_like(y)
    ws = torch.empty(P.linear_ex_workspace(L.desc, L.weight, True, True), dtype=torch.uint8,
                     device="cuda")
    P.linear_fwd_ex(L.desc, L.weight, None, xd, GP, GR, y, U, V, ws)
    W = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    P.dequantize_q4(L.W0q, L.scales, W, group)
    maps = [np.asarray(p) for p in (pP, pR)]

    def layer(f):
        u = f(host(xd))[:, maps[0]]
        v = np.einsum("tjk,jik->tji", u.reshape(T, -1, b), f(host(GP))).reshape(T, n)
        w = v @ f(host(W)).T
        z = np.einsum("tjk,jik->tji", w.reshape(T, -1, b), f(host(GR))).reshape(T, m)
        out = np.empty_like(z)
        out[:, maps[1]] = z
        return u, w, out

    u_ref, w_ref, y_ref = layer(lambda a: a.astype(np.float64))
    _, w_mag, y_mag = layer(lambda a: np.abs(a.astype(np.float64)))
    assert np.array_equal(host(U), u_ref)
    mid = 2.0 ** -16 if T <= 4 else 2.0 ** -8
    sums = ((2 * b + n) / 16 + 192) * 2.0 ** -23
    w_err, y_err = np.abs(host(V) - w_ref), np.abs(host(y) - y_ref)
    assert np.all(w_err <= 2.0 ** -8 * np.abs(w_ref) + (mid + sums) * 1.01 * w_mag)
    assert np.all(y_err <= 2.0 ** -8 * np.abs(y_ref) + (2 * mid + sums) * 1.01 * y_mag)


def test_decoding_right_behind_new_weights_and_rotations(P):
    """The launches of a decoding pass overlap: what it reads early was written by the launches
    just before it, merges and rotations that nothing waits for."""
    import torch
    T, n, m, b = 2, 512, 512, 256
    _, L, pP, pR = _layer(P, T, n, m, b, 64, save=False)
    torch.manual_seed(0)
    x = torch.randn(T, n, device="cuda").bfloat16()
    Ws = [torch.randn(m, n, device="cuda").bfloat16() for _ in range(6)]
    Gs = [torch.randn(2, n // b, b, b, device="cuda").bfloat16() for _ in range(6)]
    GP, GR = (torch.empty(n // b, b, b, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def run(i, wait):
        y = torch.empty(T, m, dtype=torch.bfloat16, device="cuda")
        GP.copy_(Gs[i][0])
        GR.copy_(Gs[i][1])
        P.quantize_q4(Ws[i], L.W0q, L.scales, 64)
        if wait:
            torch.cuda.synchronize()
        P.linear_fwd_ex(L.desc, L.weight, None, x, GP, GR, y, None, None, L.ws)
        return y

    want = [run(i, True) for i in range(6)]
    torch.cuda.synchronize()
    got = [run(i % 6, False) for i in range(60)]
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 6])


def test_layer_call_refuses_tensors_that_are_not_the_layer_s(P):
    import torch
    T, n, m, b = 3, 256, 512, 128
    _, L, _, _ = _layer(P, T, n, m, b, 64)
    GP, GR = L.G_ops()
    x, y = (torch.zeros(T, c, dtype=torch.bfloat16, device="cuda") for c in (n, m))
    good = dict(x=x, G_P=GP, G_R=GR, y=y, save_u=L.U, save_w=L.Wsave, ws=L.ws, w=L.weight)

    def fwd(**bad):
        a = {**good, **bad}
        P.linear_fwd_ex(L.desc, a["w"], None, a["x"], a["G_P"], a["G_R"], a["y"], a["save_u"],
                        a["save_w"], a["ws"])

    fwd()
    for bad in (dict(x=x.float()), dict(x=x[:2]), dict(x=x.cpu()), dict(y=y[:, :n].contiguous()),
                dict(y=y.half()), dict(G_P=GR), dict(G_R=GR.float()), dict(save_u=L.Wsave),
                dict(save_w=L.Wsave.float()), dict(w=P.LinearWeight(P.POETX_WEIGHT_Q4, 64, 0, 0)),
                dict(w=P.linear_weight_dense(torch.zeros(m, n, device="cuda"))),
                dict(w=P.linear_weight_q4(L.W0q, L.scales, 128)),
                dict(x=torch.zeros(n, T, dtype=torch.bfloat16, device="cuda").t())):
        with pytest.raises(ValueError):
            fwd(**bad)
    with pytest.raises(P.PoetxError):
        fwd(ws=L.ws[:64])
    dx, dG = torch.zeros_like(x), [L.dG[: L.nP], L.dG[L.nP:]]
    for bad in ([dG[1], dG[0]], [dG[0].bfloat16(), dG[1]]):
        with pytest.raises(ValueError):
            P.linear_bwd_ex(L.desc, L.weight, None, x, y, GP, GR, L.U, L.Wsave, dx, *bad, 0, L.ws)


def test_more_blocks_and_token_tiles_than_a_grid_has(P):
    import torch
    m, n = 1, 128 * 65537
    q, s = _buffers(P, m, n, 32)
    q.copy_(torch.randint(0, 256, q.shape, dtype=torch.uint8, device="cuda"))
    s.fill_(0.5)
    out = torch.zeros(m, n, device="cuda")
    P.dequantize_q4(q, s, out, 32)
    one_q, one_s = q[-1:].clone(), s[-1:].clone()
    one = torch.zeros(1, 128, device="cuda")
    P.dequantize_q4(one_q, one_s, one, 32)
    assert torch.equal(out[:, -128:], one) and bool((out != 0).any(1).all())
    # rows of one value: the form for any row count, tiles of 64 tokens
    T = (1 << 21) + 5
    x = torch.randn(T, 1, device="cuda").bfloat16()
    y = torch.full((T, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    P.matmul_q4(x, one_q, one_s, y, 32, transpose=True)
    for part in (slice(0, 300), slice(T - 300, T)):
        ref_y = x[part].double() * one.double()
        assert bool(((y[part].double() - ref_y).abs() <= 2.0 ** -8 * ref_y.abs()).all())
    torch.cuda.synchronize()
    assert P.device_status() == P.POETX_OK


@pytest.mark.parametrize("T,m,n,group,transpose", [(1100, 4096, 256, 64, False),
                                                   (1281, 264, 4096, 32, True),
                                                   (2049, 2560, 128, 128, False)])
def test_product_whose_last_tokens_take_the_other_kernel(P, T, m, n, group, transpose):
    import torch
    torch.manual_seed(T)
    W = torch.randn(m, n, device="cuda")
    q, s = _buffers(P, m, n, group)
    P.quantize_q4(W, q, s, group)
    P.dequantize_q4(q, s, W, group)
    K, N = (m, n) if transpose else (n, m)
    x = torch.randn(T, K, device="cuda").bfloat16()
    y = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    P.matmul_q4(x, q, s, y[:T], group, transpose=transpose)
    Wd = W.double() if transpose else W.double().t()
    want, mag = x.double() @ Wd, x.double().abs() @ Wd.abs()
    bound = 2.0 ** -8 * want.abs() + 1.01 * (K / 16 + 64) * 2.0 ** -23 * mag
    assert bool(((y[:T].double() - want).abs() <= bound).all())
    assert bool((y[T] == 7.0).all())


@pytest.mark.parametrize("T", [2, 6])
def test_infinities_pass_through_the_few_token_layer(P, T):
    """Positive weights and rotations: an infinite x gives that infinity in every output of its
    token, as the formula does, and no other token sees it."""
    import torch
    n, m, b, group = 256, 384, 128, 32
    _, L, pP, _ = _layer(P, T, n, m, b, group, save=False)
    P.quantize_q4(torch.rand(m, n, device="cuda") + 0.5, L.W0q, L.scales, group)
    GP = torch.rand(n // b, b, b, device="cuda").add(0.5).bfloat16()
    GR = torch.rand(m // b, b, b, device="cuda").add(0.5).bfloat16()
    x = torch.randn(T, n, device="cuda").bfloat16()
    y = torch.empty(T, m, dtype=torch.bfloat16, device="cuda")
    P.linear_fwd_ex(L.desc, L.weight, None, x, GP, GR, y, None, None, L.ws)
    clean = y.clone()
    x[1, 37] = float("-inf")
    P.linear_fwd_ex(L.desc, L.weight, None, x, GP, GR, y, None, None, L.ws)
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isfinite(clean).all())
    assert bool((y[1] == float("-inf")).all())


@pytest.mark.parametrize("argv", [["q4merge", "300", "512", "64"], ["q4", "2", "512", "256", "32"],
                                  ["q4", "70", "512", "256", "32"], ["q4layer", "3", "256", "512"],
                                  ["q4layer", "40", "256", "512"], ["dropout", "64", "512"]])
def test_kernel_cases_run(P, argv, capsys):
    from orthogonal_reparameterized_cnp_b200 import kernel_cases
    assert kernel_cases.main(argv) == 0
    assert f"{argv[0]} ok" in capsys.readouterr().out


FIRST_CALLS_IN_A_CAPTURE = """
import torch
from orthogonal_reparameterized_cnp_b200 import poetx as P
dev = torch.device("cuda")
bf = dict(dtype=torch.bfloat16, device=dev)
m, n, b, group = 512, 768, 128, 64
qs, ss = P.q4_shapes(m, n, group)
q, s = torch.empty(qs, dtype=torch.uint8, device=dev), torch.empty(ss, **bf)
W, out = torch.randn(m, n, **bf), torch.empty(m, n, **bf)
maps = [torch.from_numpy(a).to(dev) for a in (*P.make_perm(1, n), *P.make_perm(2, m))]
GP, GR = torch.randn(n // b, b, b, **bf), torch.randn(m // b, b, b, **bf)
calls, bufs = [], []
for T in (2, 12, 40, 9600):
    x, y = torch.randn(T, n, **bf), torch.empty(T, m, **bf)
    back, z = torch.empty(T, n, **bf), torch.empty(T, m, **bf)
    d, w = P.linear_desc(T, n, m, b, P.POETX_BF16, *maps), P.linear_weight_q4(q, s, group)
    ws = torch.empty(P.linear_ex_workspace(d, w, False, False) + 16, dtype=torch.uint8, device=dev)
    drop = P.dropout_desc(0.25, 5)
    masked, gathered = torch.empty_like(x), torch.empty_like(x)
    bufs += [y, back, z, masked, gathered]
    calls += [lambda x=x, y=y: P.matmul_q4(x, q, s, y, group),
              lambda y=y, o=back: P.matmul_q4(y, q, s, o, group, transpose=True),
              lambda x=x, z=z, d=d, w=w, ws=ws: P.linear_fwd_ex(d, w, None, x, GP, GR, z, None,
                                                                None, ws),
              lambda x=x, o=masked, d=drop: P.dropout(d, x, o),
              lambda x=x, o=gathered, d=drop: P.permute_cols_dropout(d, x, o, maps[0])]
def run():
    P.quantize_q4(W, q, s, group)
    P.dequantize_q4(q, s, out, group)
    for c in calls:
        c()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in bufs]
for t in bufs:
    t.zero_()
run()
torch.cuda.synchronize()
assert all(torch.equal(a, c) for a, c in zip(bufs, got)), "replay differs"
assert P.device_status() == P.POETX_OK
print("captured first")
"""


def test_first_calls_inside_a_capture(P):
    """A program whose first call of every kernel is a captured one."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_IN_A_CAPTURE], cwd=root, timeout=300,
                       capture_output=True, text=True)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]
