"""The layer object on every form of the merged weight: which weight its calls read, and calls on
fewer tokens than it was built for."""
import numpy as np
import pytest

from .gpu_harness import tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from orthogonal_reparameterized_cnp_b200 import poetx
    poetx.lib()
    return poetx


KINDS = ["f32", "bf16", "q8", "q4"]


def _layer(P, kind, T, n, m, b=128, dropout=None, save=True, seed=0):
    """The layer, and x, dy for it; seed: of W0 alone (rotations, maps and inputs stay)."""
    import torch
    act = torch.float32 if kind == "f32" else torch.bfloat16
    W0 = tensor(np.random.default_rng(seed).standard_normal((m, n)) / np.sqrt(n), act)
    rng = np.random.default_rng(n + m)
    th = [tensor(rng.standard_normal((k // b, b * (b - 1) // 2)) * 0.01, torch.float32)
          for k in (n, m)]
    L = P.PoetxLinear(W0, th[0], th[1], P.make_perm(1, n)[0], P.make_perm(2, m)[0], b, 4, T,
                      save_activations=save, int8_weight=kind == "q8",
                      int4_group=64 if kind == "q4" else 0, dropout=dropout)
    L.cnp_forward()
    return L, tensor(rng.standard_normal((T, n)), act), tensor(rng.standard_normal((T, m)), act)


def _run(L, x, dy):
    import torch
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    L.forward(x, y)
    L.backward(x, dy, dx)
    return y, dx, L.dG.clone()


def _equal(a, b):
    import torch
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("how", ["assigned", "storage"])
@pytest.mark.parametrize("kind", KINDS)
def test_every_call_reads_the_weight_that_the_layer_holds(P, kind, how):
    """After W0p, or W0q and scales, have become another layer's (a new tensor, or the same one
    with its storage exchanged), training with dropout (p = 0: nothing dropped, the path of a
    layer with dropout), evaluation and backward give that layer's results bit for bit."""
    L, x, dy = _layer(P, kind, 40, 256, 384, dropout=P.Dropout(0.0, 1))
    M, _, _ = _layer(P, kind, 40, 256, 384, seed=9)
    old, want = _run(L, x, dy), _run(M, x, dy)
    assert not any(u.equal(v) for u, v in zip(old[:2], want[:2]))
    names = ("W0q", "scales") if kind in ("q8", "q4") else ("W0p",)
    for name in names:
        if how == "assigned":
            setattr(L, name, getattr(M, name).clone())
        else:
            getattr(L, name).data = getattr(M, name).clone()
    for training in (True, False):
        L.training = training
        assert _equal(_run(L, x, dy), want), training
    # merging again writes the tensors that are held now
    L.merge()
    assert _equal(_run(L, x, dy), old)
    assert all(t is u for t, u in zip(L.weight.keep, (getattr(L, k) for k in names)))
    assert P.device_status() == P.POETX_OK


@pytest.mark.parametrize("kind", KINDS)
def test_refusals_of_another_weight(P, kind):
    import torch
    L, x, dy = _layer(P, kind, 4, 256, 384)
    want = _run(L, x, dy)
    coded = kind in ("q8", "q4")
    for name in (("W0q", "scales") if coded else ("W0p",)):
        t = getattr(L, name)
        for bad in (None, t.cpu(), t[:-1], t.to(torch.float16),
                    t.repeat_interleave(2, dim=-1)[..., ::2]):  # (not contiguous)
            with pytest.raises(ValueError):
                setattr(L, name, bad)
        assert getattr(L, name) is t
    for name in (("W0p",) if coded else ("W0q", "scales")):
        assert getattr(L, name) is None
        with pytest.raises(ValueError):
            setattr(L, name, L.weight.keep[0])
    assert _equal(_run(L, x, dy), want)


@pytest.mark.parametrize("save", [True, False])
@pytest.mark.parametrize("kind,T,rows", [("f32", 40, 7), ("bf16", 300, 1), ("bf16", 300, 299),
                                         ("q8", 300, 2), ("q8", 600, 257), ("q4", 300, 1),
                                         ("q4", 5, 4), ("q4", 20, 9), ("q4", 300, 16),
                                         ("q4", 300, 65), ("q4", 700, 513), ("q4", 3000, 2560)])
def test_calls_on_fewer_tokens(P, kind, T, rows, save):
    """A layer built for T tokens gives on its first `rows` of them what a layer built for `rows`
    gives, bit for bit: with and without dropout, forward and backward; T tokens afterwards give
    what they gave before, and nothing behind the rows is written."""
    import torch
    L, x, dy = _layer(P, kind, T, 256, 384, dropout=P.Dropout(0.25, 3), save=save)
    M, _, _ = _layer(P, kind, rows, 256, 384, dropout=P.Dropout(0.25, 3), save=save)
    full = _run(L, x, dy)
    xr, dyr = x[:rows], dy[:rows]
    for training in (True, False):
        L.training = M.training = training
        want = _run(M, xr.contiguous(), dyr.contiguous())
        y, dx = torch.full_like(dy, 7.0), torch.full_like(x, 7.0)
        L.forward(xr, y[:rows])
        L.backward(xr, dyr, dx[:rows])
        assert _equal((y[:rows], dx[:rows], L.dG), want), training
        assert bool((y[rows:] == 7.0).all()) and bool((dx[rows:] == 7.0).all())
    L.training = True
    assert _equal(_run(L, x, dy), full)
    assert P.device_status() == P.POETX_OK


def test_decoding_with_the_layer_that_was_trained(P):
    """A training step on T tokens, then one token and no tokens through the same object; one
    token also from a captured graph."""
    import torch
    L, x, dy = _layer(P, "q4", 300, 512, 512, dropout=P.Dropout(0.1, 7))
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    L.step(x, dy, y, dx)
    L.training = False
    L.forward(x, y)
    one = torch.empty_like(y[:1])
    L.forward(x[5:6], one)
    # A bf16 rounding is off by 2^-8 of the value at most, by 0.0017 in the root mean square; here
    # four of them meet (V, W and y of the 300 tokens, y of the one): 0.0034.  2^-7 is twice that.
    assert float((one.float() - y[5:6].float()).norm()) <= 2.0 ** -7 * float(y[5:6].float().norm())
    L.forward(x[:0], y[:0])
    L.backward(x[:0], dy[:0], dx[:0])
    assert bool((L.dG == 0).all())
    got = torch.zeros_like(one)
    src = x[5:6].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.forward(src, got)
    g.replay()
    assert torch.equal(got, one)
    src.copy_(x[6:7])
    g.replay()
    L.forward(x[6:7], one)
    assert torch.equal(got, one)


def test_group_on_fewer_tokens(P):
    import torch
    rng = np.random.default_rng(0)
    n, b = 256, 128
    th = [tensor(rng.standard_normal((2, b * (b - 1) // 2)) * 0.01, torch.float32)
          for _ in range(2)]
    pP, _ = P.make_perm(1, n)
    W0 = tensor(rng.standard_normal((n, n)) / 16, torch.bfloat16)
    x = tensor(rng.standard_normal((40, n)), torch.bfloat16)
    out = []
    for T in (40, 11):
        G = P.PoetxLinearGroup([(W0, th[0], th[1], pP, pP)] * 2, b, 4, T, int4_group=128)
        ys, dxs = ([torch.empty_like(x[:11]) for _ in range(2)] for _ in range(2))
        G.step([x[:11]] * 2, [x[:11]] * 2, ys, dxs)
        out.append((*ys, *dxs, G.cnp.dtheta.clone()))
    assert _equal(*out)


@pytest.mark.parametrize("kind", KINDS)
def test_refusals_of_token_counts(P, kind):
    import torch
    L, x, dy = _layer(P, kind, 6, 256, 384)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    more_x, more_y = torch.cat([x, x]), torch.cat([dy, dy])
    if kind == "q4":
        with pytest.raises(ValueError):
            L.forward(more_x, more_y)
        with pytest.raises(ValueError):
            L.backward(more_x, more_y, more_x)
    for a, o in ((x[:4], y[:5]), (x[:4], y[:4, :128].contiguous()),
                 (x[:4, :128].contiguous(), y[:4]), (x[:4].to(torch.float16), y[:4])):
        with pytest.raises(ValueError):
            L.forward(a, o)
    for a, d, o in ((x[:5], dy[:4], dx[:4]), (x[:4], dy[:4], dx[:5]),
                    (x[:4], dy[:4].to(torch.float16), dx[:4])):
        with pytest.raises(ValueError):
            L.backward(a, d, o)
    with pytest.raises(ValueError):  # rows that are not side by side
        L.forward(x[::2], y[:3])


@pytest.mark.parametrize("T,n,m", [(1, 256, 384), (4, 512, 256), (9, 256, 256), (40, 384, 256)])
def test_few_tokens_that_save_nothing_write_v_and_w_alone(P, T, n, m):
    """The three launches of a few tokens keep V and W in scratch (up to 4 tokens as two bf16
    numbers each), not the gathered input nor Z; the outputs are those of a call that saves."""
    import torch
    L, x, dy = _layer(P, "q4", T, n, m)
    y, z = torch.empty_like(dy), torch.empty_like(dy)
    L.forward(x, y)
    GP, GR = L.G_ops()
    room = P.linear_ex_workspace(L.desc, L.weight, False, False)
    ws = torch.full((room,), 0xA5, dtype=torch.uint8, device="cuda")
    P.linear_fwd_ex(L.desc, L.weight, None, x, GP, GR, z, None, None, ws)
    assert torch.equal(y, z)
    written = int((ws.view(torch.int16) != -23131).sum())  # (0xA5A5 as a bf16 is an unlikely value)
    halves = 2 if T <= 4 else 1
    assert 0.9 * halves * T * (n + m) <= written <= halves * T * (n + m)
    assert torch.equal(L.U, x[:, L.perm_P.long()])


@pytest.mark.parametrize("kind,T,y_roundings,dx_roundings",
                         [("f32", 70, 0, 0), ("bf16", 300, 3, 3), ("q8", 300, 3, 3),
                          ("q4", 300, 3, 3), ("q4", 64, 3, 3), ("q4", 16, 3, 3), ("q4", 4, 1, 3),
                          ("q4", 1, 1, 3)])
def test_roundings_of_y_and_dx(P, kind, T, y_roundings, dx_roundings):
    """As many bf16 roundings as the header says.  One is off by up to half of 2^-7 2^e in a value
    of [2^e, 2^(e+1)), evenly: at most 2^-7 / sqrt(12) of the value in the root mean square.  The
    rotations keep norms and the random weight does so in the mean, so k of them give sqrt(k) times
    that; a tenth more for the spread (2^8 values and more), 1e-5 for fp32 sums and second halves."""
    import torch
    n, m, b = 512, 768, 128
    L, x, dy = _layer(P, kind, T, n, m, b)
    y, dx, _ = _run(L, x, dy)
    if kind == "q4":
        W = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        P.dequantize_q4(L.W0q, L.scales, W, 64)
    else:
        W = (L.scales[:, None] * L.W0q.float()).bfloat16() if kind == "q8" else L.W0p
    W = W.double()
    GP, GR = (G.double() for G in L.G_ops())
    pP, pR = L.perm_P.long(), L.perm_R.long()

    def blocks(a, G):
        return torch.einsum("tji,jki->tjk", a.view(T, -1, b), G).reshape(T, -1)

    want_y = torch.empty(T, m, dtype=torch.float64, device="cuda")
    want_y[:, pR] = blocks(blocks(x.double()[:, pP], GP) @ W.t(), GR)
    want_dx = torch.empty(T, n, dtype=torch.float64, device="cuda")
    want_dx[:, pP] = blocks(blocks(dy.double()[:, pR], GR.transpose(1, 2)) @ W,
                            GP.transpose(1, 2))
    for got, want, k in ((y, want_y, y_roundings), (dx, want_dx, dx_roundings)):
        off = float((got.double() - want).norm() / want.norm())
        assert off <= 1.1 * (k / 12) ** 0.5 * 2.0 ** -7 + 1e-5, (off, k)


@pytest.mark.parametrize("kind", KINDS)
def test_layer_that_gave_up_w0(P, kind):
    """It trains as before, without holding the unquantised weight, and cannot merge again."""
    import gc
    import weakref
    L, x, dy = _layer(P, kind, 20, 256, 384)
    want = _run(L, x, dy)
    held = weakref.ref(L.W0)
    L.W0 = None
    gc.collect()
    assert held() is None
    assert _equal(_run(L, x, dy), want)
    with pytest.raises(ValueError):
        L.merge()
    assert _equal(_run(L, x, dy), want)
    for name in (("W0p",) if kind in ("q8", "q4") else ("W0q", "scales")):
        setattr(L, name, None)  # what the form does not have
