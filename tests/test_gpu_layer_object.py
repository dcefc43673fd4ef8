"""The layer object on every form of the merged weight: which weight its calls read."""
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
