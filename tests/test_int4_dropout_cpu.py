"""CPU tests of the 4-bit merged weight and of dropout: pins of the oracle's quantiser, packing
and generator, and the library's refusals (nothing is launched)."""
import ctypes

import numpy as np
import pytest

from oracle import poetx_ref as ref
from orthogonal_reparameterized_cnp_b200 import poetx as P

from .test_host_abi import _desc

F = ctypes.c_void_p(0x10000)
F2 = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10004)
BIG = 1 << 40


# ------------------------------------------------------------------------ oracle pins
def test_philox_known_answers():
    # the three known answers published with the generator
    assert ref.philox4x32_10([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 0xFFFFFFFF
    assert ref.philox4x32_10([ones] * 4, [ones] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6,
                                                         0x6D5451FD]
    assert ref.philox4x32_10([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344],
                             [0xA4093822, 0x299F31D0]) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420,
                                                           0x24126EA1]


def test_dropout_factor_is_the_generator_value_by_value():
    p, seed, site, row0, step = 0.3, 0x123456789ABCDEF, 5, 4000000000, 9
    f = ref.dropout_factor(3, 21, p, seed, site, row0, step)
    thr = round(p * 65536)
    for t in range(3):
        for c in range(21):
            w = ref.philox4x32_10([c // 8, row0 + t, site, step], [seed & 0xFFFFFFFF, seed >> 32])
            draw = (w[(c % 8) // 2] >> (16 * (c % 2))) & 0xFFFF
            assert f[t, c] == (65536 / (65536 - thr) if draw >= thr else 0.0)


@pytest.mark.parametrize("p", [0.05, 0.1, 0.5, 0.9])
def test_dropout_factor_keeps_the_mean(p):
    f = ref.dropout_factor(512, 1024, p, 77)
    n = f.size
    keep = (65536 - round(p * 65536)) / 65536
    # 6 standard deviations of the mean of n independent factors (0 or 1/keep)
    assert abs(f.mean() - 1.0) < 6 * np.sqrt((1 - keep) / keep / n)
    # neighbouring columns and rows are uncorrelated (6 / sqrt(n))
    d = (f - f.mean()) / f.std()
    assert abs((d[:, 1:] * d[:, :-1]).mean()) < 6 / np.sqrt(n)
    assert abs((d[1:] * d[:-1]).mean()) < 6 / np.sqrt(n)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_q4_quantiser_properties(group):
    rng = np.random.default_rng(group)
    W = (rng.standard_normal((37, 256)) * rng.uniform(1e-4, 3.0, (37, 1))).astype(np.float32)
    W[5] = 0
    q, s = ref.quantize_groups_q4(W, group)
    Wd = ref.dequantize_groups(q, s)
    # half a step everywhere: the rounded scale never clips (max|w| / s < 7.5)
    assert np.all(np.abs(Wd - W) <= 0.5 * np.repeat(s, group, axis=1) * (1 + 1e-7))
    assert np.all(s[5] == 0) and np.all(q[5] == 0)
    # 5 significant bits: the scale's mantissa times 16 is an integer
    mant, _ = np.frexp(s.astype(np.float64))
    assert np.all(mant * 32 == np.rint(mant * 32))
    # so s q is a bf16 number: the low 16 bits of the fp32 value are zero
    assert not np.any(Wd.astype(np.float32).view(np.uint32) & 0xFFFF)
    assert np.array_equal(Wd.astype(np.float32).astype(np.float64), Wd)
    # codes and scales that stand for W stand for themselves (idempotent where a code reaches 7)
    full = (np.abs(q).reshape(37, -1, group).max(axis=2) == 7)
    q2, s2 = ref.quantize_groups_q4(Wd, group)
    assert np.array_equal(s2[full], s[full])


def test_q4_quantiser_ties_and_non_finite_groups():
    W = np.zeros((1, 128), dtype=np.float32)
    W[0, :6] = [7.0, 0.5, 1.5, 2.5, -0.5, -3.5]      # scale 1: ties go to the even integer
    q, s = ref.quantize_groups_q4(W, 64)
    assert s[0, 0] == 1.0 and list(q[0, :6]) == [7, 0, 2, 2, 0, -4]
    W[0, 70] = np.inf
    q, s = ref.quantize_groups_q4(W, 64)
    assert np.isnan(s[0, 1]) and not np.any(q[0, 64:]) and s[0, 0] == 1.0
    W[0, 70] = np.nan
    assert np.isnan(ref.quantize_groups_q4(W, 64)[1][0, 1])


def test_q4_packing_one_value_at_a_time():
    rng = np.random.default_rng(3)
    q = rng.integers(-8, 8, (5, 256)).astype(np.int8)
    codes = ref.pack_q4(q)
    assert codes.shape == (2, 5, 64)
    for i, c in [(0, 0), (1, 1), (4, 255), (2, 128), (3, 37), (0, 95), (4, 130)]:
        blk, k = divmod(c, 128)
        w, t, e = k // 32, (k % 32) // 8, k % 8
        word = int.from_bytes(bytes(codes[blk, i, 16 * t + 4 * w:16 * t + 4 * w + 4]), "little")
        assert ((word >> (4 * (e // 2 + 4 * (e % 2)))) & 15) - 8 == q[i, c]


# ------------------------------------------------------------------------ refusals
def test_q4_weight_refusals():
    L = P.lib()
    merge = lambda W=F, q=F, s=F, m=4, n=256, R=F, C=F, g=64, dt=P.POETX_BF16: (  # noqa: E731
        L.poetx_merge_perm_q4(W, q, s, m, n, R, C, g, dt, None))
    assert merge(dt=9) == P.POETX_ERR_DTYPE
    assert merge(g=16) == P.POETX_ERR_SHAPE
    assert merge(g=0) == P.POETX_ERR_SHAPE
    assert merge(n=200) == P.POETX_ERR_SHAPE
    assert merge(n=-128) == P.POETX_ERR_INVALID_ARG
    assert merge(m=-1) == P.POETX_ERR_INVALID_ARG
    assert merge(W=None) == P.POETX_ERR_INVALID_ARG
    assert merge(R=None) == P.POETX_ERR_INVALID_ARG          # one map without the other
    assert merge(C=ODD) == P.POETX_ERR_ALIGN
    assert merge(q=ODD) == P.POETX_ERR_ALIGN
    assert merge(n=51328, dt=P.POETX_F32) == P.POETX_ERR_SHAPE  # rows above 200 KB
    assert merge(m=0) == P.POETX_OK and merge(n=0) == P.POETX_OK
    assert L.poetx_quantize_q4(F, F, F, 4, 100, 32, P.POETX_F32, None) == P.POETX_ERR_SHAPE
    big = (1 << 20, 1 << 16)  # 2^36 values: past the 32-bit offsets
    assert L.poetx_quantize_q4(F, F, F, *big, 32, P.POETX_BF16, None) == P.POETX_ERR_SHAPE
    assert L.poetx_dequantize_q4(F, F, F, *big, 32, P.POETX_BF16, None) == P.POETX_ERR_SHAPE
    assert L.poetx_matmul_q4(F, F, F, F, 1, *big, 32, 0, None) == P.POETX_ERR_SHAPE
    assert L.poetx_dequantize_q4(F, F, None, 4, 128, 32, P.POETX_F32, None) == \
        P.POETX_ERR_INVALID_ARG
    assert L.poetx_dequantize_q4(F, ODD, F, 4, 128, 32, P.POETX_F32, None) == P.POETX_ERR_ALIGN
    assert L.poetx_dequantize_q4(F, F, F, 4, 128, 32, 5, None) == P.POETX_ERR_DTYPE


def test_q4_product_refusals():
    L = P.lib()
    mm = lambda x=F, q=F, s=F, y=F2, T=3, m=7, n=256, g=128, tr=0: (  # noqa: E731
        L.poetx_matmul_q4(x, q, s, y, T, m, n, g, tr, None))
    assert mm(tr=2) == P.POETX_ERR_INVALID_ARG
    assert mm(T=-1) == P.POETX_ERR_INVALID_ARG
    assert mm(m=0) == P.POETX_ERR_INVALID_ARG
    assert mm(n=0) == P.POETX_ERR_INVALID_ARG
    assert mm(n=130) == P.POETX_ERR_SHAPE
    assert mm(g=256) == P.POETX_ERR_SHAPE
    assert mm(y=F) == P.POETX_ERR_INVALID_ARG                # y is x
    assert mm(s=None) == P.POETX_ERR_INVALID_ARG
    assert mm(x=ODD) == P.POETX_ERR_ALIGN
    assert mm(T=0) == P.POETX_OK


def _drop(p=0.1, row0=0, step=None):
    return P.DropoutDesc(p, 1, 0, row0, step)


def test_dropout_refusals():
    L = P.lib()

    def call(d=_drop(), i=F, o=F, rows=4, cols=8, dt=P.POETX_F32):
        return L.poetx_dropout(None if d is None else ctypes.byref(d), i, o, rows, cols, dt, None)

    assert call(d=None) == P.POETX_ERR_INVALID_ARG
    for p in (-0.1, 1.0, float("nan"), float("inf"), 0.99999):
        assert call(d=_drop(p)) == P.POETX_ERR_INVALID_ARG
    assert call(d=_drop(row0=0xFFFFFFFF), rows=2) == P.POETX_ERR_INVALID_ARG
    assert call(d=_drop(step=0x1004)) == P.POETX_ERR_ALIGN
    assert call(dt=3) == P.POETX_ERR_DTYPE
    assert call(rows=-1) == P.POETX_ERR_INVALID_ARG
    assert call(i=None) == P.POETX_ERR_INVALID_ARG
    assert call(o=ODD) == P.POETX_ERR_ALIGN
    assert call(rows=0) == P.POETX_OK and call(cols=0) == P.POETX_OK
    assert call(rows=1 << 30) == P.POETX_ERR_SHAPE and call(cols=1 << 30) == P.POETX_ERR_SHAPE

    def perm(d=_drop(), i=F, o=F2, idx=F, mode=0):
        return L.poetx_permute_cols_dropout(ctypes.byref(d), i, o, idx, 4, 8, mode, P.POETX_F32,
                                            None)

    assert perm(mode=2) == P.POETX_ERR_INVALID_ARG
    assert perm(o=F) == P.POETX_ERR_INVALID_ARG              # in place
    assert perm(idx=None) == P.POETX_ERR_INVALID_ARG
    assert perm(idx=ODD) == P.POETX_ERR_ALIGN
    assert perm(d=_drop(2.0)) == P.POETX_ERR_INVALID_ARG


def test_layer_ex_refusals():
    L = P.lib()
    f, ws = F, ctypes.c_void_p(0x40000)
    q4 = P.LinearWeight(P.POETX_WEIGHT_Q4, 64, F.value, F.value)

    def fwd(d, w=q4, drop=None, ws_bytes=BIG, x=f):
        return L.poetx_linear_fwd_ex(ctypes.byref(d) if d else None, ctypes.byref(w) if w else None,
                                     ctypes.byref(drop) if drop else None, x, f, f, f, None, None,
                                     ws, ws_bytes, None)

    def bwd(d, w=q4, drop=None, acc=0):
        return L.poetx_linear_bwd_ex(ctypes.byref(d), ctypes.byref(w),
                                     ctypes.byref(drop) if drop else None, f, f, f, f, f, f, f, f,
                                     f, acc, ws, 16, None)

    d = _desc()
    assert fwd(None) == P.POETX_ERR_INVALID_ARG
    assert fwd(d, w=None) == P.POETX_ERR_INVALID_ARG
    assert fwd(d, w=P.LinearWeight(7, 64, F.value, F.value)) == P.POETX_ERR_INVALID_ARG
    assert fwd(d, w=P.LinearWeight(2, 48, F.value, F.value)) == P.POETX_ERR_SHAPE
    assert fwd(d, w=P.LinearWeight(2, 64, None, F.value)) == P.POETX_ERR_INVALID_ARG
    assert fwd(d, w=P.LinearWeight(2, 64, F.value, ODD.value)) == P.POETX_ERR_ALIGN
    assert fwd(d, w=P.LinearWeight(1, 0, F.value, None)) == P.POETX_ERR_INVALID_ARG
    assert fwd(d, w=P.LinearWeight(0, 0, None, None)) == P.POETX_ERR_INVALID_ARG
    assert fwd(_desc(dtype=P.POETX_F32)) == P.POETX_ERR_DTYPE
    assert fwd(d, drop=_drop(1.5)) == P.POETX_ERR_INVALID_ARG
    assert fwd(d, drop=_drop(row0=0xFFFFFFF0)) == P.POETX_ERR_INVALID_ARG
    assert fwd(d, ws_bytes=16) == P.POETX_ERR_WORKSPACE
    assert fwd(d, x=None) == P.POETX_ERR_INVALID_ARG
    assert fwd(_desc(T=0)) == P.POETX_OK
    assert bwd(d) == P.POETX_ERR_WORKSPACE
    assert bwd(d, acc=3) == P.POETX_ERR_INVALID_ARG
    assert bwd(d, drop=_drop(-1.0)) == P.POETX_ERR_INVALID_ARG
    big = _desc(T=8192, n=2048, m=2048, b=256)
    assert P.linear_ex_workspace(big, q4) >= max(P.linear_fwd_workspace(big),
                                                 P.linear_bwd_workspace(big))
    q8 = P.LinearWeight(P.POETX_WEIGHT_Q8, 0, F.value, F.value)
    assert P.linear_ex_workspace(big, q8) == P.linear_ex_workspace(big, q4) + \
        P.linear_q8_scratch(big)
    few = _desc(T=4)  # a few tokens: the second halves of V and W
    dense = P.LinearWeight(P.POETX_WEIGHT_DENSE, 0, F.value, None)
    assert P.linear_ex_workspace(few, q4) >= P.linear_ex_workspace(few, dense) + \
        4 * 2 * (few.n + few.m)


def test_python_refusals_before_any_device_work():
    with pytest.raises(ValueError):
        P.q4_shapes(4, 100, 32)
    with pytest.raises(ValueError):
        P.q4_shapes(4, 128, 16)
    assert P.q4_shapes(4, 256, 32) == ((2, 4, 64), (2, 4, 4))
    with pytest.raises(ValueError):
        P.dropout_desc(0.1, 1, site=-1)
    with pytest.raises(ValueError):
        P.dropout_desc(0.1, 1, row0=1 << 32)
    with pytest.raises(ValueError):
        P.PoetxLinear.__init__(object.__new__(P.PoetxLinear), type("W", (), {"shape": (4, 4)}),
                               None, None, [0, 1, 2, 3], [0, 1, 2, 3], 2, 4, 8, int8_weight=True,
                               int4_group=64)
    # a seed of any sign and size is taken modulo 2^64
    assert P.dropout_desc(0.1, -1).seed == 2 ** 64 - 1
