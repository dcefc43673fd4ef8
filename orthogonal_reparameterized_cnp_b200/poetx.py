"""Thin ctypes binding of libpoetx (the C ABI declared in include/poetx.h).

Argument marshalling only: tensors are passed as raw device pointers, the stream as the
torch stream handle.  Every step of the layer runs in the library's CUDA kernels; there is
no fallback.  A missing library or a call without a CUDA device raises immediately.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpoetx.so")

POETX_OK = 0
POETX_ERR_INVALID_ARG = 1
POETX_ERR_SHAPE = 2
POETX_ERR_DTYPE = 3
POETX_ERR_ALIGN = 4
POETX_ERR_WORKSPACE = 5
POETX_ERR_CUDA = 6
POETX_ERR_TIMEOUT = 7

POETX_F32 = 0
POETX_BF16 = 1

_c_int = ctypes.c_int
_c_i32 = ctypes.c_int32
_c_u64 = ctypes.c_uint64
_c_size = ctypes.c_size_t
_vp = ctypes.c_void_p
_i32p = ctypes.POINTER(ctypes.c_int32)


class LinearDesc(ctypes.Structure):
    _fields_ = [("T", _c_i32), ("n", _c_i32), ("m", _c_i32), ("b", _c_i32), ("dtype", _c_i32),
                ("perm_P", _vp), ("inv_P", _vp), ("perm_R", _vp), ("inv_R", _vp)]


class DropoutDesc(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", _c_u64), ("site", ctypes.c_uint32),
                ("row0", ctypes.c_uint32), ("step", _vp)]
    keep = None  # the tensor of the step counter (dropout_desc)


POETX_WEIGHT_DENSE = 0
POETX_WEIGHT_Q8 = 1
POETX_WEIGHT_Q4 = 2


class LinearWeight(ctypes.Structure):
    _fields_ = [("kind", _c_i32), ("group", _c_i32), ("w", _vp), ("scales", _vp)]
    keep = ()  # the tensors of the weight (linear_weight_dense, _q8, _q4), on one device
    device = -1
    fits = None  # the (m, n, dtype) and addresses with which they were checked last


_descp = ctypes.POINTER(LinearDesc)
_dropp = ctypes.POINTER(DropoutDesc)
_weightp = ctypes.POINTER(LinearWeight)

# name -> (restype, argtypes); the same list is checked against include/poetx.h by the tests
SIGNATURES = {
    "poetx_status_string": (ctypes.c_char_p, [_c_int]),
    "poetx_last_error": (ctypes.c_char_p, []),
    "poetx_version": (ctypes.c_char_p, []),
    "poetx_make_perm": (_c_int, [_c_u64, _c_i32, _i32p, _i32p]),
    "poetx_invert_perm": (_c_int, [_i32p, _c_i32, _i32p]),
    "poetx_merge_perm": (_c_int, [_vp, _vp, _c_i32, _c_i32, _vp, _vp, _c_int, _vp]),
    "poetx_permute_cols": (_c_int, [_vp, _vp, _vp, _c_i32, _c_i32, _c_int, _vp]),
    "poetx_outer_merge_workspace": (_c_size, [_c_i32, _c_i32, _c_int]),
    "poetx_outer_merge": (_c_int, [_vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _vp, _vp, _vp, _vp,
                                   _vp, _c_int, _vp, _c_size, _vp]),
    "poetx_cnp_workspace": (_c_size, [_c_i32, _c_i32, _c_i32]),
    "poetx_cnp_fwd": (_c_int, [_vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _vp, _c_size, _vp]),
    "poetx_cnp_bwd": (_c_int, [_vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _vp, _c_size, _vp]),
    "poetx_cnp_fwd_static": (_c_int, [_vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _vp]),
    "poetx_cnp_fwd_save": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _vp,
                                    _c_size, _vp]),
    "poetx_cnp_bwd_saved": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _vp,
                                     _c_size, _vp]),
    "poetx_linear_fwd_workspace": (_c_size, [ctypes.POINTER(LinearDesc), _c_int, _c_int]),
    "poetx_linear_bwd_workspace": (_c_size, [ctypes.POINTER(LinearDesc), _c_int, _c_int]),
    "poetx_linear_fwd": (_c_int, [ctypes.POINTER(LinearDesc), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _c_size, _vp]),
    "poetx_linear_bwd": (_c_int, [ctypes.POINTER(LinearDesc), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _c_int, _vp, _c_size, _vp]),
    "poetx_device_status": (_c_int, [_vp]),
    "poetx_set_wait_limit": (_c_int, [_c_u64, ctypes.POINTER(_c_u64)]),
    "poetx_set_gemm_pairs": (_c_int, [_c_int, ctypes.POINTER(_c_int)]),
    "poetx_selftest_wait_timeout": (_c_int, [_vp, _vp, _c_i32, _c_i32, _c_i32, _vp, _c_size,
                                             _vp]),
    "poetx_fma_probe": (_c_int, [_vp, _c_i32, _c_i32, _vp]),
    "poetx_quantize_rows": (_c_int, [_vp, _vp, _vp, _c_i32, _c_i32, _c_int, _vp]),
    "poetx_merge_perm_q8": (_c_int, [_vp, _vp, _vp, _c_i32, _c_i32, _vp, _vp, _c_int, _vp]),
    "poetx_linear_q8_scratch": (_c_size, [ctypes.POINTER(LinearDesc)]),
    "poetx_linear_fwd_q8": (_c_int, [ctypes.POINTER(LinearDesc), _vp, _vp, _vp, _vp, _vp, _vp,
                                     _vp, _vp, _vp, _c_size, _vp]),
    "poetx_linear_bwd_q8": (_c_int, [ctypes.POINTER(LinearDesc), _vp, _vp, _vp, _vp, _vp, _vp,
                                     _vp, _vp, _vp, _vp, _vp, _c_int, _vp, _c_size, _vp]),
    "poetx_quantize_q4": (_c_int, [_vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _c_int, _vp]),
    "poetx_merge_perm_q4": (_c_int, [_vp, _vp, _vp, _c_i32, _c_i32, _vp, _vp, _c_i32, _c_int,
                                     _vp]),
    "poetx_dequantize_q4": (_c_int, [_vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _c_int, _vp]),
    "poetx_matmul_q4": (_c_int, [_vp, _vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _c_i32, _c_int,
                                 _vp]),
    "poetx_dropout": (_c_int, [_dropp, _vp, _vp, _c_i32, _c_i32, _c_int, _vp]),
    "poetx_permute_cols_dropout": (_c_int, [_dropp, _vp, _vp, _vp, _c_i32, _c_i32, _c_int,
                                            _c_int, _vp]),
    "poetx_linear_ex_workspace": (_c_size, [_descp, _weightp, _c_int, _c_int]),
    "poetx_linear_fwd_ex": (_c_int, [_descp, _weightp, _dropp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _c_size, _vp]),
    "poetx_linear_bwd_ex": (_c_int, [_descp, _weightp, _dropp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _vp, _vp, _c_int, _vp, _c_size, _vp]),
    "poetx_launch_count": (_c_u64, []),
    "poetx_profile_begin": (_c_int, [ctypes.c_char_p]),
    "poetx_profile_end": (_c_int, [_i32p, ctypes.POINTER(ctypes.c_double)]),
}

_lib = None


class PoetxError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        lib = _load()
        super().__init__(f"{where}: {lib.poetx_status_string(status).decode()} "
                         f"({status}): {lib.poetx_last_error().decode()}")


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libpoetx.so not built ({LIB_PATH}); run "
                               "`python -m orthogonal_reparameterized_cnp_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def lib():
    return _load()


def _check(status: int, where: str):
    if status != POETX_OK:
        raise PoetxError(status, where)


# ------------------------------------------------------------------------ helpers
def _ptr(t) -> int | None:
    """Device pointer of a torch tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> int | None:
    import torch
    if stream is None:  # (the raw handle: building a Stream object costs 3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return POETX_F32
    if t.dtype == torch.bfloat16:
        return POETX_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


# ------------------------------------------------------------------------ host calls
def make_perm(seed: int, n: int):
    """Seeded permutation and its inverse (numpy int32), computed by the library."""
    L = _load()
    perm = np.empty(n, dtype=np.int32)
    inv = np.empty(n, dtype=np.int32)
    _check(L.poetx_make_perm(seed & ((1 << 64) - 1), n,
                             perm.ctypes.data_as(_i32p), inv.ctypes.data_as(_i32p)),
           "poetx_make_perm")
    return perm, inv


def invert_perm(perm) -> np.ndarray:
    """Inverse of an index map (numpy int32), computed and validated by the library: a map
    that is not a bijection of range(n) raises PoetxError (POETX_ERR_INVALID_ARG)."""
    L = _load()
    p = np.ascontiguousarray(np.asarray(perm), dtype=np.int32)
    if p.ndim != 1:
        raise ValueError("an index map is a 1-D array")
    inv = np.empty_like(p)
    _check(L.poetx_invert_perm(p.ctypes.data_as(_i32p), len(p), inv.ctypes.data_as(_i32p)),
           "poetx_invert_perm")
    return inv


def set_wait_limit(ns: int) -> int:
    """Sets the kernels' bounded-wait limit (0: the 2 s default); returns the previous one."""
    prev = _c_u64(0)
    _check(_load().poetx_set_wait_limit(int(ns), ctypes.byref(prev)), "poetx_set_wait_limit")
    return int(prev.value)


def set_gemm_pairs(enable: bool) -> bool:
    """Merged-weight GEMMs on CTA pairs (True, the default) or single CTAs; returns the
    previous setting."""
    prev = ctypes.c_int(0)
    _check(_load().poetx_set_gemm_pairs(int(bool(enable)), ctypes.byref(prev)),
           "poetx_set_gemm_pairs")
    return bool(prev.value)


def cnp_workspace(nblk: int, b: int, k: int) -> int:
    return int(_load().poetx_cnp_workspace(nblk, b, k))


def linear_desc(T, n, m, b, dtype_code, perm_P, inv_P, perm_R, inv_R) -> LinearDesc:
    return LinearDesc(T, n, m, b, dtype_code, _ptr(perm_P), _ptr(inv_P), _ptr(perm_R),
                      _ptr(inv_R))


def linear_fwd_workspace(desc: LinearDesc, has_save_u=True, has_save_w=True) -> int:
    return int(_load().poetx_linear_fwd_workspace(ctypes.byref(desc), int(has_save_u),
                                                  int(has_save_w)))


def linear_bwd_workspace(desc: LinearDesc, has_save_u=True, has_save_w=True) -> int:
    return int(_load().poetx_linear_bwd_workspace(ctypes.byref(desc), int(has_save_u),
                                                  int(has_save_w)))


def launch_count() -> int:
    return int(_load().poetx_launch_count())


def profile_begin(name: str | None):
    _check(_load().poetx_profile_begin(name.encode() if name else None), "poetx_profile_begin")


def profile_end():
    n = ctypes.c_int32(0)
    ms = ctypes.c_double(0.0)
    _check(_load().poetx_profile_end(ctypes.byref(n), ctypes.byref(ms)), "poetx_profile_end")
    return int(n.value), float(ms.value)


# ------------------------------------------------------------------------ device calls
def _require_cuda():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("libpoetx needs a CUDA device (sm_100a); none is available")


def merge_perm(W0, W0p, perm_R, perm_P, stream=None):
    _require_cuda()
    m, n = W0.shape
    _check(_load().poetx_merge_perm(_ptr(W0), _ptr(W0p), m, n, _ptr(perm_R), _ptr(perm_P),
                                    _dtype_code(W0), _stream(stream)), "poetx_merge_perm")


def outer_merge_workspace(m: int, n: int, dtype_code: int) -> int:
    return int(_load().poetx_outer_merge_workspace(m, n, dtype_code))


def outer_merge(W0p, G_P, G_R, b: int, inv_P, inv_R, perm_P_new, perm_R_new, W0p_new, ws,
                stream=None):
    """W0p_new = merged weight, under the new permutations, of R W0 P (see the header)."""
    _require_cuda()
    m, n = W0p.shape
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().poetx_outer_merge(_ptr(W0p), _ptr(G_P), _ptr(G_R), m, n, b, _ptr(inv_P),
                                     _ptr(inv_R), _ptr(perm_P_new), _ptr(perm_R_new),
                                     _ptr(W0p_new), _dtype_code(W0p), _ptr(ws), ws_bytes,
                                     _stream(stream)), "poetx_outer_merge")


def permute_cols(x, out, idx, stream=None):
    _require_cuda()
    rows, cols = x.shape
    _check(_load().poetx_permute_cols(_ptr(x), _ptr(out), _ptr(idx), rows, cols, _dtype_code(x),
                                      _stream(stream)), "poetx_permute_cols")


def cnp_fwd(theta, G, G_bf16, b: int, k: int, ws, stream=None):
    _require_cuda()
    nblk = theta.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().poetx_cnp_fwd(_ptr(theta), _ptr(G), _ptr(G_bf16), nblk, b, k, _ptr(ws),
                                 ws_bytes, _stream(stream)), "poetx_cnp_fwd")


def cnp_fwd_static(theta, G, G_bf16, b: int, k: int, stream=None):
    """CNP forward with the library's fixed device scratch (no caller buffer; see the
    header for the size limit and the sharing rules)."""
    _require_cuda()
    nblk = theta.shape[0]
    _check(_load().poetx_cnp_fwd_static(_ptr(theta), _ptr(G), _ptr(G_bf16), nblk, b, k,
                                        _stream(stream)), "poetx_cnp_fwd_static")


def cnp_bwd(theta, dG, dtheta, b: int, k: int, ws, stream=None):
    _require_cuda()
    nblk = theta.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().poetx_cnp_bwd(_ptr(theta), _ptr(dG), _ptr(dtheta), nblk, b, k, _ptr(ws),
                                 ws_bytes, _stream(stream)), "poetx_cnp_bwd")


def cnp_fwd_save(theta, G, G_bf16, Q_save, S_save, F_save, b: int, k: int, ws, stream=None):
    """CNP forward that also keeps Q, S = Q^2 and F' for poetx_cnp_bwd_saved."""
    _require_cuda()
    nblk = theta.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().poetx_cnp_fwd_save(_ptr(theta), _ptr(G), _ptr(G_bf16), _ptr(Q_save),
                                      _ptr(S_save), _ptr(F_save), nblk, b, k, _ptr(ws), ws_bytes,
                                      _stream(stream)), "poetx_cnp_fwd_save")


def cnp_bwd_saved(theta, dG, Q_saved, S_saved, F_saved, dtheta, b: int, k: int, ws,
                  stream=None):
    """CNP backward reading the forward's Q, S and F' (theta unchanged since)."""
    _require_cuda()
    nblk = theta.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().poetx_cnp_bwd_saved(_ptr(theta), _ptr(dG), _ptr(Q_saved), _ptr(S_saved),
                                       _ptr(F_saved), _ptr(dtheta), nblk, b, k, _ptr(ws),
                                       ws_bytes, _stream(stream)), "poetx_cnp_bwd_saved")


def linear_fwd(desc: LinearDesc, x, G_P, G_R, W0p, y, save_u, save_w, ws, stream=None):
    _require_cuda()
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().poetx_linear_fwd(ctypes.byref(desc), _ptr(x), _ptr(G_P), _ptr(G_R),
                                    _ptr(W0p), _ptr(y), _ptr(save_u), _ptr(save_w), _ptr(ws),
                                    ws_bytes, _stream(stream)), "poetx_linear_fwd")


def linear_bwd(desc: LinearDesc, x, dy, G_P, G_R, W0p, save_u, save_w, dx, dG_P, dG_R,
               accumulate: int, ws, stream=None):
    _require_cuda()
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().poetx_linear_bwd(ctypes.byref(desc), _ptr(x), _ptr(dy), _ptr(G_P), _ptr(G_R),
                                    _ptr(W0p), _ptr(save_u), _ptr(save_w), _ptr(dx), _ptr(dG_P),
                                    _ptr(dG_R), int(accumulate), _ptr(ws), ws_bytes,
                                    _stream(stream)), "poetx_linear_bwd")


def quantize_rows(W, q, scales, stream=None):
    """Per-row symmetric int8 codes and fp32 scales of W (see the header)."""
    _require_cuda()
    m, n = W.shape
    _check(_load().poetx_quantize_rows(_ptr(W), _ptr(q), _ptr(scales), m, n, _dtype_code(W),
                                       _stream(stream)), "poetx_quantize_rows")


def merge_perm_q8(W0, q, scales, perm_R, perm_P, stream=None):
    """Int8 codes and per-row scales of W0' = W0[perm_R][:, perm_P], without forming W0'."""
    _require_cuda()
    m, n = W0.shape
    _check(_load().poetx_merge_perm_q8(_ptr(W0), _ptr(q), _ptr(scales), m, n, _ptr(perm_R),
                                       _ptr(perm_P), _dtype_code(W0), _stream(stream)),
           "poetx_merge_perm_q8")


def linear_q8_scratch(desc: LinearDesc) -> int:
    return int(_load().poetx_linear_q8_scratch(ctypes.byref(desc)))


def linear_fwd_q8(desc: LinearDesc, x, G_P, G_R, W0q, scales, y, save_u, save_w, ws,
                  stream=None):
    _require_cuda()
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().poetx_linear_fwd_q8(ctypes.byref(desc), _ptr(x), _ptr(G_P), _ptr(G_R),
                                       _ptr(W0q), _ptr(scales), _ptr(y), _ptr(save_u),
                                       _ptr(save_w), _ptr(ws), ws_bytes, _stream(stream)),
           "poetx_linear_fwd_q8")


def linear_bwd_q8(desc: LinearDesc, x, dy, G_P, G_R, W0q, scales, save_u, save_w, dx, dG_P,
                  dG_R, accumulate: int, ws, stream=None):
    _require_cuda()
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().poetx_linear_bwd_q8(ctypes.byref(desc), _ptr(x), _ptr(dy), _ptr(G_P),
                                       _ptr(G_R), _ptr(W0q), _ptr(scales), _ptr(save_u),
                                       _ptr(save_w), _ptr(dx), _ptr(dG_P), _ptr(dG_R),
                                       accumulate, _ptr(ws), ws_bytes, _stream(stream)),
           "poetx_linear_bwd_q8")


# ------------------------------------------------------------------------ 4-bit weight
def _require(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _ptrs(*tensors):
    """Device pointers of contiguous tensors on the current device (None -> NULL); the calls below
    launch on that device's stream.  (Checked here once, in plain ifs: a decoding call's time on
    the host counts.)"""
    import torch
    dev = torch.cuda.current_device()  # (raises without a CUDA device)
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        if t.get_device() != dev:  # (-1 for a CPU tensor)
            raise ValueError(f"expected tensors on the current CUDA device ({dev}), got {t.device}")
        if not t.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        out.append(t.data_ptr())
    return out


def q4_shapes(m: int, n: int, group: int):
    """Shapes of the codes (uint8) and scales (bf16) of an m x n 4-bit weight."""
    _require(group in (32, 64, 128), "group must be 32, 64 or 128")
    _require(n % 128 == 0, "n must be a multiple of 128 (4-bit weight)")
    return (n // 128, m, 64), (n // 128, m, 128 // group)


def _check_q4(q, scales, m, n, group):
    import torch
    qs, ss = q4_shapes(m, n, group)
    if q.shape != qs or q.dtype is not torch.uint8:
        raise ValueError(f"the codes of a {m} x {n} 4-bit weight are uint8 {qs}")
    if scales.shape != ss or scales.dtype is not torch.bfloat16:
        raise ValueError(f"the scales of a {m} x {n} 4-bit weight with groups of {group} are "
                         f"bfloat16 {ss}")


def _check_map(idx, n, what):
    import torch
    if idx is not None and (idx.dtype is not torch.int32 or idx.shape != (n,)):
        raise ValueError(f"{what} must be int32 with {n} entries")


def quantize_q4(W, q, scales, group: int, stream=None):
    """4-bit codes and group scales of W (format and rounding: see the header)."""
    m, n = W.shape
    _check_q4(q, scales, m, n, group)
    _check(_load().poetx_quantize_q4(*_ptrs(W, q, scales), m, n, group, _dtype_code(W),
                                     _stream(stream)), "poetx_quantize_q4")


def merge_perm_q4(W0, q, scales, perm_R, perm_P, group: int, stream=None):
    """4-bit codes and group scales of W0' = W0[perm_R][:, perm_P], without forming W0' (both
    maps None: identity)."""
    m, n = W0.shape
    _check_q4(q, scales, m, n, group)
    _check_map(perm_R, m, "perm_R")
    _check_map(perm_P, n, "perm_P")
    w, c, sc, pR, pP = _ptrs(W0, q, scales, perm_R, perm_P)
    _check(_load().poetx_merge_perm_q4(w, c, sc, m, n, pR, pP, group, _dtype_code(W0),
                                       _stream(stream)), "poetx_merge_perm_q4")


def dequantize_q4(q, scales, out, group: int, stream=None):
    """out [m, n] (bf16 or fp32) = the weight that 4-bit codes and scales stand for."""
    m, n = out.shape
    _check_q4(q, scales, m, n, group)
    _check(_load().poetx_dequantize_q4(*_ptrs(q, scales, out), m, n, group, _dtype_code(out),
                                       _stream(stream)), "poetx_dequantize_q4")


def matmul_q4(x, q, scales, y, group: int, transpose: bool = False, stream=None):
    """y = x W^T (or, transpose, y = x W) with the 4-bit weight W [m, n]; bf16, T >= 0 rows."""
    import torch
    T, k = x.shape
    Ty, o = y.shape
    m, n = (k, o) if transpose else (o, k)
    if Ty != T:
        raise ValueError("x and y must have the same number of rows")
    if x.dtype is not torch.bfloat16 or y.dtype is not torch.bfloat16:
        raise ValueError("x and y must be bfloat16")
    _check_q4(q, scales, m, n, group)
    _check(_load().poetx_matmul_q4(*_ptrs(x, q, scales, y), T, m, n, group, 1 if transpose else 0,
                                   _stream(stream)), "poetx_matmul_q4")


# ------------------------------------------------------------------------ dropout
def dropout_desc(p: float, seed: int, site: int = 0, row0: int = 0, step=None) -> DropoutDesc:
    """Dropout settings of a call; step: a one-element int64 CUDA tensor (or None)."""
    import torch
    if step is not None:
        _require(step.dtype == torch.int64 and step.numel() == 1 and step.is_cuda,
                 "step must be a one-element int64 CUDA tensor")
    _require(0 <= site < 1 << 32 and 0 <= row0 < 1 << 32, "site and row0 are 32-bit numbers")
    d = DropoutDesc(float(p), seed & ((1 << 64) - 1), site, row0,
                    None if step is None else step.data_ptr())
    d.keep = step  # the tensor lives as long as the descriptor
    return d


def dropout(drop: DropoutDesc, x, out, stream=None):
    """out = dropout(x) (out may be x); the backward is the same call on the gradient."""
    rows, cols = x.shape
    _require(out.shape == x.shape and out.dtype == x.dtype, "out must be like x")
    a, o, _ = _ptrs(x, out, drop.keep)
    _check(_load().poetx_dropout(ctypes.byref(drop), a, o, rows, cols, _dtype_code(x),
                                 _stream(stream)), "poetx_dropout")


def permute_cols_dropout(drop: DropoutDesc, x, out, idx, mask_output: bool = False, stream=None):
    """out[:, i] = dropout(x)[:, idx[i]], or (mask_output) x[:, idx[i]] masked by the output
    column: with the inverse map, the gradient of the first form."""
    rows, cols = x.shape
    _require(out.shape == x.shape and out.dtype == x.dtype, "out must be like x")
    _check_map(idx, cols, "idx")
    a, o, i, _ = _ptrs(x, out, idx, drop.keep)
    _check(_load().poetx_permute_cols_dropout(ctypes.byref(drop), a, o, i, rows, cols,
                                              1 if mask_output else 0, _dtype_code(x),
                                              _stream(stream)), "poetx_permute_cols_dropout")


class Dropout:
    """Dropout of a layer's input: probability, seed, site and a step counter in device memory
    (read by the kernels when they run, so a replayed CUDA graph draws a new mask each time the
    counter moves).  Layers of one program share the counter and differ in ``site``; a
    data-parallel rank sets ``row0`` to the first token of its shard, so that the masks do not
    depend on the sharding."""

    def __init__(self, p: float, seed: int, site: int = 0, row0: int = 0, step=None, device=None):
        import torch
        _require(0.0 <= p <= 65535 / 65536, "p must be in [0, 65535/65536]")
        if step is None:
            step = torch.zeros(1, dtype=torch.int64, device=device or "cuda")
        self.p, self.seed, self.site, self.row0, self.step = p, seed, site, row0, step

    def at_site(self, site: int) -> "Dropout":
        """The same dropout at another site (same seed and step counter)."""
        return Dropout(self.p, self.seed, site, self.row0, self.step)

    def desc(self) -> DropoutDesc:
        return dropout_desc(self.p, self.seed, self.site, self.row0, self.step)

    def advance(self, stream=None):
        """Moves the step counter (on `stream`): the next forward draws a new mask."""
        import torch
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            self.step.add_(1)


# ------------------------------------------------------------------------ layer, any weight
def _hold(w: LinearWeight, *tensors) -> LinearWeight:
    w.keep, w.device = tensors, tensors[0].get_device()
    for t in tensors:
        if t.get_device() != w.device:
            raise ValueError("the tensors of a weight must be on one device")
    return w


def linear_weight_dense(W0p) -> LinearWeight:
    return _hold(LinearWeight(POETX_WEIGHT_DENSE, 0, _ptr(W0p), None), W0p)


def linear_weight_q8(W0q, scales) -> LinearWeight:
    return _hold(LinearWeight(POETX_WEIGHT_Q8, 0, _ptr(W0q), _ptr(scales)), W0q, scales)


def linear_weight_q4(W0q, scales, group: int) -> LinearWeight:
    return _hold(LinearWeight(POETX_WEIGHT_Q4, group, _ptr(W0q), _ptr(scales)), W0q, scales)


def _check_weight(desc: LinearDesc, w: LinearWeight):
    """(Once for a weight and layer: the weight holds its tensors.)  A tensor whose storage was
    exchanged since (``tensor.data = ...``) is checked and pointed to anew."""
    if not w.keep:
        raise ValueError("a weight comes from linear_weight_dense, linear_weight_q8 or "
                         "linear_weight_q4")
    at, end = w.keep[0].data_ptr(), w.keep[-1].data_ptr()
    fits = (desc.m, desc.n, desc.dtype, at, end)
    if w.fits == fits:
        return
    if w.w != at or (w.scales or at) != end:
        for t, field in zip(w.keep, ("w", "scales")):
            if t.get_device() != w.device:
                raise ValueError("the tensors of a weight must be on one device")
            setattr(w, field, _ptr(t))
    if w.kind == POETX_WEIGHT_Q4:
        _check_q4(*w.keep, desc.m, desc.n, w.group)
    elif w.kind == POETX_WEIGHT_Q8:
        import torch
        q, s = w.keep
        _require(tuple(q.shape) == (desc.m, desc.n) and q.dtype == torch.int8 and
                 tuple(s.shape) == (desc.m,) and s.dtype == torch.float32,
                 "the int8 weight is int8 [m, n] with float32 scales [m]")
    else:
        _require(tuple(w.keep[0].shape) == (desc.m, desc.n) and
                 _dtype_code(w.keep[0]) == desc.dtype, "the merged weight is [m, n], of the "
                 "layer's type")
    w.fits = fits


def _check_device(w: LinearWeight, x):
    if w.device != x.get_device():
        raise ValueError(f"the weight is on CUDA device {w.device}, x on {x.device}")


def _drop_ref(drop):
    return None if drop is None else ctypes.byref(drop)


def linear_ex_workspace(desc: LinearDesc, weight: LinearWeight, has_save_u=True,
                        has_save_w=True) -> int:
    """Scratch bytes of linear_fwd_ex and linear_bwd_ex (the larger of the two)."""
    return int(_load().poetx_linear_ex_workspace(ctypes.byref(desc), ctypes.byref(weight),
                                                 int(has_save_u), int(has_save_w)))


def _check_layer(desc, weight, outer, G_P, G_R):
    """outer: pairs of a tensor [T, width] and its width (the tensor None: not given)."""
    import torch
    _check_weight(desc, weight)
    T, dt = desc.T, torch.bfloat16 if desc.dtype == POETX_BF16 else torch.float32
    for t, width in outer:
        if t is not None and (t.shape != (T, width) or t.dtype is not dt):
            raise ValueError(f"expected a {dt} tensor [{T}, {width}], got {t.dtype} "
                             f"{list(t.shape)}")
    for t, width in ((G_P, desc.n), (G_R, desc.m)):
        if t.numel() != width * desc.b or t.dtype is not dt:
            raise ValueError(f"G_P and G_R are {dt}, [n/b, b, b] and [m/b, b, b]")


def linear_fwd_ex(desc: LinearDesc, weight: LinearWeight, drop, x, G_P, G_R, y, save_u, save_w,
                  ws, stream=None):
    """Layer forward on any form of the merged weight, with dropout of x (drop or None)."""
    n, m = desc.n, desc.m
    _check_layer(desc, weight, ((x, n), (y, m), (save_u, n), (save_w, m)), G_P, G_R)
    ptrs = _ptrs(x, G_P, G_R, y, save_u, save_w, ws, None if drop is None else drop.keep)
    _check_device(weight, x)
    _check(_load().poetx_linear_fwd_ex(ctypes.byref(desc), ctypes.byref(weight), _drop_ref(drop),
                                       *ptrs[:7], 0 if ws is None else ws.nbytes,
                                       _stream(stream)), "poetx_linear_fwd_ex")


def linear_bwd_ex(desc: LinearDesc, weight: LinearWeight, drop, x, dy, G_P, G_R, save_u, save_w,
                  dx, dG_P, dG_R, accumulate: int, ws, stream=None):
    """Layer backward on any form of the merged weight; drop as in the forward."""
    import torch
    n, m = desc.n, desc.m
    _check_layer(desc, weight, ((x, n), (dy, m), (save_u, n), (save_w, m), (dx, n)), G_P, G_R)
    for t, G in ((dG_P, G_P), (dG_R, G_R)):
        if t.numel() != G.numel() or t.dtype is not torch.float32:
            raise ValueError("dG_P and dG_R are float32, [n/b, b, b] and [m/b, b, b]")
    ptrs = _ptrs(x, dy, G_P, G_R, save_u, save_w, dx, dG_P, dG_R, ws,
                 None if drop is None else drop.keep)
    _check_device(weight, dy)
    _check(_load().poetx_linear_bwd_ex(ctypes.byref(desc), ctypes.byref(weight), _drop_ref(drop),
                                       *ptrs[:9], int(accumulate), ptrs[9],
                                       0 if ws is None else ws.nbytes, _stream(stream)),
           "poetx_linear_bwd_ex")


def selftest_wait_timeout(theta, G, b: int, k: int, ws, stream=None):
    """Runs the CNP forward with a dependency that is never met (see the header)."""
    _require_cuda()
    nblk = theta.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_load().poetx_selftest_wait_timeout(_ptr(theta), _ptr(G), nblk, b, k, _ptr(ws),
                                               ws_bytes, _stream(stream)),
           "poetx_selftest_wait_timeout")


def fma_probe(out, ctas: int, iters: int, stream=None):
    """FP32 FMA throughput probe: ctas * 512 * 16 * iters * 2 FLOPs into out[ctas * 512]."""
    _require_cuda()
    _check(_load().poetx_fma_probe(_ptr(out), ctas, iters, _stream(stream)), "poetx_fma_probe")


def device_status(stream=None) -> int:
    _require_cuda()
    return int(_load().poetx_device_status(_stream(stream)))


# ------------------------------------------------------------------------ layer objects
class CnpBuffers:
    """Device buffers of the Cayley-Neumann parameterisation of nblk b x b blocks: theta,
    G (fp32 and, for the bf16 layer, its bf16 copy), the upstream dG, dtheta, and the Q,
    S = Q^2 and F' that the forward keeps for the backward.  One forward call and one
    backward call cover every block, whichever layers the blocks belong to."""

    def __init__(self, nblk: int, b: int, k: int, device, lowp_dtype=None):
        import torch
        self.nblk, self.b, self.k = nblk, b, k
        f32 = dict(dtype=torch.float32, device=device)
        ntri = b * (b - 1) // 2
        self.theta = torch.zeros((nblk, ntri), **f32)
        self.G = torch.empty((nblk, b, b), **f32)
        self.G_lp = torch.empty((nblk, b, b), dtype=lowp_dtype, device=device) \
            if lowp_dtype is not None else None
        self.dG = torch.zeros((nblk, b, b), **f32)
        self.dtheta = torch.empty((nblk, ntri), **f32)
        self.Q_save = torch.empty((nblk, b, b), **f32)
        self.S_save = torch.empty((nblk, b, b), **f32)
        self.F_save = torch.empty((nblk, b, b), **f32)
        self.ws = None
        self.set_order(k)

    def set_order(self, k: int):
        """Neumann order of the following calls (the scratch is resized to it)."""
        import torch
        self.k = k
        self.ws = None
        self.ws = torch.empty(max(cnp_workspace(self.nblk, self.b, k), 16), dtype=torch.uint8,
                              device=self.G.device)

    def forward(self, stream=None):
        cnp_fwd_save(self.theta, self.G, self.G_lp, self.Q_save, self.S_save, self.F_save,
                     self.b, self.k, self.ws, stream)

    def backward(self, stream=None):
        """dtheta from dG; reads the Q, S and F' of the last forward (theta unchanged)."""
        cnp_bwd_saved(self.theta, self.dG, self.Q_save, self.S_save, self.F_save, self.dtheta,
                      self.b, self.k, self.ws, stream)


def _layer_scratch_bytes(desc, save: bool, int8: bool, int4_group: int = 0) -> int:
    if int4_group:
        w = LinearWeight(POETX_WEIGHT_Q4, int4_group, None, None)
        return max(linear_ex_workspace(desc, w, save, save), 16)
    q8 = linear_q8_scratch(desc) if int8 else 0
    return max(linear_fwd_workspace(desc, save, save), linear_bwd_workspace(desc, save, save),
               16) + q8


class PoetxLinear:
    """One POET-X linear on the GPU: merged weight, CNP blocks, forward and backward.

    All buffers are torch tensors on the current device; every computation is a libpoetx
    call.  The CNP blocks are the input-side blocks first, then the output-side blocks, in
    ``cnp`` (a CnpBuffers of this layer alone unless one is shared, see PoetxLinearGroup);
    ``theta``, ``G``, ``dG``, ``dtheta`` are this layer's rows of it.  The inverse index
    maps come from the library, which rejects a perm_P or perm_R that is not a bijection.
    The permutations are merged into W0' once, at construction (and again by merge(), which W0
    is kept for: a layer that is done merging gives it up with ``layer.W0 = None``).

    The merged weight is kept in W0's type, in int8 (int8_weight) or in 4 bits with a scale per
    int4_group (32, 64 or 128) columns: ``W0p``, or ``W0q`` and ``scales``, which are the tensors of
    ``weight``, the one that every call reads.  Another tensor may be assigned to each (of the same
    shape, type and device, contiguous).  dropout (a Dropout) acts on the layer's input while
    ``training`` is true; step() moves its counter.

    W0's type is that of every tensor of the layer, those between its products included: a float32
    layer rounds nothing to fewer bits, a bfloat16 one each product once (sums are fp32).

    T is the largest number of tokens (rows) of a call: forward(), backward() and step() also take
    fewer, a last ragged batch or the few tokens of decoding, with the same weight.  A backward
    takes as many as the forward before it.
    """

    def __init__(self, W0, theta_P, theta_R, perm_P, perm_R, b: int, k: int, T: int,
                 save_activations: bool = True, int8_weight: bool = False, cnp=None,
                 first_block: int = 0, ws=None, int4_group: int = 0, dropout=None):
        import torch
        self.m, self.n = W0.shape
        if int8_weight and int4_group:
            raise ValueError("the merged weight is either int8 or 4-bit")
        # the index maps are checked (bijections) and inverted by the library, on the host,
        # before any device work
        pP = np.ascontiguousarray(np.asarray(perm_P), dtype=np.int32)
        pR = np.ascontiguousarray(np.asarray(perm_R), dtype=np.int32)
        if pP.shape != (self.n,) or pR.shape != (self.m,):
            raise ValueError("perm_P must have n entries and perm_R m entries")
        iP, iR = invert_perm(pP), invert_perm(pR)
        _require_cuda()
        dev = W0.device
        self.b, self.k, self.T = b, k, T
        self.bf16 = W0.dtype == torch.bfloat16
        self.nP, self.nR = self.n // b, self.m // b
        nblk = self.nP + self.nR
        i32 = dict(dtype=torch.int32, device=dev)
        self.perm_P, self.inv_P = torch.as_tensor(pP, **i32), torch.as_tensor(iP, **i32)
        self.perm_R, self.inv_R = torch.as_tensor(pR, **i32), torch.as_tensor(iR, **i32)
        self.W0 = W0
        if cnp is None:
            cnp = CnpBuffers(nblk, b, k, dev, W0.dtype if self.bf16 else None)
            first_block = 0
        if cnp.b != b or cnp.k != k or first_block + nblk > cnp.nblk:
            raise ValueError("the CNP buffers do not hold this layer's blocks")
        self.cnp = cnp
        rows = slice(first_block, first_block + nblk)
        self.theta, self.G, self.dG, self.dtheta = (cnp.theta[rows], cnp.G[rows], cnp.dG[rows],
                                                    cnp.dtheta[rows])
        self.G_lp = cnp.G_lp[rows] if cnp.G_lp is not None else None
        self.theta[: self.nP] = theta_P
        self.theta[self.nP:] = theta_R
        self.desc = linear_desc(T, self.n, self.m, b, POETX_BF16 if self.bf16 else POETX_F32,
                                self.perm_P, self.inv_P, self.perm_R, self.inv_R)
        act = W0.dtype
        self.save = save_activations
        if save_activations:
            self.U = torch.empty((T, self.n), dtype=act, device=dev)
            self.Wsave = torch.empty((T, self.m), dtype=act, device=dev)
        else:
            self.U = self.Wsave = None
        # int8 merged weight (POET-XQ): codes + per-row scales; the bf16 weight exists only
        # inside each layer call's scratch
        self.int8 = int8_weight
        if int8_weight:
            if not self.bf16:
                raise ValueError("the int8 base weight needs the bf16 layer")
            self.weight = linear_weight_q8(
                torch.empty((self.m, self.n), dtype=torch.int8, device=dev),
                torch.empty((self.m,), dtype=torch.float32, device=dev))
        # 4-bit merged weight: codes + group scales (bf16)
        self.int4_group = int4_group
        if int4_group:
            if not self.bf16:
                raise ValueError("the 4-bit base weight needs the bf16 layer")
            qs, ss = q4_shapes(self.m, self.n, int4_group)
            self.weight = linear_weight_q4(torch.empty(qs, dtype=torch.uint8, device=dev),
                                           torch.empty(ss, dtype=torch.bfloat16, device=dev),
                                           int4_group)
        if not int8_weight and not int4_group:
            self.weight = linear_weight_dense(torch.empty_like(W0))
        self.dropout = dropout
        self.training = True
        need = _layer_scratch_bytes(self.desc, self.save, int8_weight, int4_group)
        if ws is None:
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
        elif ws.numel() * ws.element_size() < need:
            raise ValueError("shared layer scratch too small")
        self.ws = ws
        self._fewer = {}  # descriptor and scratch by number of tokens (below T)
        self.merge()

    # The merged weight has one holder, `weight`; these are its tensors by name.
    def _weight_tensor(self, i: int, coded: bool):
        return self.weight.keep[i] if (self.weight.kind != POETX_WEIGHT_DENSE) == coded else None

    def _replace_weight(self, i: int, coded: bool, t):
        kind = self.weight.kind
        if t is None and self._weight_tensor(i, coded) is None:
            return
        if t is None or (kind != POETX_WEIGHT_DENSE) != coded:
            raise ValueError("the merged weight is W0p (a layer in W0's type), or W0q and scales "
                             "(int8, 4 bits)")
        if t.get_device() != self.weight.device:
            raise ValueError(f"the merged weight is on CUDA device {self.weight.device}")
        keep = list(self.weight.keep)
        keep[i] = t
        w = (linear_weight_q4(*keep, self.int4_group) if kind == POETX_WEIGHT_Q4 else
             linear_weight_q8(*keep) if kind == POETX_WEIGHT_Q8 else linear_weight_dense(*keep))
        _check_weight(self.desc, w)
        self.weight = w

    @property
    def W0p(self):
        """The merged weight in W0's type; None in the int8 and 4-bit forms."""
        return self._weight_tensor(0, False)

    @W0p.setter
    def W0p(self, t):
        self._replace_weight(0, False, t)

    @property
    def W0q(self):
        """The codes of the int8 or 4-bit merged weight."""
        return self._weight_tensor(0, True)

    @W0q.setter
    def W0q(self, t):
        self._replace_weight(0, True, t)

    @property
    def scales(self):
        """The scales of the int8 or 4-bit merged weight."""
        return self._weight_tensor(1, True)

    @scales.setter
    def scales(self, t):
        self._replace_weight(1, True, t)

    def _drop(self):
        """Descriptor of the active dropout, or None."""
        return self.dropout.desc() if self.dropout is not None and self.training else None

    def G_ops(self):
        G = self.G_lp if self.bf16 else self.G
        return G[: self.nP], G[self.nP:]

    def merge(self, stream=None):
        """W0' = Pi_R W0 Pi_P^T (or its int8 or 4-bit codes): once per set of permutations."""
        if self.W0 is None:
            raise ValueError("the layer has given up W0")
        if self.int4_group:
            merge_perm_q4(self.W0, self.W0q, self.scales, self.perm_R, self.perm_P,
                          self.int4_group, stream)
        elif self.int8:
            merge_perm_q8(self.W0, self.W0q, self.scales, self.perm_R, self.perm_P, stream)
        else:
            merge_perm(self.W0, self.W0p, self.perm_R, self.perm_P, stream)

    def cnp_forward(self, stream=None):
        self.cnp.forward(stream)

    def _tokens(self, lead, width):
        """Descriptor, save buffers and scratch for the tokens of `lead` ([tokens, width]), T or
        fewer."""
        T = lead.numel() // width
        if T >= self.T:  # (more: the dense and int8 calls take the first T, the others refuse them)
            return self.desc, self.U, self.Wsave, self.ws
        few = self._fewer.get(T)
        if few is None:
            desc = LinearDesc.from_buffer_copy(self.desc)
            desc.T = T
            need = _layer_scratch_bytes(desc, self.save, self.int8, self.int4_group)
            # (up to 4 tokens of a layer of 5, or another split of the dG sums, may need more)
            ws = self.ws if need <= self.ws.nbytes else self.ws.new_empty(need)
            few = self._fewer[T] = desc, ws
        desc, ws = few
        if not self.save:
            return desc, None, None, ws
        return desc, self.U[:T], self.Wsave[:T], ws

    def _check_fewer(self, desc, outer):
        """(The calls without dropout on a dense or int8 weight check no shapes themselves.)"""
        if desc.T < self.T:
            _check_layer(desc, self.weight, outer, *self.G_ops())

    def forward(self, x, y, stream=None):
        GP, GR = self.G_ops()
        drop = self._drop()
        desc, U, W, ws = self._tokens(x, self.n)
        if self.int4_group or drop is not None:
            linear_fwd_ex(desc, self.weight, drop, x, GP, GR, y, U, W, ws, stream)
            return
        self._check_fewer(desc, ((x, self.n), (y, self.m)))
        if self.int8:
            linear_fwd_q8(desc, x, GP, GR, self.W0q, self.scales, y, U, W, ws, stream)
        else:
            linear_fwd(desc, x, GP, GR, self.W0p, y, U, W, ws, stream)

    def backward(self, x, dy, dx, accumulate=0, stream=None):
        GP, GR = self.G_ops()
        drop = self._drop()
        dGP, dGR = self.dG[: self.nP], self.dG[self.nP:]
        desc, U, W, ws = self._tokens(dy, self.m)
        if self.int4_group or drop is not None:
            linear_bwd_ex(desc, self.weight, drop, x, dy, GP, GR, U, W, dx, dGP, dGR, accumulate,
                          ws, stream)
            return
        self._check_fewer(desc, ((x, self.n), (dy, self.m), (dx, self.n)))
        if self.int8:
            linear_bwd_q8(desc, x, dy, GP, GR, self.W0q, self.scales, U, W, dx, dGP, dGR,
                          accumulate, ws, stream)
        else:
            linear_bwd(desc, x, dy, GP, GR, self.W0p, U, W, dx, dGP, dGR, accumulate, ws, stream)

    def cnp_backward(self, stream=None):
        """dtheta from dG; reads Q, S and F' of the last cnp_forward (theta unchanged)."""
        self.cnp.backward(stream)

    def step(self, x, dy, y, dx, stream=None):
        """One pass of the per-step path: CNP forward, layer forward and backward, CNP
        backward (the merge of the permutations is per set of permutations, not per step)."""
        self.cnp_forward(stream)
        self.forward(x, y, stream)
        self.backward(x, dy, dx, 0, stream)
        self.cnp_backward(stream)
        if self.dropout is not None and self.training:
            self.dropout.advance(stream)


class PoetxLinearGroup:
    """Several POET-X linears (e.g. the seven of a decoder block) whose CNP forward and
    backward each run as one call over all of their blocks, and whose layer calls share one
    scratch buffer (they run one after another on one stream).

    specs: list of (W0, theta_P, theta_R, perm_P, perm_R) per linear.  int8_weight, int4_group:
    the form of every linear's merged weight; dropout: of every linear's input, linear i at
    site dropout.site + i with the shared step counter.
    """

    def __init__(self, specs, b: int, k: int, T: int, save_activations: bool = True,
                 int8_weight: bool = False, int4_group: int = 0, dropout=None):
        import torch
        _require_cuda()
        W0s = [sp[0] for sp in specs]
        dev = W0s[0].device
        bf16 = W0s[0].dtype == torch.bfloat16
        nblks = [(W.shape[1] + W.shape[0]) // b for W in W0s]
        self.cnp = CnpBuffers(sum(nblks), b, k, dev, W0s[0].dtype if bf16 else None)
        need = 16
        for W in W0s:
            m, n = W.shape
            d = LinearDesc(T, n, m, b, POETX_BF16 if bf16 else POETX_F32, None, None, None, None)
            need = max(need, _layer_scratch_bytes(d, save_activations, int8_weight, int4_group))
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)
        self.layers = []
        off = 0
        for sp, nb in zip(specs, nblks):
            W0, tP, tR, pP, pR = sp
            self.layers.append(PoetxLinear(W0, tP, tR, pP, pR, b, k, T, save_activations,
                                           int8_weight, cnp=self.cnp, first_block=off,
                                           ws=self.ws, int4_group=int4_group,
                                           dropout=None if dropout is None else
                                           dropout.at_site(dropout.site + len(self.layers))))
            off += nb
        self.dropout = dropout
        self.training = True
        self.b, self.k, self.T = b, k, T

    def train(self, mode: bool = True):
        """Dropout on (mode) or off, in every linear."""
        self.training = mode
        for L in self.layers:
            L.training = mode

    def merge(self, stream=None):
        for L in self.layers:
            L.merge(stream)

    def cnp_forward(self, stream=None):
        self.cnp.forward(stream)

    def forward(self, xs, ys, stream=None):
        for L, x, y in zip(self.layers, xs, ys):
            L.forward(x, y, stream)

    def backward(self, xs, dys, dxs, accumulate=0, stream=None):
        for L, x, dy, dx in reversed(list(zip(self.layers, xs, dys, dxs))):
            L.backward(x, dy, dx, accumulate, stream)

    def cnp_backward(self, stream=None):
        self.cnp.backward(stream)

    def step(self, xs, dys, ys, dxs, stream=None):
        """CNP forward (every block, one call), every layer's forward, every layer's
        backward (last layer first), CNP backward (one call)."""
        self.cnp_forward(stream)
        self.forward(xs, ys, stream)
        self.backward(xs, dys, dxs, 0, stream)
        self.cnp_backward(stream)
        if self.dropout is not None and self.training:
            self.dropout.advance(stream)
