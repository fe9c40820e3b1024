"""Python binding of libtq.so, the CUDA library of rotated-codebook quantization.

Argument marshalling only: every function here checks shapes, allocates the
output tensors with torch (device memory), and calls the C entry point of the
same name on torch's current CUDA stream.  All arithmetic runs in the library's
kernels.  There is no CPU fallback: if the library cannot be loaded, ``load()``
raises.
"""
from __future__ import annotations

import collections
import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtq.so")

TQ_F32, TQ_BF16, TQ_F16 = 0, 1, 2
TQ_OK, TQ_ERR_INVALID, TQ_ERR_UNSUPPORTED, TQ_ERR_CUDA, TQ_ERR_TIMEOUT, TQ_ERR_DEVICE = range(6)
TQ_DEVERR_BAD_ID, TQ_DEVERR_TIMEOUT, TQ_DEVERR_BAD_BOOK, TQ_DEVERR_BAD_PAGE, TQ_DEVERR_NO_PAGE = 1, 2, 4, 8, 16
TQ_ROPE_HALF, TQ_ROPE_INTERLEAVED = 0, 1
TQ_ROPE_NONE, TQ_ROPE_LINEAR, TQ_ROPE_BASE, TQ_ROPE_PARTS = range(4)

_c_p = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_u32 = ctypes.c_uint32
_sz = ctypes.c_size_t


class tq_codebook_t(ctypes.Structure):
    _fields_ = [("levels", _i32), ("centroids", _c_p), ("thresholds", _c_p)]


class tq_rotation_t(ctypes.Structure):
    _fields_ = [("dim", _i32), ("block", _i32), ("signs", _c_p)]


class tq_qweight_t(ctypes.Structure):
    _fields_ = [("codes", _c_p), ("scales", _c_p), ("experts", _i32), ("rows", _i32), ("cols", _i32),
                ("group", _i32), ("row_stride_words", _i64), ("expert_stride_words", _i64),
                ("expert_stride_scales", _i64), ("cb", tq_codebook_t)]


class tq_rope_t(ctypes.Structure):
    _fields_ = [("dim", _i32), ("rotary", _i32), ("layout", _i32), ("factor", ctypes.c_float), ("steps", _c_p)]


class tq_rope_scaling_t(ctypes.Structure):
    _fields_ = [("kind", _i32), ("factor", ctypes.c_double), ("original", ctypes.c_double),
                ("slow_turns", ctypes.c_double), ("fast_turns", ctypes.c_double)]


class tq_kv_pages_t(ctypes.Structure):
    _fields_ = [("kcodes", _c_p), ("kscales", _c_p), ("vcodes", _c_p), ("vscales", _c_p), ("Hkv", _i32), ("D", _i32),
                ("group", _i32), ("page", _i32), ("pages", _i64), ("page_stride", _i64), ("head_stride", _i64),
                ("kcb", tq_codebook_t), ("vcb", tq_codebook_t), ("rot", tq_rotation_t)]


class tq_page_pool_t(ctypes.Structure):
    _fields_ = [("table", _c_p), ("held", _c_p), ("free", _c_p), ("n_free", _c_p), ("batch", _i32), ("width", _i32),
                ("page", _i32), ("pages", _i64)]


class tq_latent_pages_t(ctypes.Structure):
    _fields_ = [("rows", _c_p), ("dt", _i32), ("latent", _i32), ("rope", _i32), ("page", _i32), ("pages", _i64),
                ("page_stride", _i64)]


class tq_layer_desc_t(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 64), ("experts", _i32), ("rows", _i32), ("cols", _i32), ("group", _i32),
                ("row_stride_words", _i64), ("levels", _i32), ("rot_dim", _i32), ("rot_block", _i32),
                ("rot_seed", ctypes.c_uint64), ("centroids", _c_p), ("codes", _c_p), ("scales", _c_p)]


class tq_tier_policy_t(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("down_levels", "down_group", "expert_levels", "expert_group", "mlp_levels",
                                    "mlp_group", "attn_levels", "attn_group", "other_levels", "other_group")]


_P = ctypes.POINTER
# name -> (restype, argtypes), exactly the declarations of include/tq.h
_SIGS = {
    "tq_status_string": (ctypes.c_char_p, [_i32]),
    "tq_codes_per_word": (_i32, [_i32]),
    "tq_row_words": (_i64, [_i32, _i32]),
    "tq_row_stride_words": (_i64, [_i32, _i32]),
    "tq_codebook": (_i32, [_i32, _P(ctypes.c_double), _P(ctypes.c_double)]),
    "tq_rotation_signs": (_i32, [ctypes.c_uint64, _i32, _P(ctypes.c_int8)]),
    "tq_rotate": (_i32, [_P(tq_rotation_t), _c_p, _i32, _i64, _c_p, _i32, _c_p]),
    "tq_quantize": (_i32, [_c_p, _i32, _i64, _i32, _i32, _P(tq_rotation_t), _P(tq_codebook_t), _c_p, _c_p, _i64,
                           _c_p]),
    "tq_qmv": (_i32, [_P(tq_qweight_t), _c_p, _i32, _c_p, _i32, _c_p]),
    "tq_qmv_tc": (_i32, [_P(tq_qweight_t), _c_p, _i32, _c_p, _c_p, _sz, _c_p, _c_p]),
    "tq_qmv_tc_workspace_bytes": (_sz, [_i32, _i32]),
    "tq_gather_qmv": (_i32, [_P(tq_qweight_t), _c_p, _c_p, _i32, _i32, _c_p, _i32, _c_p, _sz, _c_p, _c_p]),
    "tq_gather_qmv_workspace_bytes": (_sz, [_P(tq_qweight_t), _i32, _i32]),
    "tq_multi_gather_qmv": (_i32, [_P(tq_qweight_t), _c_p, _c_p, _i32, _c_p, _i32, _c_p, _sz, _c_p, _c_p]),
    "tq_multi_gather_qmv_workspace_bytes": (_sz, [_P(tq_qweight_t), _i32]),
    "tq_gather_qmv_rotate": (_i32, [_P(tq_qweight_t), _c_p, _i32, _P(tq_rotation_t), _c_p, _i32, _i32, _c_p, _i32,
                                    _c_p, _c_p]),
    "tq_multi_gather_qmv_swiglu": (_i32, [_P(tq_qweight_t), _c_p, _P(tq_rotation_t), _c_p, _i32, _c_p, _i32, _c_p,
                                          _c_p]),
    "tq_moe_route": (_i32, [_c_p, _i32, _i32, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "tq_route_workspace_bytes": (_sz, [_i32]),
    "tq_swiglu_rotate": (_i32, [_c_p, _i64, _i32, _P(tq_rotation_t), _c_p, _i32, _c_p]),
    "tq_moe_combine": (_i32, [_c_p, _c_p, _c_p, _i32, _i32, _i32, _c_p, _i32, _c_p]),
    "tq_gather_qmm": (_i32, [_P(tq_qweight_t), _c_p, _i32, _c_p, _c_p, _i32, _i32, _i32, _c_p, _i32, _c_p, _sz,
                             _c_p, _c_p]),
    "tq_gather_qmm_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "tq_dequant_experts": (_i32, [_P(tq_qweight_t), _c_p, _i32, _c_p, _i32, _c_p, _c_p]),
    "tq_kv_quantize": (_i32, [_c_p, _c_p, _i32, _i32, _i32, _i32, _i64, _i64, _P(tq_rotation_t),
                              _P(tq_codebook_t), _P(tq_codebook_t), _i32, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "tq_kv_attend": (_i32, [_c_p, _i32, _i32, _i32, _i32, _i64, _i64, _P(tq_rotation_t), _P(tq_codebook_t),
                            _P(tq_codebook_t), _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _sz, _c_p]),
    "tq_kv_attend_workspace_bytes": (_sz, [_i32, _i32, _i64]),
    "tq_kv_attend_noalloc": (_i32, [_c_p, _i32, _i32, _i32, _i32, _i64, _i64, _P(tq_rotation_t), _P(tq_codebook_t),
                                    _P(tq_codebook_t), _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "tq_kv_attend_noalloc_max_scratch_bytes": (_sz, []),
    "tq_moe_decode_layer_workspace_bytes": (_sz, [_P(tq_qweight_t), _P(tq_qweight_t), _i32]),
    "tq_moe_decode_layer": (_i32, [_P(tq_qweight_t), _P(tq_qweight_t), _P(tq_rotation_t), _P(tq_rotation_t), _c_p,
                                   _c_p, _i32, _i32, _c_p, _i32, _c_p, _sz, _c_p, _c_p]),
    "tq_rope_steps": (_i32, [_i32, ctypes.c_double, _P(tq_rope_scaling_t), _c_p, _P(ctypes.c_float)]),
    "tq_rope": (_i32, [_P(tq_rope_t), _c_p, _i64, _i32, _i32, _c_p, _i64, _i32, _c_p, _i64, _c_p, _i64, _i32, _c_p,
                       _i64, _c_p]),
    "tq_kv_append": (_i32, [_P(tq_kv_pages_t), _c_p, _i64, _c_p, _i64, _i32, _i64, _c_p, _P(tq_rope_t), _c_p, _c_p,
                            _c_p]),
    "tq_kv_fetch": (_i32, [_P(tq_kv_pages_t), _c_p, _i64, _c_p, _c_p, _i32, _c_p, _c_p]),
    "tq_kv_attend_tree": (_i32, [_P(tq_kv_pages_t), _c_p, _i64, _i32, _i32, _i32, _i32, _c_p, _i32, _c_p, _i64, _c_p,
                                 _i64, _c_p, _i64, _c_p, _c_p, ctypes.c_float, _c_p, _c_p, _sz, _c_p, _c_p]),
    "tq_kv_attend_tree_workspace_bytes": (_sz, [_P(tq_kv_pages_t), _i32, _i32, _i32, _i64]),
    "tq_kv_plan": (_i32, [_P(tq_page_pool_t), _c_p, _c_p, _c_p, _i32, _i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "tq_verify_tree": (_i32, [_c_p, _i64, _c_p, _i64, _i32, _i32, _i32, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                              _c_p]),
    "tq_latent_append": (_i32, [_P(tq_latent_pages_t), _c_p, _i64, _c_p, _i64, _i32, _i64, _c_p, _P(tq_rope_t), _c_p, _c_p,
                                _c_p]),
    "tq_latent_attend_tree": (_i32, [_P(tq_latent_pages_t), _c_p, _i64, _i32, _i32, _i32, _c_p, _i32, _c_p, _i64, _c_p, _i64,
                                     _c_p, _c_p, ctypes.c_float, _c_p, _c_p, _sz, _c_p, _c_p]),
    "tq_latent_attend_tree_workspace_bytes": (_sz, [_P(tq_latent_pages_t), _i32, _i32, _i32, _i64]),
    "tq_latent_attend_prompt": (_i32, [_c_p, _i64, _c_p, _c_p, _i64, _i64, _c_p, _i64, _i32, _i32, _i32, _i64, _i64, _c_p, _c_p,
                                       _i32, ctypes.c_float, _c_p, _c_p, _sz, _c_p, _c_p]),
    "tq_latent_attend_prompt_workspace_bytes": (_sz, [_i32, _i32, _i64, _i64]),
    "tq_check_error": (_i32, [_c_p, _P(_u32), _c_p]),
    "tq_set_wait_budget": (_i32, [_i64]),
    "tq_rotation_dense": (_i32, [ctypes.c_uint64, _i32, _P(ctypes.c_double)]),
    "tq_rotate_dense": (_i32, [_c_p, _i32, _c_p, _i32, _i64, _c_p, _i32, _c_p]),
    "tq_layer_tier": (_i32, [ctypes.c_char_p, _P(tq_tier_policy_t), _P(_i32), _P(_i32)]),
    "tq_pack_file_write": (_i32, [ctypes.c_char_p, _P(tq_layer_desc_t), _i32]),
    "tq_pack_file_info": (_i32, [ctypes.c_char_p, _P(_i32), _P(tq_layer_desc_t), _i32]),
    "tq_pack_file_read_layer": (_i32, [ctypes.c_char_p, _i32, _c_p, _c_p, _c_p]),
    "tq_expert_cache_create": (_i32, [_P(tq_qweight_t), _i32, _c_p, _c_p, _P(_c_p)]),
    "tq_expert_cache_destroy": (None, [_c_p]),
    "tq_expert_cache_plan": (_i32, [_c_p, _c_p, _i32, _c_p, _c_p]),
    "tq_expert_cache_map": (_i32, [_c_p, _c_p, _i32, _c_p, _c_p]),
    "tq_expert_cache_stats": (_i32, [_c_p, _P(_i64), _P(_i64), _P(_i64)]),
    "tq_selftest_trit_decode": (_i32, [_u32, _u32, _c_p, _c_p]),
}

_lib = None


def load(path: str | None = None):
    """Load libtq.so (raises if it is missing) and declare every entry point."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libtq.so not built ({p}); run __graft_entry__.build()")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


class TQError(RuntimeError):
    pass


def _check(status: int, what: str):
    if status != TQ_OK:
        raise TQError(f"{what}: {load().tq_status_string(status).decode()} ({status})")


# ---------------------------------------------------------------- torch marshalling

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream():
    return ctypes.c_void_p(_torch().cuda.current_stream().cuda_stream)


_dtype_codes = {}


def _dt(t) -> int:
    if not _dtype_codes:
        torch = _torch()
        _dtype_codes.update({torch.float32: TQ_F32, torch.bfloat16: TQ_BF16, torch.float16: TQ_F16})
    return _dtype_codes[t.dtype]


def _torch_dtype(code: int):
    torch = _torch()
    return {TQ_F32: torch.float32, TQ_BF16: torch.bfloat16, TQ_F16: torch.float16}[code]


def _contig(t, name):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t


# ---------------------------------------------------------------- host helpers

def codes_per_word(levels: int) -> int:
    return int(load().tq_codes_per_word(levels))


def row_words(levels: int, cols: int) -> int:
    return int(load().tq_row_words(levels, cols))


def row_stride_words(levels: int, cols: int) -> int:
    return int(load().tq_row_stride_words(levels, cols))


def codebook(levels: int):
    """Host fp64 Gaussian Lloyd-Max book: (centroids[levels], thresholds[levels-1]) numpy arrays."""
    c = np.zeros(levels, dtype=np.float64)
    t = np.zeros(max(levels - 1, 1), dtype=np.float64)
    _check(load().tq_codebook(levels, c.ctypes.data_as(_P(ctypes.c_double)), t.ctypes.data_as(_P(ctypes.c_double))),
           "tq_codebook")
    return c, t[:levels - 1]


def rotation_signs(seed: int, dim: int) -> np.ndarray:
    s = np.zeros(dim, dtype=np.int8)
    _check(load().tq_rotation_signs(ctypes.c_uint64(seed), dim, s.ctypes.data_as(_P(ctypes.c_int8))),
           "tq_rotation_signs")
    return s


def rotation_dense(seed: int, dim: int) -> np.ndarray:
    """Host fp64 dense rotation [dim, dim] of the QR fallback (see include/tq.h, tq_rotation_dense)."""
    R = np.zeros((dim, dim), dtype=np.float64)
    _check(load().tq_rotation_dense(ctypes.c_uint64(seed), dim, R.ctypes.data_as(_P(ctypes.c_double))),
           "tq_rotation_dense")
    return R


# ---------------------------------------------------------------- device descriptors

class Codebook:
    """A codebook on the device: fp32 centroids and thresholds."""

    def __init__(self, levels: int, device="cuda", centroids=None, thresholds=None):
        torch = _torch()
        if centroids is None:
            centroids, thresholds = codebook(levels)
        self.levels = int(levels)
        self.centroids = torch.tensor(np.asarray(centroids, np.float32), device=device)
        self.thresholds = torch.tensor(np.asarray(thresholds, np.float32).reshape(-1), device=device)
        if self.thresholds.numel() == 0:
            self.thresholds = torch.zeros(1, dtype=torch.float32, device=device)

    def c(self) -> tq_codebook_t:
        return tq_codebook_t(self.levels, self.centroids.data_ptr(), self.thresholds.data_ptr())


class Rotation:
    """R = blockdiag(H_block) diag(signs) / sqrt(block) over vectors of length dim."""

    def __init__(self, dim: int, block: int, seed: int | None = None, signs=None, device="cuda"):
        torch = _torch()
        if signs is None:
            signs = rotation_signs(seed, dim)
        self.dim, self.block = int(dim), int(block)
        self.signs = torch.tensor(np.asarray(signs, np.int8), device=device)

    def c(self) -> tq_rotation_t:
        return tq_rotation_t(self.dim, self.block, self.signs.data_ptr())


class DenseRotation:
    """The QR-fallback rotation of a dimension on the device (fp32 [dim, dim]), from its seed or given."""

    def __init__(self, dim: int, seed: int | None = None, R=None, device="cuda"):
        torch = _torch()
        if R is None:
            R = rotation_dense(seed, dim)
        self.dim = int(dim)
        self.R = torch.tensor(np.asarray(R, np.float32), device=device)

    def identity(self, device="cuda") -> "Rotation":
        """The identity rotation of this dim (block 1, signs +1): what tq_quantize takes after rotate_dense."""
        return Rotation(self.dim, 1, signs=np.ones(self.dim, np.int8), device=device)


class QWeight:
    """A bank of quantized matrices [experts, rows, cols] as written by ``quantize``."""

    def __init__(self, codes, scales, experts: int, rows: int, cols: int, group: int, cb: Codebook,
                 row_stride: int | None = None):
        self.codes, self.scales, self.cb = codes, scales, cb
        self.experts, self.rows, self.cols, self.group = int(experts), int(rows), int(cols), int(group)
        self.row_stride = int(row_stride if row_stride is not None else row_stride_words(cb.levels, cols))

    def c(self) -> tq_qweight_t:
        esw = self.rows * self.row_stride
        ess = self.rows * (self.cols // self.group)
        return tq_qweight_t(self.codes.data_ptr(), self.scales.data_ptr(), self.experts, self.rows, self.cols,
                            self.group, self.row_stride, esw, ess, self.cb.c())


# ---------------------------------------------------------------- device entry points

def rotate(x, rot: Rotation, out_dtype=None):
    torch = _torch()
    _contig(x, "x")
    out = torch.empty(x.shape, dtype=out_dtype or torch.float32, device=x.device)
    r = rot.c()
    _check(load().tq_rotate(ctypes.byref(r), _ptr(x), _dt(x), x.numel() // rot.dim, _ptr(out), _dt(out), _stream()),
           "tq_rotate")
    return out


def rotate_dense(x, rot: DenseRotation, precise: bool = False):
    """R x for every row of x (f32 out); precise accumulates in fp64."""
    torch = _torch()
    _contig(x, "x")
    out = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    _check(load().tq_rotate_dense(_ptr(rot.R), rot.dim, _ptr(x), _dt(x), x.numel() // rot.dim, _ptr(out),
                                  int(precise), _stream()), "tq_rotate_dense")
    return out


def quantize_dense(W, group: int, rot: DenseRotation, cb: Codebook, row_stride: int | None = None):
    """Encode rows of W with the dense rotation: rotate (fp64 sums), then group RMS, snap and pack."""
    return quantize(rotate_dense(W, rot, precise=True), group, rot.identity(device=W.device), cb, row_stride)


def quantize(W, group: int, rot: Rotation, cb: Codebook, row_stride: int | None = None):
    """Encode rows of W [rows, cols] -> (codes uint32 [rows, stride] as int32 storage, scales fp16 bits)."""
    torch = _torch()
    _contig(W, "W")
    rows, cols = W.shape
    stride = row_stride if row_stride is not None else row_stride_words(cb.levels, cols)
    codes = torch.empty((rows, stride), dtype=torch.int32, device=W.device)
    scales = torch.empty((rows, cols // group), dtype=torch.int16, device=W.device)
    r, b = rot.c(), cb.c()
    _check(load().tq_quantize(_ptr(W), _dt(W), rows, cols, group, ctypes.byref(r), ctypes.byref(b), _ptr(codes),
                              _ptr(scales), stride, _stream()), "tq_quantize")
    return codes, scales


def qmv(w: QWeight, x_rot, out_dtype=None, tensor_cores=True):
    """y = W x_rot for every row of x_rot.  With tensor_cores, an f32 output and two or more
    rows, the tq_qmv_tc form runs where it applies (fp16 operands, fp32 sums; at one row the
    CUDA-core kernel is as fast); elsewhere tq_qmv."""
    torch = _torch()
    _contig(x_rot, "x_rot")
    T = x_rot.shape[0]
    y = torch.empty((T, w.rows), dtype=out_dtype or torch.float32, device=x_rot.device)
    q = w.c()
    if tensor_cores and y.dtype == torch.float32 and T >= 2:
        nb = int(load().tq_qmv_tc_workspace_bytes(T, w.cols))
        ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=x_rot.device)
        st = load().tq_qmv_tc(ctypes.byref(q), _ptr(x_rot), T, _ptr(y), _ptr(ws), nb, None, _stream())
        if st != TQ_ERR_UNSUPPORTED:
            _check(st, "tq_qmv_tc")
            return y
    _check(load().tq_qmv(ctypes.byref(q), _ptr(x_rot), T, _ptr(y), _dt(y), _stream()), "tq_qmv")
    return y


def qmv_tc(w: QWeight, x_rot, err=None):
    """The tensor-core dense matvec alone (raises TQError where it does not apply)."""
    torch = _torch()
    _contig(x_rot, "x_rot")
    T = x_rot.shape[0]
    y = torch.empty((T, w.rows), dtype=torch.float32, device=x_rot.device)
    nb = int(load().tq_qmv_tc_workspace_bytes(T, w.cols))
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=x_rot.device)
    q = w.c()
    _check(load().tq_qmv_tc(ctypes.byref(q), _ptr(x_rot), T, _ptr(y), _ptr(ws), nb, _ptr(err), _stream()),
           "tq_qmv_tc")
    return y


def _workspace(nbytes: int, device, ws=None):
    """A caller's scratch buffer if it is large enough, else a new one (None when nothing is needed)."""
    if nbytes <= 0:
        return None
    if ws is not None and ws.numel() * ws.element_size() >= nbytes:
        return ws
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device)


def gather_qmv(w: QWeight, x_rot, ids, out_dtype=None, err=None, ws=None, use_ws=True):
    """y[t, j] = W_{ids[t, j]} x_rot[t].  use_ws=False passes no scratch (the single-pass kernel
    then takes rows the table-lookup kernel would split)."""
    torch = _torch()
    _contig(x_rot, "x_rot")
    _contig(ids, "ids")
    T, k = ids.shape
    y = torch.empty((T, k, w.rows), dtype=out_dtype or torch.float32, device=x_rot.device)
    q = w.c()
    nb = int(load().tq_gather_qmv_workspace_bytes(ctypes.byref(q), T, k)) if use_ws else 0
    ws = _workspace(nb, x_rot.device, ws)
    _check(load().tq_gather_qmv(ctypes.byref(q), _ptr(x_rot), _ptr(ids), T, k, _ptr(y), _dt(y), _ptr(ws), nb,
                                _ptr(err), _stream()), "tq_gather_qmv")
    return y


def multi_gather_qmv(w: QWeight, x_rot, ids, out_dtype=None, err=None, ws=None, use_ws=True):
    """y[p] = W_{ids[p]} x_rot[p] (use_ws as for gather_qmv)."""
    torch = _torch()
    _contig(x_rot, "x_rot")
    _contig(ids, "ids")
    P = ids.shape[0]
    y = torch.empty((P, w.rows), dtype=out_dtype or torch.float32, device=x_rot.device)
    q = w.c()
    nb = int(load().tq_multi_gather_qmv_workspace_bytes(ctypes.byref(q), P)) if use_ws else 0
    ws = _workspace(nb, x_rot.device, ws)
    _check(load().tq_multi_gather_qmv(ctypes.byref(q), _ptr(x_rot), _ptr(ids), P, _ptr(y), _dt(y), _ptr(ws), nb,
                                      _ptr(err), _stream()), "tq_multi_gather_qmv")
    return y


def gather_qmv_rotate(w: QWeight, x, rot: Rotation, ids, out_dtype=None, err=None):
    """gather_qmv of R x with the rotation done inside the matvec (x: f32 or bf16 [T, cols])."""
    torch = _torch()
    _contig(x, "x")
    _contig(ids, "ids")
    T, k = ids.shape
    y = torch.empty((T, k, w.rows), dtype=out_dtype or torch.float32, device=x.device)
    q, r = w.c(), rot.c()
    _check(load().tq_gather_qmv_rotate(ctypes.byref(q), _ptr(x), _dt(x), ctypes.byref(r), _ptr(ids), T, k, _ptr(y),
                                       _dt(y), _ptr(err), _stream()), "tq_gather_qmv_rotate")
    return y


def multi_gather_qmv_swiglu(w: QWeight, gate_up, rot: Rotation, ids, out_dtype=None, err=None):
    """multi_gather_qmv of R (silu(gate) * up) per pair, SwiGLU and rotation inside (gate_up: f32 [P, 2*cols])."""
    torch = _torch()
    _contig(gate_up, "gate_up")
    _contig(ids, "ids")
    P = ids.shape[0]
    y = torch.empty((P, w.rows), dtype=out_dtype or torch.float32, device=gate_up.device)
    q, r = w.c(), rot.c()
    _check(load().tq_multi_gather_qmv_swiglu(ctypes.byref(q), _ptr(gate_up), ctypes.byref(r), _ptr(ids), P, _ptr(y),
                                             _dt(y), _ptr(err), _stream()), "tq_multi_gather_qmv_swiglu")
    return y


def moe_route(logits, k: int, sort: bool = True):
    """-> ids [T,k] int32, probs [T,k] f32, perm [T*k], pair_pos [T*k], offsets [E+1].

    With sort=False only ids and probs are computed (the other three are None).
    """
    torch = _torch()
    _contig(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    probs = torch.empty((T, k), dtype=torch.float32, device=dev)
    if not sort:
        _check(load().tq_moe_route(_ptr(logits), T, E, k, _ptr(ids), _ptr(probs), None, None, None, None, 0,
                                   _stream()), "tq_moe_route")
        return ids, probs, None, None, None
    perm = torch.empty(T * k, dtype=torch.int32, device=dev)
    pos = torch.empty(T * k, dtype=torch.int32, device=dev)
    off = torch.empty(E + 1, dtype=torch.int32, device=dev)
    nb = int(load().tq_route_workspace_bytes(E))
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
    _check(load().tq_moe_route(_ptr(logits), T, E, k, _ptr(ids), _ptr(probs), _ptr(perm), _ptr(pos), _ptr(off),
                               _ptr(ws), nb, _stream()), "tq_moe_route")
    return ids, probs, perm, pos, off


def swiglu_rotate(gate_up, inter: int, rot: Rotation, out_dtype=None):
    torch = _torch()
    _contig(gate_up, "gate_up")
    P = gate_up.numel() // (2 * inter)
    out = torch.empty((P, inter), dtype=out_dtype or torch.float32, device=gate_up.device)
    r = rot.c()
    _check(load().tq_swiglu_rotate(_ptr(gate_up), P, inter, ctypes.byref(r), _ptr(out), _dt(out), _stream()),
           "tq_swiglu_rotate")
    return out


def moe_combine(y, probs, k: int, pair_pos=None, out_dtype=None):
    torch = _torch()
    _contig(y, "y")
    H = y.shape[-1]
    T = probs.numel() // k
    out = torch.empty((T, H), dtype=out_dtype or torch.float32, device=y.device)
    _check(load().tq_moe_combine(_ptr(y), _ptr(probs), _ptr(pair_pos), T, k, H, _ptr(out), _dt(out), _stream()),
           "tq_moe_combine")
    return out


def gather_qmm(w: QWeight, x, perm, offsets, k: int, per_pair_input: bool = False, out_dtype=None, err=None):
    torch = _torch()
    _contig(x, "x")
    P = int(perm.numel()) if not per_pair_input else int(x.shape[0])
    y = torch.empty((P, w.rows), dtype=out_dtype or torch.float32, device=x.device)
    nb = int(load().tq_gather_qmm_workspace_bytes(P, w.cols, int(per_pair_input)))
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=x.device)
    q = w.c()
    _check(load().tq_gather_qmm(ctypes.byref(q), _ptr(x), _dt(x), _ptr(perm), _ptr(offsets), P, k,
                                int(per_pair_input), _ptr(y), _dt(y), _ptr(ws), nb, _ptr(err), _stream()),
           "tq_gather_qmm")
    return y


def dequant_experts(w: QWeight, ids, out_dtype=None, err=None):
    torch = _torch()
    _contig(ids, "ids")
    n = ids.numel()
    out = torch.empty((n, w.rows, w.cols), dtype=out_dtype or torch.float32, device=ids.device)
    q = w.c()
    _check(load().tq_dequant_experts(ctypes.byref(q), _ptr(ids), n, _ptr(out), _dt(out), _ptr(err), _stream()),
           "tq_dequant_experts")
    return out


class KVCache:
    """Compressed KV cache: codes and fp16 scales per (kv head, position)."""

    def __init__(self, capacity: int, heads: int, dim: int, group: int, kcb: Codebook, vcb: Codebook,
                 rot: Rotation, device="cuda"):
        torch = _torch()
        self.capacity, self.heads, self.dim, self.group = capacity, heads, dim, group
        self.kcb, self.vcb, self.rot = kcb, vcb, rot
        self.kw, self.vw = row_words(kcb.levels, dim), row_words(vcb.levels, dim)
        self.kcodes = torch.zeros((heads, capacity, self.kw), dtype=torch.int32, device=device)
        self.vcodes = torch.zeros((heads, capacity, self.vw), dtype=torch.int32, device=device)
        self.kscales = torch.zeros((heads, capacity, dim // group), dtype=torch.int16, device=device)
        self.vscales = torch.zeros((heads, capacity, dim // group), dtype=torch.int16, device=device)
        self.length = 0


def kv_quantize(cache: KVCache, k, v, pos: int | None = None):
    _contig(k, "k")
    _contig(v, "v")
    T = k.shape[0]
    pos = cache.length if pos is None else pos
    r, kb, vb = cache.rot.c(), cache.kcb.c(), cache.vcb.c()
    _check(load().tq_kv_quantize(_ptr(k), _ptr(v), _dt(k), T, cache.heads, cache.dim, pos, cache.capacity,
                                 ctypes.byref(r), ctypes.byref(kb), ctypes.byref(vb), cache.group, _ptr(cache.kcodes),
                                 _ptr(cache.kscales), _ptr(cache.vcodes), _ptr(cache.vscales), _stream()),
           "tq_kv_quantize")
    cache.length = max(cache.length, pos + T)


def kv_attend(cache: KVCache, q, ctx: int | None = None, ws=None):
    torch = _torch()
    _contig(q, "q")
    Hq = q.shape[0]
    ctx = cache.length if ctx is None else ctx
    o = torch.empty((Hq, cache.dim), dtype=torch.float32, device=q.device)
    nb = int(load().tq_kv_attend_workspace_bytes(Hq, cache.dim, ctx))
    if ws is None:
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=q.device)
    r, kb, vb = cache.rot.c(), cache.kcb.c(), cache.vcb.c()
    _check(load().tq_kv_attend(_ptr(q), _dt(q), Hq, cache.heads, cache.dim, ctx, cache.capacity, ctypes.byref(r),
                               ctypes.byref(kb), ctypes.byref(vb), cache.group, _ptr(cache.kcodes),
                               _ptr(cache.kscales), _ptr(cache.vcodes), _ptr(cache.vscales), _ptr(o), _ptr(ws),
                               ws.numel(), _stream()), "tq_kv_attend")
    return o


def kv_attend_noalloc(cache: KVCache, q, ctx: int | None = None):
    """kv_attend with the library's fixed device scratch instead of a workspace (see include/tq.h)."""
    torch = _torch()
    _contig(q, "q")
    Hq = q.shape[0]
    ctx = cache.length if ctx is None else ctx
    o = torch.empty((Hq, cache.dim), dtype=torch.float32, device=q.device)
    r, kb, vb = cache.rot.c(), cache.kcb.c(), cache.vcb.c()
    _check(load().tq_kv_attend_noalloc(_ptr(q), _dt(q), Hq, cache.heads, cache.dim, ctx, cache.capacity,
                                       ctypes.byref(r), ctypes.byref(kb), ctypes.byref(vb), cache.group,
                                       _ptr(cache.kcodes), _ptr(cache.kscales), _ptr(cache.vcodes),
                                       _ptr(cache.vscales), _ptr(o), _stream()), "tq_kv_attend_noalloc")
    return o


# ---------------------------------------------------------------- rotary positions

class Rope:
    """Rotary positions of heads of length ``dim``: the first ``rotary`` elements (default: all) turn.

    ``layout``: "half" (element i pairs with i + rotary/2) or "interleaved" (2i with 2i + 1).  ``scaling``
    for long contexts: None or a dict with "kind" ("linear", "base" or "parts"), "factor" and, for
    parts, "original" (positions) and optionally "slow_turns" / "fast_turns" (1 and 32); see tq_rope_steps
    in include/tq.h.  ``steps`` (int64 [rotary/2], the phase per position in 2^-64 turns) and ``factor``
    take the place of ``base`` and ``scaling`` where a model brings frequencies of its own.
    """

    def __init__(self, dim: int, rotary: int | None = None, base: float = 10000.0, layout: str = "half",
                 scaling: dict | None = None, steps=None, factor: float | None = None, device="cuda"):
        torch = _torch()
        self.dim, self.rotary = int(dim), int(dim if rotary is None else rotary)
        if layout not in ("half", "interleaved"):
            raise ValueError(f"layout must be 'half' or 'interleaved', not {layout!r}")
        self.layout = layout
        if not 2 <= self.rotary <= self.dim or self.rotary % 2:
            raise ValueError(f"rotary must be even and between 2 and dim = {self.dim}, not {self.rotary}")
        if steps is None:
            host, own = rope_steps(self.rotary, base, scaling)
            steps, factor = torch.from_numpy(host), own if factor is None else factor
        elif scaling is not None:
            raise ValueError("steps are the scaled frequencies: scaling must be None")
        if steps.dtype != torch.int64 or steps.numel() != self.rotary // 2:
            raise ValueError(f"steps must be int64 [{self.rotary // 2}]")
        self.steps = steps.to(device).contiguous()
        self.factor = 1.0 if factor is None else float(factor)

    def c(self) -> tq_rope_t:
        """The descriptor of what the handle holds now."""
        steps = self.steps
        if steps.dtype is not _torch().int64 or steps.numel() != self.rotary // 2 or not steps.is_contiguous():
            raise ValueError(f"steps must be contiguous int64 [{self.rotary // 2}]")
        return tq_rope_t(self.dim, self.rotary, TQ_ROPE_INTERLEAVED if self.layout == "interleaved" else TQ_ROPE_HALF,
                         self.factor, steps.data_ptr())

    def ref(self):
        return ctypes.byref(self.c())


def rope_steps(rotary: int, base: float = 10000.0, scaling: dict | None = None):
    """(steps int64 [rotary/2], factor) of scaled rotary frequencies, on the host."""
    steps = np.zeros(max(rotary // 2, 1), np.int64)
    factor = ctypes.c_float(1.0)
    sc = None
    if scaling is not None:
        kinds = {"linear": TQ_ROPE_LINEAR, "base": TQ_ROPE_BASE, "parts": TQ_ROPE_PARTS}
        if scaling.get("kind") not in kinds:
            raise ValueError(f"scaling kind must be one of {sorted(kinds)}, not {scaling.get('kind')!r}")
        sc = ctypes.byref(tq_rope_scaling_t(kinds[scaling["kind"]], float(scaling["factor"]),
                                            float(scaling.get("original", 0.0)), float(scaling.get("slow_turns", 1.0)),
                                            float(scaling.get("fast_turns", 32.0))))
    _check(load().tq_rope_steps(rotary, float(base), sc, steps.ctypes.data, ctypes.byref(factor)), "tq_rope_steps")
    return steps, float(factor.value)


# A decode step's calls last about as long on the GPU as their arguments take to check, so the calls below keep their
# Python short: plain integers for pointers, one shape and one stride query a tensor, a cache's descriptor kept while all that it
# is made of stays the same, torch.empty (1.6 us; new_empty takes 3.6).

def _raw_stream(t) -> int:
    """torch's current stream on the tensor's device, as a number.  Launches go to the current device, so it has to be that one."""
    torch, device = _torch(), t.get_device()
    if device != torch.cuda.current_device():
        raise ValueError(f"the tensors are on device {device}, the current device is {torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(device)


def _word(err, device) -> int:
    """The address of a device error word (None: none)."""
    if err is None:
        return 0
    if err.get_device() != device or err.element_size() != 4 or err.is_floating_point() or err.numel() < 1:
        raise ValueError("err must hold a 32-bit integer on the same device as the others")
    return err.data_ptr()


def _heads(x, name, dim):
    """(tokens, heads, token stride) of x [..., heads, dim] whose heads lie one after another."""
    shape = x.shape
    nd = len(shape)
    if not x.is_cuda or nd < 3 or shape[-1] != dim:
        raise ValueError(f"{name} must be a CUDA tensor [..., heads, {dim}]")
    stride, heads = x.stride(), shape[-2]
    tokens, step = 1, None
    for i in range(nd - 3, -1, -1):
        size = shape[i]
        if size == 1:
            continue
        if size == 0:
            return 0, heads, heads * dim
        if step is None:
            step = stride[i]
        elif stride[i] != step * tokens:
            raise ValueError(f"{name}'s tokens must lie at one stride")
        tokens *= size
    if heads and (stride[-1] != 1 or (heads > 1 and stride[-2] != dim)):
        raise ValueError(f"{name}'s heads must lie one after another")
    return tokens, heads, (heads * dim if step is None else step)


def _ints(t, name, count, device, dtype=None):
    """The address of a contiguous integer tensor of `count` entries (int32 unless told otherwise)."""
    if dtype is None:
        dtype = _torch().int32
    if t.dtype is not dtype or t.numel() != count or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {count} {dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the same device as the others")
    return t.data_ptr()


def rope(q, positions, r: Rope, k=None, inverse: bool = False, inplace: bool = False):
    """Rotary positions of q [..., Hq, dim] and, in the same launch, k [..., Hkv, dim] (views of a fused
    projection are fine); positions: int32 with one entry per token.  Returns q's result, or (q's, k's)."""
    dim, dev = r.dim, q.get_device()
    T, hq, qs = _heads(q, "q", dim)
    pos = _ints(positions, "positions", T, dev)
    if r.steps.get_device() != dev:
        raise ValueError("the rotary frequencies must be on q's device")
    yq, yqs = (q, qs) if inplace else (_torch().empty(q.shape, dtype=q.dtype, device=q.device), hq * dim)
    if k is None:
        kp = ks = hk = yp = yks = 0
        yk = None
    else:
        Tk, hk, ks = _heads(k, "k", dim)
        if Tk != T or k.dtype is not q.dtype or k.get_device() != dev:
            raise ValueError("k must have q's tokens, dtype and device")
        yk, yks = (k, ks) if inplace else (_torch().empty(k.shape, dtype=k.dtype, device=k.device), hk * dim)
        kp, yp = k.data_ptr(), yk.data_ptr()
    _check(load().tq_rope(r.ref(), pos, T, _dt(q), int(inverse), q.data_ptr(), qs, hq, yq.data_ptr(), yqs, kp, ks, hk, yp,
                          yks, _raw_stream(q)), "tq_rope")
    return yq if k is None else (yq, yk)


# ---------------------------------------------------------------- paged compressed KV cache

class PagedKVCache:
    """A compressed KV cache in pages shared by many sequences: codes and fp16 scales [pages, heads, page, ...].

    ``page`` tokens to a page; a token's slot is page id * page + offset.  Which pages a sequence owns is
    the caller's table.  ``storage``: (kcodes, kscales, vcodes, vscales) tensors to use instead of new ones.
    """

    def __init__(self, pages: int, page: int, heads: int, dim: int, group: int, kcb: Codebook, vcb: Codebook,
                 rot: Rotation, device="cuda", storage=None):
        torch = _torch()
        self.pages, self.page, self.heads, self.dim, self.group = int(pages), int(page), int(heads), int(dim), int(group)
        self.kcb, self.vcb, self.rot = kcb, vcb, rot
        self.kw, self.vw = row_words(kcb.levels, dim), row_words(vcb.levels, dim)
        self.page_stride, self.head_stride = self.heads * self.page, self.page
        lead = (self.pages, self.heads, self.page)
        if storage is None:
            self.kcodes = torch.zeros((*lead, self.kw), dtype=torch.int32, device=device)
            self.vcodes = torch.zeros((*lead, self.vw), dtype=torch.int32, device=device)
            self.kscales = torch.zeros((*lead, dim // group), dtype=torch.int16, device=device)
            self.vscales = torch.zeros((*lead, dim // group), dtype=torch.int16, device=device)
        else:
            self.kcodes, self.kscales, self.vcodes, self.vscales = storage
            for t, width, size in ((self.kcodes, self.kw, 4), (self.kscales, dim // group, 2), (self.vcodes, self.vw, 4),
                                   (self.vscales, dim // group, 2)):
                if tuple(_contig(t, "storage").shape) != (*lead, width) or t.element_size() != size:
                    raise ValueError(f"storage must be contiguous [{self.pages}, {self.heads}, {self.page}, words or groups]")

    @classmethod
    def of(cls, cache: KVCache, page: int = 64) -> "PagedKVCache":
        """One sequence's contiguous cache seen as pages, in order (its capacity a multiple of the page)."""
        if cache.capacity % page:
            raise ValueError("the cache's capacity must be a multiple of the page")
        self = cls.__new__(cls)
        self.pages, self.page, self.heads, self.dim, self.group = (cache.capacity // page, int(page), cache.heads,
                                                                   cache.dim, cache.group)
        self.kcb, self.vcb, self.rot, self.kw, self.vw = cache.kcb, cache.vcb, cache.rot, cache.kw, cache.vw
        self.page_stride, self.head_stride = self.page, cache.capacity
        self.kcodes, self.kscales, self.vcodes, self.vscales = cache.kcodes, cache.kscales, cache.vcodes, cache.vscales
        return self

    def c(self) -> tq_kv_pages_t:
        """The descriptor of what the handle holds now."""
        torch, dev = _torch(), self.kcodes.get_device()
        kcb, vcb, rot, rows = self.kcb, self.vcb, self.rot, self.pages * self.page * self.heads
        if (self.pages - 1) * self.page_stride + (self.heads - 1) * self.head_stride + self.page > rows and self.pages > 0:
            raise ValueError("the cache's strides pass the end of its arrays")
        for name, width, size in (("kcodes", row_words(kcb.levels, self.dim), 4), ("kscales", self.dim // self.group, 2),
                                  ("vcodes", row_words(vcb.levels, self.dim), 4), ("vscales", self.dim // self.group, 2)):
            t = getattr(self, name)
            if t.numel() != rows * width or t.element_size() != size or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous: {rows} rows of {width} {8 * size}-bit words")
        for t, least, dtype in ((kcb.centroids, kcb.levels, torch.float32), (kcb.thresholds, kcb.levels - 1, torch.float32),
                                (vcb.centroids, vcb.levels, torch.float32), (vcb.thresholds, vcb.levels - 1, torch.float32),
                                (rot.signs, rot.dim, torch.int8)):
            if t.numel() < least or t.dtype is not dtype or not t.is_contiguous():
                raise ValueError("a book or the rotation's signs are too short, of another type or not contiguous")
        for t in (self.kcodes, self.kscales, self.vcodes, self.vscales, kcb.centroids, kcb.thresholds, vcb.centroids, vcb.thresholds,
                  rot.signs):
            if not t.is_cuda or t.get_device() != dev:
                raise ValueError("a cache's arrays, books and rotation must be on one CUDA device")
        return tq_kv_pages_t(self.kcodes.data_ptr(), self.kscales.data_ptr(), self.vcodes.data_ptr(),
                             self.vscales.data_ptr(), self.heads, self.dim, self.group, self.page, self.pages,
                             self.page_stride, self.head_stride, kcb.c(), vcb.c(), rot.c())

    _kept = None

    def _now(self):
        """(tensors, descriptor, workspace sizes, addresses, sizes), kept while all that the descriptor is made of, compared on
        every call, is the same."""
        kcb, vcb, rot = self.kcb, self.vcb, self.rot
        sizes = (kcb.levels, vcb.levels, rot.dim, rot.block, self.pages, self.page, self.heads, self.dim, self.group,
                 self.page_stride, self.head_stride)
        kept = self._kept
        if kept is not None and kept[4] == sizes:
            # a tensor may be another object at the same address (a view of other strides) or the same object at another
            (a, b, c, d, e, f, g, h, i), (pa, pb, pc, pd, pe, pf, pg, ph, pi) = kept[0], kept[3]
            if (self.kcodes is a and self.kscales is b and self.vcodes is c and self.vscales is d and kcb.centroids is e
                    and kcb.thresholds is f and vcb.centroids is g and vcb.thresholds is h and rot.signs is i
                    and a.data_ptr() == pa and b.data_ptr() == pb and c.data_ptr() == pc and d.data_ptr() == pd and e.data_ptr() == pe
                    and f.data_ptr() == pf and g.data_ptr() == pg and h.data_ptr() == ph and i.data_ptr() == pi):
                return kept
        tensors = (self.kcodes, self.kscales, self.vcodes, self.vscales, kcb.centroids, kcb.thresholds, vcb.centroids,
                   vcb.thresholds, rot.signs)
        kept = (tensors, self.c(), {}, tuple(t.data_ptr() for t in tensors), sizes)
        self._kept = kept  # in one piece: another thread finds the old or the new
        return kept

    def ref(self):
        return ctypes.byref(self._now()[1])

    def tree_bytes(self, B, n, hq, max_len) -> int:
        """Workspace of kv_attend_tree at these sizes."""
        return self._tree_bytes(self._now(), B, n, hq, max_len)

    def _tree_bytes(self, now, B, n, hq, max_len) -> int:
        c, sizes = now[1], now[2]
        key = (B, n, hq, max_len)
        nb = sizes.get(key)
        if nb is None:
            if len(sizes) > 4096:
                sizes.clear()
            nb = sizes[key] = int(load().tq_kv_attend_tree_workspace_bytes(ctypes.byref(c), B, n, hq, max_len))
        return nb


def kv_append(cache: PagedKVCache, k, v, slots, rope: Rope | None = None, positions=None, err=None):
    """Write tokens k, v [..., heads, dim] (f32 or bf16) to ``slots`` (int32, one per token; negative: skipped).

    With ``rope`` and ``positions`` the keys get their rotary positions on the way."""
    T, h, ks = _heads(k, "k", cache.dim)
    Tv, hv, vs = _heads(v, "v", cache.dim)
    dev = k.get_device()
    if T != Tv or h != hv or h != cache.heads or k.dtype is not v.dtype or v.get_device() != dev:
        raise ValueError("k and v must have the same tokens, the cache's heads, one dtype and one device")
    if cache.kcodes.get_device() != dev:
        raise ValueError("the cache must be on the tokens' device")
    at = _ints(slots, "slots", T, dev)
    turn, pos = None, 0
    if rope is not None:
        if positions is None:
            raise ValueError("rope needs positions")
        if rope.steps.get_device() != dev:
            raise ValueError("the rotary frequencies must be on the tokens' device")
        turn, pos = rope.ref(), _ints(positions, "positions", T, dev)
    _check(load().tq_kv_append(cache.ref(), k.data_ptr(), ks, v.data_ptr(), vs, _dt(k), T, at, turn, pos,
                               _word(err, dev), _raw_stream(k)), "tq_kv_append")


def kv_fetch(cache: PagedKVCache, slots, out_dtype=None, err=None):
    """The tokens of ``slots`` (int32 [T]) as (k, v) [T, heads, dim], bf16 unless told otherwise; a negative slot is zeros."""
    T, dev = slots.numel(), cache.kcodes.get_device()
    at = _ints(slots, "slots", T, dev)
    torch = _torch()
    shape, dtype, device = (T, cache.heads, cache.dim), out_dtype or torch.bfloat16, slots.device
    k, v = torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device)
    _check(load().tq_kv_fetch(cache.ref(), at, T, k.data_ptr(), v.data_ptr(), _dt(k), _word(err, dev),
                              _raw_stream(slots)), "tq_kv_fetch")
    return k, v


def kv_attend_tree(cache: PagedKVCache, q, table, lens, k_new=None, v_new=None, mask=None, n_tok=None,
                   max_len: int | None = None, scale: float | None = None, err=None, ws=None):
    """Attention of drafted tokens q [B, n, Hq, dim] (bf16) over each sequence's cached context and over the drafts.

    table: int32 [B, pages] page ids in order; lens: int32 [B] cached tokens; max_len: a bound on lens that
    the host knows (default: what the table can hold).  k_new, v_new: the drafts' own keys and values
    [B, n, heads, dim] (bf16); mask: int64 [B, n, ceil(n/64)], bit j of row i set where draft i sees draft j
    (None: a chain, j <= i); n_tok: int32 [B] drafts in use.  Returns [B, n, Hq, dim] bf16."""
    if q.dim() != 4:
        raise ValueError("q must be [B, n, heads, dim]")
    dim, dev = cache.dim, q.get_device()
    _, hq, qs = _heads(q, "q", dim)
    B, n, _, _ = q.shape
    if table.dim() != 2 or table.shape[0] != B:
        raise ValueError(f"table must be [{B}, pages]")
    wide = table.shape[1]
    tp, lp = _ints(table, "table", B * wide, dev), _ints(lens, "lens", B, dev)
    kp = vp = ks = vs = 0
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new go together")
    if k_new is not None:
        want = (B, n, cache.heads, dim)
        if k_new.shape != want or v_new.shape != want or k_new.dtype is not q.dtype or v_new.dtype is not q.dtype:
            raise ValueError(f"k_new and v_new must be {list(want)} of q's dtype")
        if k_new.get_device() != dev or v_new.get_device() != dev:
            raise ValueError("k_new and v_new must be on q's device")
        kp, ks, vp, vs = k_new.data_ptr(), _heads(k_new, "k_new", dim)[2], v_new.data_ptr(), _heads(v_new, "v_new", dim)[2]
    if cache.kcodes.get_device() != dev:
        raise ValueError("the cache must be on q's device")
    mp = 0 if mask is None else _ints(mask, "mask", B * n * (-(-n // 64)), dev, _torch().int64)
    np_ = 0 if n_tok is None else _ints(n_tok, "n_tok", B, dev)
    max_len = wide * cache.page if max_len is None else int(max_len)
    torch, device = _torch(), q.device
    o = torch.empty((B, n, hq, dim), dtype=torch.bfloat16, device=device)
    now = cache._now()
    nb = cache._tree_bytes(now, B, n, hq, max_len)
    if ws is not None and (ws.get_device() != dev or not ws.is_contiguous()):
        raise ValueError("ws must be contiguous, on q's device")
    if ws is None or ws.numel() * ws.element_size() < nb:
        ws = torch.empty(nb, dtype=torch.uint8, device=device)
    _check(load().tq_kv_attend_tree(ctypes.byref(now[1]), q.data_ptr(), qs, _dt(q), B, n, hq, tp, wide, lp, max_len, kp, ks, vp, vs, mp,
                                    np_, dim ** -0.5 if scale is None else scale, o.data_ptr(), ws.data_ptr(), nb,
                                    _word(err, dev), _raw_stream(q)), "tq_kv_attend_tree")
    return o


# ---------------------------------------------------------------- pages of a step

class PagePool:
    """The pages of a paged cache and which sequence holds which, on the device.

    ``table`` int32 [batch, width] (page ids in order, -1 past the pages held), ``held`` int32 [batch], ``free`` int32 [pages] (a
    stack: its first ``n_free`` entries) and ``n_free`` int32 [1]; ``storage``: these four instead of new ones."""

    def __init__(self, pages: int, page: int, batch: int, width: int, device="cuda", storage=None):
        torch = _torch()
        self.pages, self.page, self.batch, self.width = int(pages), int(page), int(batch), int(width)
        if storage is None:
            self.table = torch.full((self.batch, self.width), -1, dtype=torch.int32, device=device)
            self.held = torch.zeros(self.batch, dtype=torch.int32, device=device)
            self.free = torch.arange(self.pages - 1, -1, -1, dtype=torch.int32, device=device)  # page 0 is the first to go
            self.n_free = torch.full((1,), self.pages, dtype=torch.int32, device=device)
        else:
            self.table, self.held, self.free, self.n_free = storage

    _kept = None

    def _refs(self):
        """(descriptor, device, tensors, what they and the sizes were), kept while all of it, compared on every call, is the same."""
        table, held, free, n_free = tensors = self.table, self.held, self.free, self.n_free
        now = (table.data_ptr(), held.data_ptr(), free.data_ptr(), n_free.data_ptr(), self.batch, self.width, self.page, self.pages)
        kept = self._kept
        if kept is not None and kept[3] == now:
            a, b, c, d = kept[2]
            if table is a and held is b and free is c and n_free is d:
                return kept
        dev = table.get_device()
        if not self.table.is_cuda:
            raise ValueError("a pool's tensors must be on a CUDA device")
        c = tq_page_pool_t(_ints(table, "table", self.batch * self.width, dev), _ints(held, "held", self.batch, dev),
                           _ints(free, "free", self.pages, dev), _ints(n_free, "n_free", 1, dev), self.batch, self.width, self.page,
                           self.pages)
        self._kept = kept = (c, dev, tensors, now)  # in one piece: another thread finds the old or the new
        return kept


Plan = collections.namedtuple("Plan", "slots positions lens starts")


def kv_plan(pool: PagePool, lens, n_new, n: int | None = None, tokens: int | None = None, path=None, err=None) -> Plan:
    """Pages for n_new[b] tokens that join sequences of lens[b] tokens (int32 [batch]), taken from or given back to the pool.

    ``n``: slots and positions as int32 [batch, n], token i of a sequence in column i, or in column path[b, i] (int32 [batch, n]:
    the accepted nodes of ``verify_tree``).  ``tokens`` instead: packed as int32 [tokens], sequence b's from starts[b] on.  Places
    without a token have slot -1.  Returns (slots, positions, the lengths afterwards, starts or None)."""
    if (n is None) == (tokens is None):
        raise ValueError("either n (padded) or tokens (packed) is given")
    if n is not None and n < 1 or tokens is not None and (tokens < 0 or path is not None):
        raise ValueError("n must be at least 1, tokens at least 0 and without a path")
    torch = _torch()
    (c, dev, _, _), B = pool._refs(), pool.batch
    lp, wp = _ints(lens, "lens", B, dev), _ints(n_new, "n_new", B, dev)
    pp = 0 if path is None else _ints(path, "path", B * n, dev)
    shape, device = ((B, n) if n is not None else (tokens,)), lens.device
    slots = torch.empty(shape, dtype=torch.int32, device=device)
    positions = torch.empty(shape, dtype=torch.int32, device=device)
    after = torch.empty(B, dtype=torch.int32, device=device)
    starts = None if n is not None else torch.empty(B + 1, dtype=torch.int32, device=device)
    _check(load().tq_kv_plan(ctypes.byref(c), lp, wp, pp, n or 0, tokens or 0, slots.data_ptr(), positions.data_ptr(), after.data_ptr(),
                             0 if starts is None else starts.data_ptr(), _word(err, dev), _raw_stream(pool.table)), "tq_kv_plan")
    return Plan(slots, positions, after, starts)


# ---------------------------------------------------------------- verification of drafted tokens

def _distributions(t, name, B, n, V):
    """Row stride of distributions [B, n, V] whose rows lie at one stride."""
    if t.shape != (B, n, V) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [{B}, {n}, {V}]")
    sb, sn, sv = t.stride()
    if (V > 1 and sv != 1) or (B > 1 and n > 1 and sb != n * sn):
        raise ValueError(f"{name}'s rows must be contiguous and lie at one stride")
    step = sn if n > 1 else sb if B > 1 else V
    if step < V:
        raise ValueError(f"{name}'s rows must not overlap (an expanded tensor has to be made contiguous)")
    return step


def verify_tree(p, tokens, parent, u, q=None, n_tok=None, err=None):
    """Verifies drafted trees against the target's probabilities p [B, n, V] (f32, bf16 or f16) from uniform numbers u f32 [B, n].

    Node 0 of a tree is its root; node i has tokens[b, i], parent[b, i] < i (int32 [B, n]).  q [B, n, V]: the distributions that each
    node's children were drawn from, independently of one another and with replacement (else the tokens do not follow the target, without
    an error); None: they were chosen, as a draft's likeliest tokens are, not drawn.  n_tok: int32 [B] nodes in use.
    Returns (path int32 [B, n]: the accepted nodes in order, then -1; count int32 [B]; next int32 [B]: the token after them)."""
    if p.dim() != 3:
        raise ValueError("p must be [B, n, V]")
    torch, dev = _torch(), p.get_device()
    B, n, V = p.shape
    ps, qs, qp = _distributions(p, "p", B, n, V), 0, 0
    if q is not None:
        if q.dtype is not p.dtype or q.get_device() != dev:
            raise ValueError("q must have p's dtype and device")
        qs, qp = _distributions(q, "q", B, n, V), q.data_ptr()
    tp, pp = _ints(tokens, "tokens", B * n, dev), _ints(parent, "parent", B * n, dev)
    up = _ints(u, "u", B * n, dev, torch.float32)
    cp = 0 if n_tok is None else _ints(n_tok, "n_tok", B, dev)
    path = torch.empty((B, n), dtype=torch.int32, device=p.device)
    count = torch.empty(B, dtype=torch.int32, device=p.device)
    following = torch.empty(B, dtype=torch.int32, device=p.device)
    _check(load().tq_verify_tree(p.data_ptr(), ps, qp, qs, _dt(p), B, n, V, tp, pp, up, cp, path.data_ptr(), count.data_ptr(),
                                 following.data_ptr(), _word(err, dev), _raw_stream(p)), "tq_verify_tree")
    return path, count, following


# ---------------------------------------------------------------- latent attention

class LatentCache:
    """A paged cache of latent attention: rows [pages, page, latent + rope] (bf16 or f16), a token's latent vector and its rotary
    key, shared by all heads.  ``storage``: a tensor to use instead of a new one."""

    def __init__(self, pages: int, page: int, latent: int = 512, rope: int = 64, dtype=None, device="cuda", storage=None):
        torch = _torch()
        self.pages, self.page, self.latent, self.rope = int(pages), int(page), int(latent), int(rope)
        self.rows = storage
        if storage is None:
            self.rows = torch.zeros((self.pages, self.page, self.latent + self.rope), dtype=dtype or torch.bfloat16, device=device)
        elif dtype is not None and storage.dtype is not dtype:
            raise ValueError("storage must have the cache's dtype")
        self.c()

    def c(self) -> tq_latent_pages_t:
        """The descriptor of what the handle holds now."""
        t = self.rows
        if not t.is_cuda or tuple(t.shape) != (self.pages, self.page, self.latent + self.rope) or not t.is_contiguous():
            raise ValueError(f"rows must be a contiguous CUDA tensor [{self.pages}, {self.page}, {self.latent + self.rope}]")
        if t.element_size() != 2 or not t.is_floating_point():
            raise ValueError("rows must be bf16 or f16")
        return tq_latent_pages_t(t.data_ptr(), _dt(t), self.latent, self.rope, self.page, self.pages, self.page)

    _kept = None

    def _now(self):
        """(rows, descriptor, workspace sizes, what they were), kept while all that the descriptor is made of is the same."""
        rows = self.rows
        now = (rows.data_ptr(), self.latent, self.rope, self.page, self.pages)
        kept = self._kept
        if kept is None or kept[0] is not rows or kept[3] != now:
            self._kept = kept = (rows, self.c(), {}, now)  # in one piece: another thread finds the old or the new
        return kept

    def _tree_bytes(self, now, B, n, H, max_len) -> int:
        sizes, key = now[2], (B, n, H, max_len)
        nb = sizes.get(key)
        if nb is None:
            if len(sizes) > 4096:
                sizes.clear()
            nb = sizes[key] = int(load().tq_latent_attend_tree_workspace_bytes(ctypes.byref(now[1]), B, n, H, max_len))
        return nb


def _rows_at(t, name, width):
    """(rows, row stride) of t [..., width] whose rows lie at one stride."""
    if t.is_cuda:  # the usual cases, without a view (which takes as long as the call itself)
        shape, strides = t.shape, t.stride()
        if len(shape) == 2 and shape[1] == width and strides[1] == 1:
            return shape[0], strides[0] if shape[0] > 1 else width
        if len(shape) == 3 and shape[2] == width and strides[2] == 1:
            (a, b, _), (sa, sb, _) = shape, strides
            if b == 1:
                return a, sa if a > 1 else width
            if a == 1 or (a > 1 and b > 1 and sa == b * sb):
                return a * b, sb
    tokens, _, stride = _heads(t.unsqueeze(-2), name, width)
    return tokens, stride


def latent_append(cache: LatentCache, c, k_rope, slots, rope: Rope | None = None, positions=None, err=None):
    """Write latent vectors c [..., latent] and rotary keys k_rope [..., rope] (f32, bf16 or f16; views of a fused projection are
    fine) to ``slots`` (int32, one per token; negative: skipped).  With ``rope`` and ``positions`` the keys get their rotary
    positions on the way."""
    T, cs = _rows_at(c, "c", cache.latent)
    Tk, ks = _rows_at(k_rope, "k_rope", cache.rope)
    dev = c.get_device()
    if T != Tk or c.dtype is not k_rope.dtype or k_rope.get_device() != dev or cache.rows.get_device() != dev:
        raise ValueError("c, k_rope and the cache must have the same tokens, dtype and device")
    at = _ints(slots, "slots", T, dev)
    turn, pos = None, 0
    if rope is not None:
        if positions is None:
            raise ValueError("rope needs positions")
        if rope.steps.get_device() != dev:
            raise ValueError("the rotary frequencies must be on the tokens' device")
        turn, pos = rope.ref(), _ints(positions, "positions", T, dev)
    _check(load().tq_latent_append(ctypes.byref(cache._now()[1]), c.data_ptr(), cs, k_rope.data_ptr(), ks, _dt(c), T, at, turn, pos,
                                   _word(err, dev), _raw_stream(c)), "tq_latent_append")


def latent_attend_tree(cache: LatentCache, q, table, lens, scale: float, new=None, mask=None, n_tok=None,
                       max_len: int | None = None, err=None, ws=None):
    """Attention of drafted tokens over the latent cache (the absorbed form): q [B, n, H, latent + rope] of the cache's dtype, each
    head's query through its key projection and its rotary part.

    table, lens, max_len, mask, n_tok: as of ``kv_attend_tree``; new: the drafts' own rows [B, n, latent + rope].  scale: of the
    scores, 1 / sqrt(length of an expanded query) in a model.  Returns [B, n, H, latent] (each head's value projection is to follow)."""
    if q.dim() != 4:
        raise ValueError("q must be [B, n, heads, latent + rope]")
    width, dev = cache.latent + cache.rope, q.get_device()
    _, H, qs = _heads(q, "q", width)
    B, n, _, _ = q.shape
    if q.dtype is not cache.rows.dtype or cache.rows.get_device() != dev:
        raise ValueError("q must have the cache's dtype and device")
    if table.dim() != 2 or table.shape[0] != B:
        raise ValueError(f"table must be [{B}, pages]")
    wide = table.shape[1]
    tp, lp = _ints(table, "table", B * wide, dev), _ints(lens, "lens", B, dev)
    fp = fs = 0
    if new is not None:
        if new.shape != (B, n, width) or new.dtype is not q.dtype or new.get_device() != dev:
            raise ValueError(f"new must be {[B, n, width]} of q's dtype and device")
        fp, fs = new.data_ptr(), _rows_at(new, "new", width)[1]
    mp = 0 if mask is None else _ints(mask, "mask", B * n * (-(-n // 64)), dev, _torch().int64)
    np_ = 0 if n_tok is None else _ints(n_tok, "n_tok", B, dev)
    max_len = wide * cache.page if max_len is None else int(max_len)
    torch, device, now = _torch(), q.device, cache._now()
    o = torch.empty((B, n, H, cache.latent), dtype=q.dtype, device=device)
    nb = cache._tree_bytes(now, B, n, H, max_len)
    if ws is not None and (ws.get_device() != dev or not ws.is_contiguous()):
        raise ValueError("ws must be contiguous, on q's device")
    if ws is None or ws.numel() * ws.element_size() < nb:
        ws = torch.empty(nb, dtype=torch.uint8, device=device)
    _check(load().tq_latent_attend_tree(ctypes.byref(now[1]), q.data_ptr(), qs, B, n, H, tp, wide, lp, max_len, fp, fs, mp, np_, scale,
                                        o.data_ptr(), ws.data_ptr(), nb, _word(err, dev), _raw_stream(q)), "tq_latent_attend_tree")
    return o


def latent_attend_prompt(q, k, v, k_rope, q_starts, kv_starts, scale: float, causal: bool = True, err=None, ws=None):
    """Attention of packed prompts over keys and values expanded from the latents (the expanded form).

    q [Tq, H, 192] (the last 64 with rotary positions), k and v [Tkv, H, 128] (the two halves of one expansion [Tkv, H, 256] are
    fine), k_rope [Tkv, 64] for all heads, bf16 or f16; q_starts, kv_starts: int32 [B + 1], sequence b's queries and keys.  Its
    last query stands at its last key; a query sees the keys up to its own place (causal=False: all).  Returns [Tq, H, 128]; queries of
    no sequence (behind the last one, or of starts that are out of order, which err reports) give zeros."""
    torch, dev = _torch(), q.get_device()
    Tq, H, qs = _heads(q, "q", 192)
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape or k.shape[1:] != (H, 128):
        raise ValueError("q must be [Tq, H, 192], k and v [Tkv, H, 128]")
    Tkv = k.shape[0]
    if k.stride() != v.stride() or k.stride(-1) != 1:
        raise ValueError("k and v must have the same strides, their heads' elements one after another")
    Tr, rs = _rows_at(k_rope, "k_rope", 64)
    if Tr != Tkv or not k.dtype is v.dtype is k_rope.dtype is q.dtype:
        raise ValueError("k, v and k_rope must have the same tokens and q's dtype")
    if not k.get_device() == v.get_device() == k_rope.get_device() == dev:
        raise ValueError("k, v and k_rope must be on q's device")
    B = q_starts.numel() - 1
    if B < 0:
        raise ValueError("q_starts must have an entry more than there are sequences")
    qp, kp = _ints(q_starts, "q_starts", B + 1, dev), _ints(kv_starts, "kv_starts", B + 1, dev)
    hs = k.stride(1) if H > 1 else 128
    ks = k.stride(0) if Tkv > 1 else max(k.stride(0), (H - 1) * hs + 128)
    o = (torch.empty if B else torch.zeros)((Tq, H, 128), dtype=q.dtype, device=q.device)
    nb = int(load().tq_latent_attend_prompt_workspace_bytes(B, H, Tq, Tkv))
    if ws is not None and (ws.get_device() != dev or not ws.is_contiguous()):
        raise ValueError("ws must be contiguous, on q's device")
    if ws is None or ws.numel() * ws.element_size() < nb:
        ws = torch.empty(nb, dtype=torch.uint8, device=q.device)
    _check(load().tq_latent_attend_prompt(q.data_ptr(), qs, k.data_ptr(), v.data_ptr(), ks, hs, k_rope.data_ptr(), rs, _dt(q), B, H, Tq,
                                          Tkv, qp, kp, int(causal), scale, o.data_ptr(), ws.data_ptr(), nb, _word(err, dev), _raw_stream(q)),
           "tq_latent_attend_prompt")
    return o


def moe_decode_layer(gate_up: QWeight, down: QWeight, rot_h: Rotation, rot_i: Rotation, logits, x, k: int,
                     out_dtype=None, err=None, ws=None):
    """One token through the MoE layer in one launch: route, rotate, gate||up, SwiGLU + rotate, down,
    combine.  logits: f32 [E] (or [1, E]); x: [H] (or [1, H]) f32/bf16/f16.  Returns out [1, H]."""
    torch = _torch()
    _contig(logits, "logits")
    _contig(x, "x")
    H = gate_up.cols
    out = torch.empty((1, H), dtype=out_dtype or torch.float32, device=x.device)
    g, d, rh, ri = gate_up.c(), down.c(), rot_h.c(), rot_i.c()
    nb = int(load().tq_moe_decode_layer_workspace_bytes(ctypes.byref(g), ctypes.byref(d), k))
    ws = _workspace(nb, x.device, ws)
    _check(load().tq_moe_decode_layer(ctypes.byref(g), ctypes.byref(d), ctypes.byref(rh), ctypes.byref(ri),
                                      _ptr(logits), _ptr(x), _dt(x), k, _ptr(out), _dt(out), _ptr(ws), nb, _ptr(err),
                                      _stream()), "tq_moe_decode_layer")
    return out


def check_error(err) -> int:
    """Synchronises, returns the device error bits and clears them."""
    bits = _u32(0)
    st = load().tq_check_error(_ptr(err), ctypes.byref(bits), _stream())
    if st not in (TQ_OK, TQ_ERR_TIMEOUT, TQ_ERR_DEVICE):
        _check(st, "tq_check_error")
    return int(bits.value)


def set_wait_budget(cycles: int) -> None:
    """Test hook: cycle budget of the tensor-core kernels' bounded waits (-1: the default)."""
    _check(load().tq_set_wait_budget(int(cycles)), "tq_set_wait_budget")


def selftest_trit_decode(first: int = 0, count: int = 3 ** 20) -> int:
    torch = _torch()
    m = torch.zeros(1, dtype=torch.int64, device="cuda")
    _check(load().tq_selftest_trit_decode(first, count, _ptr(m), _stream()), "tq_selftest_trit_decode")
    return int(m.item())


# ---------------------------------------------------------------- per-layer tiers and the packed file

# "How it works": ternary experts, 4-bit down projections, 3-bit protected layers; group 16 for
# MLP and expert layers.
DEFAULT_TIERS = {"down": (16, 16), "expert": (3, 16), "mlp": (8, 16), "attn": (8, 64), "other": (8, 64)}


def tier_policy(tiers: dict | None = None) -> tq_tier_policy_t:
    t = dict(DEFAULT_TIERS, **(tiers or {}))
    return tq_tier_policy_t(t["down"][0], t["down"][1], t["expert"][0], t["expert"][1], t["mlp"][0], t["mlp"][1],
                            t["attn"][0], t["attn"][1], t["other"][0], t["other"][1])


def layer_tier(name: str, policy: tq_tier_policy_t | None = None) -> tuple[int, int]:
    """(codebook size, group) of layer `name` under the tier policy."""
    lv, g = _i32(0), _i32(0)
    pol = policy if policy is not None else tier_policy()
    _check(load().tq_layer_tier(name.encode(), ctypes.byref(pol), ctypes.byref(lv), ctypes.byref(g)), "tq_layer_tier")
    return int(lv.value), int(g.value)


class PackedLayer:
    """A layer as stored in a packed file: host numpy arrays and their metadata."""

    def __init__(self, name, codes, scales, centroids, group, rot_block, rot_seed):
        self.name = name
        self.codes = np.ascontiguousarray(codes, dtype=np.uint32)        # [experts, rows, row_stride]
        self.scales = np.ascontiguousarray(scales).view(np.uint16)        # [experts, rows, cols/group]
        self.centroids = np.ascontiguousarray(centroids, dtype=np.float64)
        self.experts, self.rows, self.row_stride = self.codes.shape
        self.group = int(group)
        self.cols = self.scales.shape[-1] * self.group
        self.rot_block, self.rot_seed = int(rot_block), int(rot_seed)

    @property
    def levels(self) -> int:
        return len(self.centroids)

    def qweight(self, device="cuda") -> "QWeight":
        """The layer on the device (its codebook's thresholds are the midpoints of the centroids)."""
        torch = _torch()
        c = self.centroids
        cb = Codebook(self.levels, device=device, centroids=c, thresholds=(c[1:] + c[:-1]) / 2)
        codes = torch.from_numpy(self.codes.view(np.int32)).to(device)
        scales = torch.from_numpy(self.scales.view(np.int16)).to(device)
        return QWeight(codes, scales, self.experts, self.rows, self.cols, self.group, cb, row_stride=self.row_stride)


def save_packed(path: str, layers: list[PackedLayer]) -> None:
    descs = (tq_layer_desc_t * max(len(layers), 1))()
    for d, L in zip(descs, layers):
        d.name = L.name.encode()
        d.experts, d.rows, d.cols, d.group = L.experts, L.rows, L.cols, L.group
        d.row_stride_words, d.levels = L.row_stride, L.levels
        d.rot_dim, d.rot_block, d.rot_seed = L.cols, L.rot_block, L.rot_seed
        d.centroids = L.centroids.ctypes.data
        d.codes = L.codes.ctypes.data
        d.scales = L.scales.ctypes.data
    _check(load().tq_pack_file_write(path.encode(), descs, len(layers)), "tq_pack_file_write")


def load_packed(path: str) -> list[PackedLayer]:
    lib = load()
    n = _i32(0)
    _check(lib.tq_pack_file_info(path.encode(), ctypes.byref(n), None, 0), "tq_pack_file_info")
    infos = (tq_layer_desc_t * max(n.value, 1))()
    _check(lib.tq_pack_file_info(path.encode(), ctypes.byref(n), infos, n.value), "tq_pack_file_info")
    out = []
    for i in range(n.value):
        d = infos[i]
        c = np.zeros(d.levels, np.float64)
        codes = np.zeros((d.experts, d.rows, d.row_stride_words), np.uint32)
        scales = np.zeros((d.experts, d.rows, d.cols // d.group), np.uint16)
        _check(lib.tq_pack_file_read_layer(path.encode(), i, c.ctypes.data, codes.ctypes.data, scales.ctypes.data),
               "tq_pack_file_read_layer")
        out.append(PackedLayer(d.name.decode(), codes, scales, c, d.group, d.rot_block, d.rot_seed))
    return out


# ---------------------------------------------------------------- expert streaming

class ExpertCache:
    """Experts of a bank held in host memory, streamed into ``slots`` device slots (LRU).

    ``codes`` (int32/uint32 [experts, rows, row_stride]) and ``scales`` (16-bit
    [experts, rows, cols/group]) are host arrays: pinned torch CPU tensors for
    ``map`` (the copies are asynchronous), or numpy arrays for ``plan`` alone.
    ``view`` is the slot bank on the device, a QWeight with ``slots`` experts
    that the gather entry points run on with ids remapped to slots.
    """

    def __init__(self, codes, scales, experts: int, rows: int, cols: int, group: int, cb: Codebook, slots: int,
                 row_stride: int | None = None, device="cuda"):
        self.host_codes, self.host_scales = codes, scales
        self.row_stride = int(row_stride if row_stride is not None else row_stride_words(cb.levels, cols))
        self.experts, self.rows, self.cols, self.group, self.slots = experts, rows, cols, group, int(slots)
        self.cb = cb
        cp = codes.data_ptr() if hasattr(codes, "data_ptr") else codes.ctypes.data
        sp = scales.data_ptr() if hasattr(scales, "data_ptr") else scales.ctypes.data
        host = tq_qweight_t(cp, sp, experts, rows, cols, group, self.row_stride, rows * self.row_stride,
                            rows * (cols // group), cb.c())
        self.view = None
        dc = ds = None
        if device is not None:
            torch = _torch()
            dcodes = torch.empty((self.slots, rows, self.row_stride), dtype=torch.int32, device=device)
            dscales = torch.empty((self.slots, rows, cols // group), dtype=torch.int16, device=device)
            self.view = QWeight(dcodes, dscales, self.slots, rows, cols, group, cb, row_stride=self.row_stride)
            dc, ds = dcodes.data_ptr(), dscales.data_ptr()
        h = _c_p()
        _check(load().tq_expert_cache_create(ctypes.byref(host), self.slots, dc, ds, ctypes.byref(h)),
               "tq_expert_cache_create")
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            _lib.tq_expert_cache_destroy(h)
            self._h = None

    @staticmethod
    def _ids(ids) -> np.ndarray:
        if hasattr(ids, "detach"):
            ids = ids.detach().to("cpu").numpy()
        return np.ascontiguousarray(np.asarray(ids).reshape(-1), dtype=np.int32)

    def plan(self, ids):
        """LRU bookkeeping only (host): (slot of each id, 1 where the id is a first miss)."""
        a = self._ids(ids)
        slots = np.zeros(a.size, np.int32)
        miss = np.zeros(a.size, np.uint8)
        _check(load().tq_expert_cache_plan(self._h, a.ctypes.data, a.size, slots.ctypes.data, miss.ctypes.data),
               "tq_expert_cache_plan")
        return slots, miss

    def map(self, ids):
        """Brings the experts of ``ids`` into the slots on the current stream; their slots (host int32)."""
        a = self._ids(ids)
        slots = np.zeros(a.size, np.int32)
        _check(load().tq_expert_cache_map(self._h, a.ctypes.data, a.size, slots.ctypes.data, _stream()),
               "tq_expert_cache_map")
        return slots

    def stats(self) -> tuple[int, int, int]:
        """(hits, misses, bytes copied) since creation."""
        h, m, b = _i64(0), _i64(0), _i64(0)
        _check(load().tq_expert_cache_stats(self._h, ctypes.byref(h), ctypes.byref(m), ctypes.byref(b)),
               "tq_expert_cache_stats")
        return int(h.value), int(m.value), int(b.value)

    def gather_qmv(self, x_rot, ids, out_dtype=None, err=None):
        """gather_qmv of the host bank: maps ``ids`` [T, k], then gathers from the slots."""
        torch = _torch()
        shape = tuple(ids.shape)
        slots = torch.from_numpy(self.map(ids)).reshape(shape).pin_memory().to(x_rot.device, non_blocking=True)
        return gather_qmv(self.view, x_rot, slots, out_dtype=out_dtype, err=err)
