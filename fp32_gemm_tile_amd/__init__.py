"""fp32_gemm_tile_amd -- true-fp32 SGEMM for MI355X (gfx950) behind a C ABI.

    C = alpha * op(A) * op(B) + beta * C     (row-major, see include/fp32gemm.h)

This module is a thin ctypes binding over ``libfp32gemm.so``: it marshals
arguments and nothing else; every step of the product runs in the library's
HIP kernels. There is no fallback: if the library is missing or cannot load,
importing the binding's functions raises.

Entry points (same names as the C ABI):
  fg_sgemm(...), fg_sgemm_ex(...)      raw pointers and sizes
  fg_sgemm_splitk(...), fg_sgemm_splitk_workspace_size(M, N, S)
  fg_num_configs(), fg_get_config(i), fg_select_config(...)
  fg_last_bad_arg(), fg_last_error(), fg_status_string(s), fg_abi_version()
  fg_quantize_fp8(...), fg_gemm_fp8(...), fg_moe(layer, ...)
Convenience:
  sgemm(A, B, C, alpha, beta, transA, transB, config=-1, stream=None)
      for torch tensors on the GPU (PyTorch only supplies memory and stream).
  quantize_fp8(X, Q, S, QT, ST, block), gemm_fp8(A, SA, B, SB, C, alpha, beta),
  empty_fp8(rows, cols, block)
      e4m3 codes with a scale for each block of 128 (include/fp32gemm_fp8.h)
  moe(x, gate, up, down, ids, weights, out, router, ...)
      a mixture-of-experts layer for a few tokens (include/fp32gemm_moe.h)
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp32gemm.so")

FG_OP_N, FG_OP_T = 0, 1
FG_OK, FG_ERR_INVALID_ARG, FG_ERR_HIP, FG_ERR_UNSUPPORTED = 0, 1, 2, 3
FG_KIND_MFMA, FG_KIND_VALU, FG_KIND_SKINNY = 1, 2, 3
FG_MAX_LD = 2097152


class FgError(RuntimeError):
    def __init__(self, status, bad_arg, message):
        self.status = status
        self.bad_arg = bad_arg
        super().__init__(f"{status_name(status)} (bad argument {bad_arg}): {message}")


class fg_config(ctypes.Structure):
    _fields_ = [("id", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("bm", ctypes.c_int32), ("bn", ctypes.c_int32), ("bk", ctypes.c_int32),
                ("wm", ctypes.c_int32), ("wn", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("lds_bytes", ctypes.c_int32), ("mr", ctypes.c_int32),
                ("name", ctypes.c_char * 40)]

    def as_dict(self):
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["name"] = self.name.decode()
        return d


FG_ACT_NONE, FG_ACT_RELU, FG_ACT_GELU, FG_ACT_SILU = 0, 1, 2, 3
_ACTS = {"none": FG_ACT_NONE, "relu": FG_ACT_RELU, "gelu": FG_ACT_GELU, "silu": FG_ACT_SILU}


class fg_epilogue(ctypes.Structure):
    _fields_ = [("row_scale", ctypes.c_void_p), ("col_scale", ctypes.c_void_p),
                ("row_bias", ctypes.c_void_p), ("col_bias", ctypes.c_void_p),
                ("activation", ctypes.c_int32)]


FG_QUANT_NONE, FG_QUANT_BF16, FG_QUANT_INT8_ROW = 0, 1, 2
_QUANTS = {"none": FG_QUANT_NONE, "bf16": FG_QUANT_BF16, "int8_row": FG_QUANT_INT8_ROW}


class fg_quant(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("out", ctypes.c_void_p), ("ldq", ctypes.c_int64),
                ("row_factor", ctypes.c_void_p)]


FG_TYPE_F32, FG_TYPE_BF16, FG_TYPE_E4M3 = 0, 1, 2
FG_BLOCK_ROW, FG_BLOCK_TILE = 0, 1
_BLOCKS = {"row": FG_BLOCK_ROW, "tile": FG_BLOCK_TILE}
FG_MOE_MAX_TOKENS, FG_MOE_MAX_TOP_K, FG_MOE_MAX_EXPERTS = 64, 16, 512


class fg_experts(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("ld", ctypes.c_int64), ("stride", ctypes.c_int64),
                ("scales", ctypes.c_void_p), ("lds", ctypes.c_int64),
                ("scale_stride", ctypes.c_int64)]


class fg_moe_layer(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inner", ctypes.c_int32),
                ("type", ctypes.c_int32), ("weight_type", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("gate", fg_experts), ("up", fg_experts), ("down", fg_experts),
                ("router", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("router_type", ctypes.c_int32), ("ids", ctypes.c_void_p),
                ("weights", ctypes.c_void_p), ("out", ctypes.c_void_p), ("ldo", ctypes.c_int64)]


def make_quant(kind, out, ldq, row_factor=0):
    """fg_quant from a format ("bf16", "int8_row" or an fg_quant_kind), the
    device address of Q, its leading dimension and (int8_row) the device
    address of the M row factors."""
    k = _QUANTS[kind] if isinstance(kind, str) else int(kind)
    return fg_quant(k, out or None, ldq, row_factor or None)


def activation_code(act) -> int:
    """fg_activation value of "none" / "relu" / "gelu" / "silu" (or an int)."""
    if isinstance(act, str):
        if act not in _ACTS:
            raise ValueError(f"unknown activation {act!r}")
        return _ACTS[act]
    return int(act)


def make_epilogue(row_scale=0, col_scale=0, row_bias=0, col_bias=0, activation="none"):
    """fg_epilogue from device addresses (0 = not used) and an activation."""
    return fg_epilogue(row_scale or None, col_scale or None, row_bias or None,
                       col_bias or None, activation_code(activation))


_lib = None


def load_library(path: str = LIB_PATH):
    """Load (once) and return the ctypes handle. Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`"
            " (there is no non-HIP fallback)")
    # One HIP runtime per process: PyTorch ships its own libamdhip64 (same
    # SONAME as the system one). Importing torch first makes the dynamic
    # loader bind this library to that copy, so torch's streams and device
    # pointers are the ones the library's runtime knows.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    i64, i32, f32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p
    gemm_args = [i32, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
    lib.fg_sgemm.argtypes = gemm_args
    lib.fg_sgemm.restype = i32
    lib.fg_sgemm_ex.argtypes = gemm_args + [i32]
    lib.fg_sgemm_ex.restype = i32
    lib.fg_sgemm_splitk.argtypes = gemm_args[:13] + [i32, vp, ctypes.c_size_t, vp]
    lib.fg_sgemm_splitk.restype = i32
    lib.fg_sgemm_splitk_noalloc.argtypes = gemm_args[:13] + [i32, vp]
    lib.fg_sgemm_splitk_noalloc.restype = i32
    lib.fg_sgemm_splitk_noalloc_max_bytes.argtypes = []
    lib.fg_sgemm_splitk_noalloc_max_bytes.restype = ctypes.c_size_t
    lib.fg_sgemm_splitk_workspace_size.argtypes = [i64, i64, i32]
    lib.fg_sgemm_splitk_workspace_size.restype = ctypes.c_size_t
    lib.fg_num_configs.argtypes = []
    lib.fg_num_configs.restype = i32
    lib.fg_get_config.argtypes = [i32, ctypes.POINTER(fg_config)]
    lib.fg_get_config.restype = i32
    lib.fg_select_config.argtypes = [i32, i32, i64, i64, i64, vp, i64, vp, i64, vp, i64,
                                     ctypes.POINTER(fg_config)]
    lib.fg_select_config.restype = i32
    lib.fg_select_config_quant.argtypes = [i32, i32, i64, i64, i64, vp, i64, vp, i64, vp, i64,
                                           i32, ctypes.POINTER(fg_config)]
    lib.fg_select_config_quant.restype = i32
    lib.fg_select_config_ex.argtypes = [i32, i32, i64, i64, i64, vp, i64, vp, i64, f32, vp, i64,
                                        i32, ctypes.c_size_t, i32, ctypes.POINTER(fg_config),
                                        ctypes.POINTER(i32)]
    lib.fg_select_config_ex.restype = i32
    lib.fg_last_bad_arg.argtypes = []
    lib.fg_last_bad_arg.restype = i32
    lib.fg_last_error.argtypes = []
    lib.fg_last_error.restype = ctypes.c_char_p
    lib.fg_status_string.argtypes = [i32]
    lib.fg_status_string.restype = ctypes.c_char_p
    lib.fg_abi_version.argtypes = []
    lib.fg_abi_version.restype = i32
    lib.fg_sgemm_streamk.argtypes = gemm_args[:13] + [vp, ctypes.c_size_t, vp]
    lib.fg_sgemm_streamk.restype = i32
    lib.fg_sgemm_streamk_workspace_size.argtypes = [i32, i32, i64, i64, i64, vp, i64, vp, i64]
    lib.fg_sgemm_streamk_workspace_size.restype = ctypes.c_size_t
    lib.fg_sgemm_fused.argtypes = gemm_args[:13] + [ctypes.POINTER(fg_epilogue), vp, i32]
    lib.fg_sgemm_fused.restype = i32
    lib.fg_sgemm_quant.argtypes = gemm_args[:13] + [ctypes.POINTER(fg_epilogue),
                                                    ctypes.POINTER(fg_quant), vp, i32]
    lib.fg_sgemm_quant.restype = i32
    lib.fg_quantize_fp8.argtypes = [i32, i32, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp,
                                    i64, vp]
    lib.fg_quantize_fp8.restype = i32
    lib.fg_gemm_fp8.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, vp, i64, vp, i64, i32, f32,
                                vp, i64, i32, vp, ctypes.c_size_t, vp]
    lib.fg_gemm_fp8.restype = i32
    lib.fg_fp8_num_tiles.argtypes = []
    lib.fg_fp8_num_tiles.restype = i32
    lib.fg_fp8_tile.argtypes = [i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]
    lib.fg_fp8_tile.restype = i32
    lib.fg_select_fp8.argtypes = [i64, i64, i64, ctypes.c_size_t, ctypes.POINTER(i32),
                                  ctypes.POINTER(i32)]
    lib.fg_select_fp8.restype = i32
    lib.fg_set_fp8_tile.argtypes = [i32]
    lib.fg_set_fp8_tile.restype = i32
    lib.fg_gemm_fp8_workspace_size.argtypes = [i64, i64, i64]
    lib.fg_gemm_fp8_workspace_size.restype = ctypes.c_size_t
    if _MOE_RECORD.size != ctypes.sizeof(fg_moe_layer):
        raise ImportError("fg_moe_layer: the packed record does not match the structure")
    lib.fg_moe.argtypes = [ctypes.POINTER(fg_moe_layer), vp, ctypes.c_size_t, vp]
    lib.fg_moe.restype = i32
    lib.fg_moe_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.fg_moe_workspace_size.restype = ctypes.c_size_t
    lib.fg_estimate_seconds.argtypes = [i64, i64, i64, i32, i32, i32]
    lib.fg_estimate_seconds.restype = ctypes.c_double
    lib.fg_get_efficiency.argtypes = [i32, ctypes.POINTER(ctypes.c_double),
                                      ctypes.POINTER(ctypes.c_double)]
    lib.fg_get_efficiency.restype = i32
    lib.fg_set_efficiency.argtypes = [i32, ctypes.c_double, ctypes.c_double]
    lib.fg_set_efficiency.restype = i32
    lib.fg_set_raster.argtypes = [i32, i32]
    lib.fg_set_raster.restype = i32
    lib.fg_get_raster.argtypes = [ctypes.POINTER(i32), ctypes.POINTER(i32)]
    lib.fg_get_raster.restype = i32
    lib.fg_set_few_row_threads.argtypes = [i32]
    lib.fg_set_few_row_threads.restype = i32
    lib.fg_set_few_row_kernel.argtypes = [i32]
    lib.fg_set_few_row_kernel.restype = i32
    lib.fg_get_model_constant.argtypes = [i32, ctypes.POINTER(ctypes.c_double)]
    lib.fg_get_model_constant.restype = i32
    lib.fg_set_model_constant.argtypes = [i32, ctypes.c_double]
    lib.fg_set_model_constant.restype = i32
    lib.fg_set_streamk_policy.argtypes = [i32]
    lib.fg_set_streamk_policy.restype = i32
    lib.fg_probe_mfma.argtypes = [i32, i32, vp, vp]
    lib.fg_probe_mfma.restype = i32
    lib.fg_probe_mfma_flops.argtypes = [i32, i32]
    lib.fg_probe_mfma_flops.restype = ctypes.c_double
    lib.fg_probe_lds_dma.argtypes = [vp, i32, vp, vp]
    lib.fg_probe_lds_dma.restype = i32
    lib.fg_probe_read.argtypes = [vp, i64, i32, vp, vp]
    lib.fg_probe_read.restype = i32
    _lib = lib
    return lib


def _op(t) -> int:
    if t in (0, 1):
        return int(t)
    if isinstance(t, str) and t.upper() in ("N", "T"):
        return FG_OP_T if t.upper() == "T" else FG_OP_N
    return int(t)  # let the library reject out-of-domain values


def status_name(s: int) -> str:
    return load_library().fg_status_string(int(s)).decode()


def _raise_if(st: int):
    if st != FG_OK:
        lib = load_library()
        raise FgError(st, lib.fg_last_bad_arg(), lib.fg_last_error().decode())


# ---- C-ABI mirror ---------------------------------------------------------

def fg_sgemm(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0):
    """Raw call: A, B, C are device addresses (int), stream a hipStream_t (int)."""
    return load_library().fg_sgemm(_op(transA), _op(transB), M, N, K, alpha, A, lda,
                                   B, ldb, beta, C, ldc, stream or None)


def fg_sgemm_ex(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0,
                config_id=-1):
    return load_library().fg_sgemm_ex(_op(transA), _op(transB), M, N, K, alpha, A, lda,
                                      B, ldb, beta, C, ldc, stream or None, config_id)


def fg_sgemm_splitk(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, splits,
                    workspace, workspace_bytes, stream=0):
    """Raw split-K call (see include/fp32gemm.h); workspace is a device address."""
    return load_library().fg_sgemm_splitk(_op(transA), _op(transB), M, N, K, alpha, A, lda,
                                          B, ldb, beta, C, ldc, splits, workspace or None,
                                          workspace_bytes, stream or None)


def fg_sgemm_splitk_noalloc(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                            splits, stream=0):
    """Split-K with the library's own device-resident scratch (no workspace
    argument, nothing allocated); see include/fp32gemm.h."""
    return load_library().fg_sgemm_splitk_noalloc(_op(transA), _op(transB), M, N, K, alpha, A,
                                                  lda, B, ldb, beta, C, ldc, splits,
                                                  stream or None)


def fg_sgemm_splitk_noalloc_max_bytes() -> int:
    return load_library().fg_sgemm_splitk_noalloc_max_bytes()


def fg_sgemm_splitk_workspace_size(M, N, splits) -> int:
    return load_library().fg_sgemm_splitk_workspace_size(M, N, splits)


def fg_num_configs() -> int:
    return load_library().fg_num_configs()


def fg_get_config(i: int) -> dict:
    c = fg_config()
    _raise_if(load_library().fg_get_config(i, ctypes.byref(c)))
    return c.as_dict()


def fg_select_config(transA, transB, M, N, K, A=0, lda=None, B=0, ldb=None, C=0,
                     ldc=None, quant=None) -> dict:
    """The entry fg_sgemm would run (with quant, a format name or FG_QUANT_*
    code: the entry fg_sgemm_quant would run)."""
    ta, tb = _op(transA), _op(transB)
    lda = lda if lda is not None else max(1, K if ta == FG_OP_N else M)
    ldb = ldb if ldb is not None else max(1, N if tb == FG_OP_N else K)
    ldc = ldc if ldc is not None else max(1, N)
    c = fg_config()
    lib = load_library()
    if quant is None:
        _raise_if(lib.fg_select_config(ta, tb, M, N, K, A or None, lda, B or None, ldb,
                                       C or None, ldc, ctypes.byref(c)))
    else:
        kind = quant if isinstance(quant, int) else _QUANTS[quant]
        _raise_if(lib.fg_select_config_quant(ta, tb, M, N, K, A or None, lda, B or None, ldb,
                                             C or None, ldc, kind, ctypes.byref(c)))
    return c.as_dict()


def fg_select_config_ex(transA, transB, M, N, K, A=0, lda=None, B=0, ldb=None, beta=0.0, C=0,
                        ldc=None, splits=1, workspace_bytes=0, quant=None):
    """(entry, split-K slices) a call runs with config_id -1: fg_sgemm
    (splits=1), fg_sgemm_splitk (splits 0 = library choice bounded by
    workspace_bytes, or a count) or fg_sgemm_quant (quant, a format name or
    FG_QUANT_* code), with beta taken into account."""
    ta, tb = _op(transA), _op(transB)
    lda = lda if lda is not None else max(1, K if ta == FG_OP_N else M)
    ldb = ldb if ldb is not None else max(1, N if tb == FG_OP_N else K)
    ldc = ldc if ldc is not None else max(1, N)
    kind = 0 if quant is None else (quant if isinstance(quant, int) else _QUANTS[quant])
    c = fg_config()
    n = ctypes.c_int32(0)
    _raise_if(load_library().fg_select_config_ex(ta, tb, M, N, K, A or None, lda, B or None, ldb,
                                                 beta, C or None, ldc, splits, workspace_bytes,
                                                 kind, ctypes.byref(c), ctypes.byref(n)))
    return c.as_dict(), n.value


def fg_last_bad_arg() -> int:
    return load_library().fg_last_bad_arg()


def fg_last_error() -> str:
    return load_library().fg_last_error().decode()


def fg_status_string(s: int) -> str:
    return status_name(s)


def fg_abi_version() -> int:
    return load_library().fg_abi_version()


def fg_sgemm_streamk(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                     workspace, workspace_bytes, stream=0):
    """Raw call with the stream-K tail (device addresses as ints)."""
    return load_library().fg_sgemm_streamk(_op(transA), _op(transB), M, N, K, alpha, A, lda,
                                           B, ldb, beta, C, ldc, workspace or None,
                                           workspace_bytes, stream or None)


def fg_sgemm_streamk_workspace_size(transA, transB, M, N, K, A=0, lda=None, B=0,
                                    ldb=None) -> int:
    ta, tb = _op(transA), _op(transB)
    lda = lda if lda is not None else max(1, M if ta else K)
    ldb = ldb if ldb is not None else max(1, K if tb else N)
    return load_library().fg_sgemm_streamk_workspace_size(ta, tb, M, N, K, A or None, lda,
                                                          B or None, ldb)


def fg_sgemm_fused(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                   epilogue=None, stream=0, config=-1):
    """Raw call with a fused epilogue (an fg_epilogue, or None for none)."""
    ep = ctypes.byref(epilogue) if epilogue is not None else None
    return load_library().fg_sgemm_fused(_op(transA), _op(transB), M, N, K, alpha, A, lda,
                                         B, ldb, beta, C, ldc, ep, stream or None, config)


def fg_sgemm_quant(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                   epilogue=None, quant=None, stream=0, config=-1):
    """Raw call: the fused GEMM plus a quantised copy Q of C (an fg_quant, or
    None for none); see include/fp32gemm.h."""
    ep = ctypes.byref(epilogue) if epilogue is not None else None
    q = ctypes.byref(quant) if quant is not None else None
    return load_library().fg_sgemm_quant(_op(transA), _op(transB), M, N, K, alpha, A, lda,
                                         B, ldb, beta, C, ldc, ep, q, stream or None, config)


def fg_estimate_seconds(M, N, K, config_id, splits=1, beta_zero=True) -> float:
    """Cost-model estimate of one call with a given entry (fp32gemm_tune.h)."""
    return load_library().fg_estimate_seconds(M, N, K, config_id, splits, int(bool(beta_zero)))


def fg_get_efficiency(config_id):
    """(eff, eff1) of a matrix-core entry."""
    e, e1 = ctypes.c_double(), ctypes.c_double()
    _raise_if(load_library().fg_get_efficiency(config_id, ctypes.byref(e), ctypes.byref(e1)))
    return e.value, e1.value


def fg_set_efficiency(config_id, eff, eff1) -> int:
    return load_library().fg_set_efficiency(config_id, eff, eff1)


def fg_set_streamk_policy(policy) -> int:
    """0: split the stream-K tail when the model expects a gain; 1: always."""
    return load_library().fg_set_streamk_policy(policy)


def fg_set_raster(group_m, xcd_remap) -> int:
    """Raster order of the matrix-core kernels (fp32gemm_tune.h): band height
    in tile rows (0 = default) and the XCD renumbering (1 on, 0 off)."""
    return load_library().fg_set_raster(group_m, xcd_remap)


def fg_set_few_row_threads(threads) -> int:
    """Workgroup size of the few-row kernel, B stored K x N (fp32gemm_tune.h):
    0 = automatic, else 256, 512 or 1024."""
    return load_library().fg_set_few_row_threads(threads)


MODEL_CONSTANTS = ("launch", "store_bw", "store_exposed", "stream_bw", "split_bw", "few_fixed",
                   "few_mfma")   # fg_model_constant, in order


def fg_get_model_constant(which) -> float:
    """A constant of the cost model (index or name of MODEL_CONSTANTS)."""
    w = which if isinstance(which, int) else MODEL_CONSTANTS.index(which)
    v = ctypes.c_double()
    _raise_if(load_library().fg_get_model_constant(w, ctypes.byref(v)))
    return v.value


def fg_set_model_constant(which, value) -> int:
    w = which if isinstance(which, int) else MODEL_CONSTANTS.index(which)
    return load_library().fg_set_model_constant(w, value)


def fg_set_few_row_kernel(kernel):
    """Few-row kernel family: 0 automatic, 1 vector ALU, 2 matrix cores
    (include/fp32gemm_tune.h)."""
    return load_library().fg_set_few_row_kernel(kernel)


def fg_get_raster():
    """(group_m, xcd_remap) in use."""
    g, x = ctypes.c_int32(), ctypes.c_int32()
    _raise_if(load_library().fg_get_raster(ctypes.byref(g), ctypes.byref(x)))
    return g.value, x.value


def fg_probe_mfma(workgroups, iterations, out, stream=0) -> int:
    """MFMA-only loop (fp32gemm_probe.h); out: device pointer, workgroups*256 floats."""
    return load_library().fg_probe_mfma(workgroups, iterations, out or None, stream or None)


def fg_probe_mfma_flops(workgroups, iterations) -> float:
    return load_library().fg_probe_mfma_flops(workgroups, iterations)


def fg_probe_lds_dma(src, bytes_per_lane, out, stream=0) -> int:
    """One direct-to-LDS load with lanes reversed, LDS copied to out
    (fp32gemm_probe.h); src and out: 64 * bytes_per_lane / 4 floats."""
    return load_library().fg_probe_lds_dma(src or None, bytes_per_lane, out or None,
                                           stream or None)


def fg_probe_read(x, n, workgroups, out, stream=0) -> int:
    """Streaming read of n floats (fp32gemm_probe.h); out: workgroups*4 floats."""
    return load_library().fg_probe_read(x or None, n, workgroups, out or None, stream or None)


def fg_quantize_fp8(type, block, M, N, X, ldx, Q=0, ldq=0, S=0, lds=0, QT=0, ldqt=0, ST=0,
                    ldst=0, stream=0):
    """Raw call (device addresses as ints); see include/fp32gemm_fp8.h."""
    return load_library().fg_quantize_fp8(type, block, M, N, X or None, ldx, Q or None, ldq,
                                          S or None, lds, QT or None, ldqt, ST or None, ldst,
                                          stream or None)


def fg_gemm_fp8(M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, block_b, beta, C, ldc,
                type_c, workspace=0, workspace_bytes=0, stream=0):
    """Raw call (device addresses as ints); see include/fp32gemm_fp8.h."""
    return load_library().fg_gemm_fp8(M, N, K, alpha, A or None, lda, SA or None, ldsa,
                                      B or None, ldb, SB or None, ldsb, block_b, beta, C or None,
                                      ldc, type_c, workspace or None, workspace_bytes,
                                      stream or None)


def fg_gemm_fp8_workspace_size(M, N, K) -> int:
    return load_library().fg_gemm_fp8_workspace_size(M, N, K)


def fg_fp8_tiles() -> list:
    """(rows of A, rows of B) of every tile of fg_gemm_fp8 (include/fp32gemm_tune.h)."""
    lib, out = load_library(), []
    for t in range(lib.fg_fp8_num_tiles()):
        a, b = ctypes.c_int32(), ctypes.c_int32()
        _raise_if(lib.fg_fp8_tile(t, ctypes.byref(a), ctypes.byref(b)))
        out.append((a.value, b.value))
    return out


def fg_select_fp8(M, N, K, workspace_bytes=0):
    """(tile, slices of K) that fg_gemm_fp8 runs (include/fp32gemm_tune.h)."""
    t, s = ctypes.c_int32(), ctypes.c_int32()
    _raise_if(load_library().fg_select_fp8(M, N, K, workspace_bytes, ctypes.byref(t),
                                           ctypes.byref(s)))
    return t.value, s.value


def fg_set_fp8_tile(tile) -> int:
    """Tile of every later fg_gemm_fp8; -1: the library's choice."""
    return load_library().fg_set_fp8_tile(tile)


def fg_moe(layer, workspace, workspace_bytes, stream=0):
    """Raw call with an fg_moe_layer; see include/fp32gemm_moe.h."""
    ref = ctypes.byref(layer) if layer is not None else None
    return load_library().fg_moe(ref, workspace or None, workspace_bytes, stream or None)


def fg_moe_workspace_size(tokens, top_k, experts, hidden, inner) -> int:
    return load_library().fg_moe_workspace_size(tokens, top_k, experts, hidden, inner)


def configs() -> list:
    return [fg_get_config(i) for i in range(fg_num_configs())]


# ---- torch convenience ----------------------------------------------------

def _ld(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    return t.stride(0) if t.size(0) > 1 else max(1, t.size(1))


def sgemm(A, B, C, alpha=1.0, beta=0.0, transA="N", transB="N", config=-1, stream=None,
          row_scale=None, col_scale=None, row_bias=None, col_bias=None, activation="none"):
    """C <- alpha * op(A) @ op(B) + beta * C for float32 GPU tensors (row-major,
    unit inner stride; leading dimensions are taken from the row strides).
    With any of row_scale / col_scale / row_bias / col_bias (contiguous float32
    GPU vectors of length M or N) or an activation ("relu", "gelu", "silu"),
    C <- act(alpha * r_i * c_j * (op(A) op(B))_ij + beta * C_ij + u_i + w_j)
    through fg_sgemm_fused. Returns C. Enqueued on ``stream`` (default:
    torch's current stream)."""
    import torch
    for name, t in (("A", A), ("B", B), ("C", C)):
        if t.dtype != torch.float32:
            raise TypeError(f"{name} must be float32")
        if not t.is_cuda:
            raise ValueError(f"{name} must be on the GPU")
    ta, tb = _op(transA), _op(transB)
    M, N = C.shape
    K = A.shape[1] if ta == FG_OP_N else A.shape[0]
    if (A.shape[0] if ta == FG_OP_N else A.shape[1]) != M:
        raise ValueError("op(A) rows != C rows")
    if (B.shape[0] if tb == FG_OP_N else B.shape[1]) != K:
        raise ValueError("op(B) rows != op(A) columns")
    if (B.shape[1] if tb == FG_OP_N else B.shape[0]) != N:
        raise ValueError("op(B) columns != C columns")
    vecs = []
    for name, v, n in (("row_scale", row_scale, M), ("col_scale", col_scale, N),
                       ("row_bias", row_bias, M), ("col_bias", col_bias, N)):
        if v is None:
            vecs.append(0)
            continue
        if v.dtype != torch.float32 or not v.is_cuda or not v.is_contiguous() or v.numel() != n:
            raise ValueError(f"{name} must be a contiguous float32 GPU vector of length {n}")
        vecs.append(v.data_ptr())
    if stream is None:
        stream = torch.cuda.current_stream(C.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if any(vecs) or activation_code(activation) != FG_ACT_NONE:
        st = fg_sgemm_fused(ta, tb, M, N, K, float(alpha), A.data_ptr(), _ld(A, "A"),
                            B.data_ptr(), _ld(B, "B"), float(beta), C.data_ptr(), _ld(C, "C"),
                            make_epilogue(*vecs, activation), stream, config)
    else:
        st = fg_sgemm_ex(ta, tb, M, N, K, float(alpha), A.data_ptr(), _ld(A, "A"),
                         B.data_ptr(), _ld(B, "B"), float(beta), C.data_ptr(), _ld(C, "C"),
                         stream, config)
    _raise_if(st)
    return C


# ---- 8-bit matrices and mixture of experts: torch convenience --------------
# (Short calls on purpose: a decode step's kernels take a few microseconds, and
# so does the marshalling.)

_codes_of = {}   # torch dtype -> fg_type, filled on first use
_torch = None


def _torch_types():
    global _torch
    if _torch is None:
        import torch
        _codes_of.update({torch.float32: FG_TYPE_F32, torch.bfloat16: FG_TYPE_BF16,
                          torch.float8_e4m3fn: FG_TYPE_E4M3, torch.uint8: FG_TYPE_E4M3})
        _torch = torch
    return _torch, _codes_of


def _wrong(name, what):
    raise ValueError(f"{name} must {what}")


def _value_type(types, t, name):
    ty = types.get(t.dtype)
    if ty != FG_TYPE_F32 and ty != FG_TYPE_BF16:
        raise TypeError(f"{name} must be float32 or bfloat16")
    return ty


def _gpu(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on the GPU")
    return dev


def _run_on(torch, dev, stream, fn, args):
    """fn(*args, hipStream_t) with device `dev` current; stream: a torch stream,
    a raw handle or None (torch's current stream of that device)."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, stream or None)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream or None)
    if st != FG_OK:
        _raise_if(st)


def _codes(types, t, name, dev, rows, cols):
    """Leading dimension of a rows x cols tensor of codes."""
    if types.get(t.dtype) != FG_TYPE_E4M3:
        raise TypeError(f"{name} must be float8_e4m3fn (or uint8 codes)")
    if t.shape != (rows, cols) or t.get_device() != dev:
        _wrong(name, f"be {rows} x {cols} on device {dev}, is {tuple(t.shape)} on {t.device}")
    ld, inner = t.stride()
    if cols > 1 and inner != 1:
        _wrong(name, "have unit stride along its rows")
    # (one row: its stride is free, and codes need a multiple of 16)
    return ld if rows > 1 else (max(1, cols) + 15) // 16 * 16


def _scales(torch, t, name, dev, blocks, outer):
    """Leading dimension of a [column blocks, rows or row blocks] tensor."""
    if t is None or t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    if t.shape != (blocks, outer) or t.get_device() != dev:
        _wrong(name, f"be {blocks} x {outer} on device {dev}, is {tuple(t.shape)} on {t.device}")
    ld, inner = t.stride()
    if outer > 1 and inner != 1:
        _wrong(name, "have unit stride along its rows")
    return ld if blocks > 1 else max(outer, 1)   # (the library refuses one below `outer`)


def _workspace(t, dev):
    if t is None:
        return None, 0
    if not t.is_contiguous() or t.get_device() != dev:
        _wrong("workspace", f"be contiguous on device {dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def empty_fp8(rows, cols, block="row", device="cuda"):
    """(codes, scales) for a rows x cols matrix: uninitialised float8_e4m3fn
    codes whose rows start at multiples of 16 bytes, and float32 scales
    [ceil(cols / 128), rows] ("row") or [ceil(cols / 128), ceil(rows / 128)]
    ("tile")."""
    import torch
    wide = (max(1, cols) + 15) // 16 * 16
    q = torch.empty(rows, wide, dtype=torch.float8_e4m3fn, device=device)[:, :cols]
    outer = rows if _BLOCKS[block] == FG_BLOCK_ROW else (rows + 127) // 128
    return q, torch.empty((cols + 127) // 128, outer, dtype=torch.float32, device=device)


def quantize_fp8(X, Q=None, S=None, QT=None, ST=None, block="row", stream=None):
    """X (2-D, float32 or bfloat16, unit inner stride) to e4m3 codes with a
    float32 scale for each block of 128 columns of a row ("row") or each
    128 x 128 block ("tile"): X's own order into Q and S, its transpose into QT
    and ST (either pair may be None; empty_fp8 makes them). X is read once.
    Enqueued on ``stream`` (default: torch's current stream)."""
    torch, types = _torch_types()
    dev = _gpu(X, "X")
    kind, ldx = _BLOCKS[block], _ld(X, "X")
    M, N = X.shape
    q = s = qt = st = None
    ldq = lds = ldqt = ldst = 0
    if Q is not None:
        ldq = _codes(types, Q, "Q", dev, M, N)
        lds = _scales(torch, S, "S", dev, (N + 127) // 128, (M + 127) // 128 if kind else M)
        q, s = Q.data_ptr() or None, S.data_ptr() or None
    if QT is not None:
        ldqt = _codes(types, QT, "QT", dev, N, M)
        ldst = _scales(torch, ST, "ST", dev, (M + 127) // 128, (N + 127) // 128 if kind else N)
        qt, st = QT.data_ptr() or None, ST.data_ptr() or None
    if M == 0 or N == 0:
        return
    _run_on(torch, dev, stream, load_library().fg_quantize_fp8,
            (_value_type(types, X, "X"), kind, M, N, X.data_ptr(), ldx, q, ldq, s, lds, qt, ldqt,
             st, ldst))


def gemm_fp8(A, SA, B, SB, C, alpha=1.0, beta=0.0, workspace=None, stream=None):
    """C <- alpha * A @ B.T + beta * C for e4m3 codes A (M x K, scales SA
    [ceil(K / 128), M]) and B (N x K, scales SB [ceil(K / 128), N] or
    [ceil(K / 128), ceil(N / 128)]) into float32 or bfloat16 C. workspace: a
    contiguous GPU tensor that no call running at the same time uses
    (fg_gemm_fp8_workspace_size bytes are useful), or None. Returns C.
    Enqueued on ``stream`` (default: torch's current stream)."""
    torch, types = _torch_types()
    dev = _gpu(C, "C")
    M, N = C.shape
    K = A.shape[1]
    kb = (K + 127) // 128
    tile = SB.dim() == 2 and SB.shape[1] != N
    outer = (N + 127) // 128 if tile else N
    strides = A.stride() + SA.stride() + B.stride() + SB.stride() + C.stride()
    if (N > 1 < kb and M > 0 and len(strides) == 10 and strides[1::2] == (1, 1, 1, 1, 1)
            and A.shape == (M, K) and B.shape == (N, K) and SA.shape == (kb, M)
            and SB.shape == (kb, outer) and SA.dtype is SB.dtype is torch.float32
            and types.get(A.dtype) == FG_TYPE_E4M3 == types.get(B.dtype)
            and A.get_device() == B.get_device() == SA.get_device() == SB.get_device() == dev):
        lda, ldsa, ldb, ldsb, ldc = strides[::2]   # (nothing to look at one by one)
        if M == 1:                                 # (one row: its stride is free)
            lda, ldc = (K + 15) // 16 * 16, N
    else:
        lda, ldb = _codes(types, A, "A", dev, M, K), _codes(types, B, "B", dev, N, K)
        ldsa = _scales(torch, SA, "SA", dev, kb, M)
        ldsb = _scales(torch, SB, "SB", dev, kb, outer)
        ldc = _ld(C, "C")
    ws, ws_bytes = _workspace(workspace, dev) if workspace is not None else (None, 0)
    _run_on(torch, dev, stream, (_lib or load_library()).fg_gemm_fp8,
            (M, N, K, alpha, A.data_ptr() or None, lda, SA.data_ptr() or None, ldsa,
             B.data_ptr() or None, ldb, SB.data_ptr() or None, ldsb, 1 if tile else 0, beta,
             C.data_ptr() or None, ldc, _value_type(types, C, "C"), ws, ws_bytes))
    return C


# fg_moe_layer as one packed record (quicker than a ctypes constructor)
_MOE_RECORD = struct.Struct("@9iPq" + 3 * "PqqPqq" + "PqiPPPq")


def _experts(torch, types, w, s, name, dev, E, R, C):
    """fg_type and the values of fg_experts of an [E, R, C] tensor."""
    if w.shape != (E, R, C) or w.get_device() != dev:
        _wrong(name, f"be {E} x {R} x {C} on device {dev}, is {tuple(w.shape)} on {w.device}")
    ty = types.get(w.dtype)
    if ty is None:
        raise TypeError(f"{name} must be float32, bfloat16 or e4m3 codes")
    stride, ld, inner = w.stride()
    if C > 1 and inner != 1:
        _wrong(name, "have unit stride along its rows")
    if R == 1:
        per = 16 // w.element_size()
        ld = (C + per - 1) // per * per
    if E == 1:
        stride = 0
    if ty != FG_TYPE_E4M3:
        return ty, (w.data_ptr(), ld, stride, 0, 0, 0)
    if s is None or s.dtype != torch.float32:
        raise TypeError(f"{name} needs float32 scales")
    kb, rb = (C + 127) // 128, (R + 127) // 128
    if s.shape != (E, kb, rb) or s.get_device() != dev:
        _wrong(f"scales of {name}", f"be {E} x {kb} x {rb} on device {dev}")
    sstride, lds, inner = s.stride()
    if rb > 1 and inner != 1:
        _wrong(f"scales of {name}", "have unit inner stride")
    return ty, (w.data_ptr(), ld, stride, s.data_ptr(), lds if kb > 1 else rb,
                sstride if E > 1 else 0)


def moe(x, gate, up, down, ids, weights, out, router=None, renormalize=True, scales=None,
        activation="silu", workspace=None, stream=None):
    """out[t] <- sum_s weights[t, s] * down_e @ (act(gate_e @ x[t]) * (up_e @ x[t])),
    e = ids[t, s], for at most 64 tokens x [T, H] (float32 or bfloat16).
    gate and up [E, I, H], down [E, H, I]: float32, bfloat16, or e4m3 codes
    with scales = (gate's, up's, down's), each [E, ceil(columns / 128),
    ceil(rows / 128)]. ids (int32) and weights (float32) are contiguous
    [T, k]: with a router [E, H] they are written (the k largest logits,
    softmax over those or, without renormalize, over all), else read, and an id
    outside 0 .. E - 1 is an empty slot. workspace: a contiguous GPU tensor of
    at least fg_moe_workspace_size(T, k, E, H, I) bytes that no call running at
    the same time uses; None allocates one with torch. Returns out. Enqueued on
    ``stream`` (default: torch's current stream)."""
    torch, types = _torch_types()
    dev = _gpu(x, "x")
    T, H = x.shape
    E, I = gate.shape[0], gate.shape[1]
    sg, su, sd = scales if scales is not None else (None, None, None)
    wt, g = _experts(torch, types, gate, sg, "gate", dev, E, I, H)
    ut, u = _experts(torch, types, up, su, "up", dev, E, I, H)
    dt, d = _experts(torch, types, down, sd, "down", dev, E, H, I)
    if not wt == ut == dt:
        raise TypeError("gate, up and down must have one type")
    if out.shape != (T, H) or out.dtype != x.dtype or out.get_device() != dev:
        _wrong("out", "have x's shape, type and device")
    if ids.dim() != 2 or ids.shape[0] != T or ids.dtype != torch.int32 \
            or not ids.is_contiguous() or ids.get_device() != dev:
        _wrong("ids", "be a contiguous int32 tensor of T rows on x's device")
    k = ids.shape[1]
    if weights.shape != (T, k) or weights.dtype != torch.float32 \
            or not weights.is_contiguous() or weights.get_device() != dev:
        _wrong("weights", "be a contiguous float32 tensor of ids' shape on x's device")
    rt = rp = ldr = 0
    if router is not None:
        if router.shape != (E, H) or router.get_device() != dev:
            _wrong("router", f"be {E} x {H} on x's device")
        rt, rp, ldr = _value_type(types, router, "router"), router.data_ptr(), _ld(router, "router")
    if workspace is None:
        if stream is not None and not hasattr(stream, "cuda_stream"):
            raise ValueError("a raw stream handle needs a workspace")
        need = fg_moe_workspace_size(T, k, E, H, I)
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(dev)):
            workspace = torch.empty(max(16, need), dtype=torch.uint8, device=x.device)
    ws, ws_bytes = _workspace(workspace, dev)
    layer = fg_moe_layer.from_buffer_copy(_MOE_RECORD.pack(
        T, E, k, H, I, _value_type(types, x, "x"), wt, activation_code(activation),
        1 if renormalize else 0, x.data_ptr(), _ld(x, "x"), *g, *u, *d, rp, ldr, rt,
        ids.data_ptr(), weights.data_ptr(), out.data_ptr(), _ld(out, "out")))
    _run_on(torch, dev, stream, load_library().fg_moe, (layer, ws, ws_bytes))
    return out
