"""ctypes binding of libkroquant.so: argument marshalling only.

Every computation runs in the library (HIP kernels on the GPU, or the C++
host helpers).  Device functions take torch tensors that already live on the
GPU and enqueue on the given stream (default: torch's current stream); they
return without synchronising.  There is no fallback: if the library is not
built, importing this module raises.
"""
import collections
import ctypes
import os
import struct

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkroquant.so")

KQ_OK = 0
KQ_ERR_ARG = 1
KQ_ERR_SHAPE = 2
KQ_ERR_ALIGN = 3
KQ_ERR_SINGULAR = 4
KQ_ERR_HIP = 5
KQ_ERR_OVERLAP = 6

KQ_VARIANT_AUTO = 0
KQ_VARIANT_MFMA = 1
KQ_VARIANT_BUTTERFLY = 2

# every symbol the public header declares
EXPORTS = (
    "kq_quantize", "kq_quantize_ex", "kq_transform_f32", "sq_quantize", "mx_quantize_f32",
    "kq_factor_inverse", "kq_block_matrix", "kq_block_inverse", "kq_fold_weight",
    "kq_quantize_lu", "kq_transform_lu_f32", "fwht_quantize", "fwht_transform_f32", "kq_lu_factors", "mx_gemm",
    "kq_adaln_quantize", "adaln_modulate", "kq_quantize16", "kq_transform16_f32", "kq_status_string",
    "kq_build_info", "kq_last_hip_error", "kq_hip_error_name",
    # measurement and test interface
    "kq_quantize_tuned", "kq_transform_tuned", "mx_gemm_tuned", "kq_adaln_quantize_tuned", "kq_launch_shape",
    "kq_flat_launch_shape",
    "kq_measure_copy41",
    # for callers that cannot allocate
    "kq_adaln_quantize_noalloc",
    # few-row products and the 4-bit key/value cache
    "mx_gemv", "mx_cache_write", "mx_cache_read", "mx_cache_attention", "mx_cache_attention_workspace",
)
KQ_GEMV_MAX_ROWS = 64
KQ_NOALLOC_MAX_ROWS = 131072
KQ_COPY_FORMS = 10

# launch-shape overrides (kq_tuning in kroquant.h); 0 keeps the automatic choice
TUNING_FIELDS = ("mfma_tiles_per_wg", "mfma_groups", "mfma_strip", "mfma_order", "code_stores",
                 "stream_rows_per_wave", "gemm_kernel", "adaln_pass", "adaln_strip", "adaln_blocks_per_wave",
                 "shared_form", "flat_wgs", "flat_ring", "mfma_ring")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built: run `python -m mxfp4_act_quantizer_amd.build` "
                      "(or __graft_entry__.build()) first")

_lib = ctypes.CDLL(LIB_PATH)
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int


class Tuning(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in TUNING_FIELDS]


def _tuning(tuning):
    """A kq_tuning pointer from a dict of overrides (None: automatic)."""
    if not tuning:
        return None
    unknown = set(tuning) - set(TUNING_FIELDS)
    if unknown:
        raise ValueError(f"unknown tuning fields {sorted(unknown)}")
    return ctypes.byref(Tuning(**{k: int(v) for k, v in tuning.items()}))


# mx_cache and mx_batch of kroquant.h as the bytes that a call is given
_CACHE = struct.Struct("8q")  # kq, ks, vq, vs, pages, page_size, heads, dim
_BATCH = struct.Struct("6q")  # page_table, row_start, lengths, seqs, width, rows

_lib.kq_quantize.argtypes = [_P, _I64, _I64, _P, _I64, _P, _P, _P]
_lib.kq_quantize_ex.argtypes = [_P, _I64, _I64, _P, _I64, _P, _P, _INT, _P]
_lib.kq_transform_f32.argtypes = [_P, _I64, _I64, _P, _I64, _P, _P]
_lib.kq_quantize_tuned.argtypes = [_P, _I64, _I64, _P, _I64, _P, _P, _INT, _P, _P]
_lib.kq_transform_tuned.argtypes = [_P, _I64, _I64, _P, _I64, _P, _INT, _P, _P]
_lib.mx_gemm_tuned.argtypes = [_P, _P, _I64, _P, _P, _I64, _I64, _P, _INT, _P, _P]
_lib.kq_adaln_quantize_tuned.argtypes = [_P, _I64, _I64, _P, _P, _I64, ctypes.c_float, _P, _I64, _P, _P, _P, _P, _P]
_lib.kq_launch_shape.argtypes = [_I64, _I64, _INT, _P, _P]
_lib.kq_flat_launch_shape.argtypes = [_I64, _I64, _P, _P]
_lib.sq_quantize.argtypes = [_P, _I64, _I64, _P, _P, _P, _P]
_lib.mx_quantize_f32.argtypes = [_P, _I64, _I64, _P, _P, _P]
_lib.kq_quantize_lu.argtypes = [_P, _I64, _I64, _P, _I64, _P, _P, _P]
_lib.kq_transform_lu_f32.argtypes = [_P, _I64, _I64, _P, _I64, _P, _P]
_lib.fwht_quantize.argtypes = [_P, _I64, _I64, _P, _P, _P]
_lib.fwht_transform_f32.argtypes = [_P, _I64, _I64, _P, _P]
_lib.kq_lu_factors.argtypes = [_P, _I64, _P]
_lib.mx_gemm.argtypes = [_P, _P, _I64, _P, _P, _I64, _I64, _P, _INT, _P]
_lib.mx_gemv.argtypes = [_P, _I64, _P, _P, _I64, _I64, _P, _INT, _P]
_lib.mx_cache_write.argtypes = [_P, _I64, _P, _I64, _P, _I64, _P, _P, _P]
_lib.mx_cache_read.argtypes = [_P, _P, _P, _P, _P]
_lib.mx_cache_attention.argtypes = [_P, _I64, _I64, _P, _P, ctypes.c_float, _I64, _I64, _P, _I64, _P, _I64, _P]
_lib.mx_cache_attention_workspace.argtypes = [_I64, _P, _P, _I64, _I64, _P]
_lib.kq_quantize16.argtypes = [_P, _I64, _I64, _P, _I64, _P, _P, _P]
_lib.kq_transform16_f32.argtypes = [_P, _I64, _I64, _P, _I64, _P, _P]
_lib.kq_adaln_quantize.argtypes = [_P, _I64, _I64, _P, _P, _I64, ctypes.c_float, _P, _I64, _P, _P, _P, _P]
_lib.kq_adaln_quantize_noalloc.argtypes = [_P, _I64, _I64, _P, _P, _I64, ctypes.c_float, _P, _I64, _P, _P, _P]
_lib.adaln_modulate.argtypes = [_P, _I64, _I64, _P, _P, _I64, ctypes.c_float, _P, _P, _P]
_lib.kq_factor_inverse.argtypes = [_P, _I64, _P]
_lib.kq_block_matrix.argtypes = [_P, _I64, _P]
_lib.kq_block_inverse.argtypes = [_P, _I64, _P]
_lib.kq_fold_weight.argtypes = [_P, _I64, _I64, _P, _I64, _P]
_lib.kq_status_string.argtypes = [_INT]
_lib.kq_status_string.restype = ctypes.c_char_p
_lib.kq_build_info.argtypes = []
_lib.kq_build_info.restype = ctypes.c_char_p
_lib.kq_last_hip_error.argtypes = []
_lib.kq_hip_error_name.argtypes = [_INT]
_lib.kq_hip_error_name.restype = ctypes.c_char_p
_lib.kq_measure_copy41.argtypes = [_P, _I64, _P, _INT, _P]
for _name in EXPORTS:
    if _name not in ("kq_status_string", "kq_build_info", "kq_hip_error_name"):
        getattr(_lib, _name).restype = _INT


class KQError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = f"{where}: {kq_status_string(status)} (status {status})"
        if status == KQ_ERR_HIP:
            self.hip_error = _lib.kq_last_hip_error()
            msg += f": {_lib.kq_hip_error_name(self.hip_error).decode()} ({self.hip_error})"
        super().__init__(msg)


def kq_status_string(status):
    return _lib.kq_status_string(int(status)).decode()


def kq_build_info():
    return _lib.kq_build_info().decode()


def lib():
    """The loaded ctypes library (raw C entry points)."""
    return _lib


def _check(st, where):
    if st != KQ_OK:
        raise KQError(st, where)


# ---------------------------------------------------------------------------
# device entry points (torch tensors on the GPU)
# ---------------------------------------------------------------------------
def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_torch_module = None


def _stream_handle(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t, dtypes, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a torch tensor on the GPU")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _bf16_types():
    global _bf16_dtypes
    if _bf16_dtypes is None:
        torch = _torch()
        _bf16_dtypes = (torch.bfloat16, torch.int16, torch.uint16)
    return _bf16_dtypes


_bf16_dtypes = None


def _outputs(x, M, d, q, s):
    torch = _torch()
    if q is None:
        q = torch.empty((M, d // 2), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty((M, d // 32), dtype=torch.uint8, device=x.device)
    return q, s


def _md(x):
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, d]")
    return int(x.shape[0]), int(x.shape[1])


def _nT(factors):
    n = factors.numel()
    if n % 20:
        raise ValueError("factors must hold [nT, 5, 2, 2] float32 values")
    return n // 20


def kq_quantize(x, factors, q=None, s=None, stream=None, variant=KQ_VARIANT_AUTO, tuning=None):
    """KroQuant quantizer: returns (q [M, d/2] u8, s [M, d/32] u8).  `tuning`
    (a dict of kq_tuning fields) pins the launch shape, for measurements."""
    torch = _torch()
    M, d = _md(x)
    q, s = _outputs(x, M, d, q, s)
    args = (_dev(x, _bf16_types(), "x"), M, d, _dev(factors, (torch.float32,), "factors"), _nT(factors),
            _dev(q, (torch.uint8,), "q"), _dev(s, (torch.uint8,), "s"))
    if tuning:
        st = _lib.kq_quantize_tuned(*args, int(variant), _tuning(tuning), _stream_handle(stream))
    elif variant == KQ_VARIANT_AUTO:
        st = _lib.kq_quantize(*args, _stream_handle(stream))
    else:
        st = _lib.kq_quantize_ex(*args, int(variant), _stream_handle(stream))
    _check(st, "kq_quantize")
    return q, s


def kq_quantize_ex(x, factors, q, s, variant, stream=None):
    return kq_quantize(x, factors, q, s, stream, variant)


def kq_transform_f32(x, factors, y=None, stream=None, variant=KQ_VARIANT_AUTO, tuning=None):
    """Transformed values y = x_blk . K_j (fp32) as the quantizer computes them."""
    torch = _torch()
    M, d = _md(x)
    if y is None:
        y = torch.empty((M, d), dtype=torch.float32, device=x.device)
    args = (_dev(x, _bf16_types(), "x"), M, d, _dev(factors, (torch.float32,), "factors"), _nT(factors),
            _dev(y, (torch.float32,), "y"))
    if tuning or variant != KQ_VARIANT_AUTO:
        st = _lib.kq_transform_tuned(*args, int(variant), _tuning(tuning), _stream_handle(stream))
    else:
        st = _lib.kq_transform_f32(*args, _stream_handle(stream))
    _check(st, "kq_transform_f32")
    return y


def kq_launch_shape(M, d, adaln=False, tuning=None):
    """Launch shape of the MFMA quantizer for [M, d] on the current device:
    dict of strip, tiles_per_wg, interleave, flat, grid, nt_codes, ring."""
    out = (ctypes.c_int64 * 7)()
    _check(_lib.kq_launch_shape(int(M), int(d), 1 if adaln else 0, _tuning(tuning), out), "kq_launch_shape")
    return dict(zip(("strip", "tiles_per_wg", "interleave", "flat", "grid", "nt_codes", "ring"),
                    (int(v) for v in out)))


def kq_flat_launch_shape(M, d, tuning=None):
    """Launch shape of the flat form (one shared factor set) for [M, d] on the
    current device: dict of ring, workgroups, nt_codes."""
    out = (ctypes.c_int64 * 3)()
    _check(_lib.kq_flat_launch_shape(int(M), int(d), _tuning(tuning), out), "kq_flat_launch_shape")
    return dict(zip(("ring", "workgroups", "nt_codes"), (int(v) for v in out)))


def _nT_lu(lu):
    n = lu.numel()
    if n % 15:
        raise ValueError("lu must hold [nT, 5, 3] float32 values")
    return n // 15


def kq_quantize_lu(x, lu, q=None, s=None, stream=None):
    """K2 form of the KroQuant quantizer: factor sets as LU scalars [nT, 5, 3]."""
    torch = _torch()
    M, d = _md(x)
    q, s = _outputs(x, M, d, q, s)
    st = _lib.kq_quantize_lu(_dev(x, _bf16_types(), "x"), M, d, _dev(lu, (torch.float32,), "lu"), _nT_lu(lu),
                             _dev(q, (torch.uint8,), "q"), _dev(s, (torch.uint8,), "s"), _stream_handle(stream))
    _check(st, "kq_quantize_lu")
    return q, s


def kq_transform_lu_f32(x, lu, y=None, stream=None):
    torch = _torch()
    M, d = _md(x)
    if y is None:
        y = torch.empty((M, d), dtype=torch.float32, device=x.device)
    st = _lib.kq_transform_lu_f32(_dev(x, _bf16_types(), "x"), M, d, _dev(lu, (torch.float32,), "lu"), _nT_lu(lu),
                                  _dev(y, (torch.float32,), "y"), _stream_handle(stream))
    _check(st, "kq_transform_lu_f32")
    return y


def fwht_quantize(x, q=None, s=None, stream=None):
    """Walsh-Hadamard-32 comparison quantizer (fixed transform, then MXFP4)."""
    torch = _torch()
    M, d = _md(x)
    q, s = _outputs(x, M, d, q, s)
    st = _lib.fwht_quantize(_dev(x, _bf16_types(), "x"), M, d, _dev(q, (torch.uint8,), "q"),
                            _dev(s, (torch.uint8,), "s"), _stream_handle(stream))
    _check(st, "fwht_quantize")
    return q, s


def fwht_transform_f32(x, y=None, stream=None):
    torch = _torch()
    M, d = _md(x)
    if y is None:
        y = torch.empty((M, d), dtype=torch.float32, device=x.device)
    st = _lib.fwht_transform_f32(_dev(x, _bf16_types(), "x"), M, d, _dev(y, (torch.float32,), "y"),
                                 _stream_handle(stream))
    _check(st, "fwht_transform_f32")
    return y


def mx_gemm(qa, sa, qb, sb, out=None, out_dtype=None, stream=None, tuning=None):
    """W4A4 product out = A . B^T of two MXFP4 matrices (codes [rows, K/2] u8,
    scales [rows, K/32] u8), accumulated in fp32; out float32 or bfloat16."""
    torch = _torch()
    M, K = int(qa.shape[0]), int(qa.shape[1]) * 2
    N = int(qb.shape[0])
    if int(qb.shape[1]) * 2 != K or sa.shape != (M, K // 32) or sb.shape != (N, K // 32):
        raise ValueError("operand shapes do not match")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or torch.float32, device=qa.device)
    bf = 1 if out.dtype == torch.bfloat16 else 0
    if out.dtype not in (torch.float32, torch.bfloat16) or tuple(out.shape) != (M, N):
        raise ValueError("out must be float32 or bfloat16 [M, N]")
    u8 = (torch.uint8,)
    args = (_dev(qa, u8, "qa"), _dev(sa, u8, "sa"), M, _dev(qb, u8, "qb"), _dev(sb, u8, "sb"), N, K,
            _dev(out, (torch.float32, torch.bfloat16), "out"), bf)
    if tuning:
        st = _lib.mx_gemm_tuned(*args, _tuning(tuning), _stream_handle(stream))
    else:
        st = _lib.mx_gemm(*args, _stream_handle(stream))
    _check(st, "mx_gemm")
    return out


def sq_quantize(x, scale, q=None, s=None, stream=None):
    """SmoothQuant comparison quantizer: y = x * fl32(1/scale_c), then MXFP4."""
    torch = _torch()
    M, d = _md(x)
    q, s = _outputs(x, M, d, q, s)
    st = _lib.sq_quantize(_dev(x, _bf16_types(), "x"), M, d, _dev(scale, (torch.float32,), "scale"),
                          _dev(q, (torch.uint8,), "q"), _dev(s, (torch.uint8,), "s"), _stream_handle(stream))
    _check(st, "sq_quantize")
    return q, s


def mx_quantize_f32(x, q=None, s=None, stream=None):
    """Plain MXFP4 quantization of an fp32 matrix."""
    torch = _torch()
    M, d = _md(x)
    q, s = _outputs(x, M, d, q, s)
    st = _lib.mx_quantize_f32(_dev(x, (torch.float32,), "x"), M, d, _dev(q, (torch.uint8,), "q"),
                              _dev(s, (torch.uint8,), "s"), _stream_handle(stream))
    _check(st, "mx_quantize_f32")
    return q, s


def _nT16(factors):
    n = factors.numel()
    if n % 16:
        raise ValueError("factors must hold [nT, 4, 2, 2] float32 values")
    return n // 16


def kq_quantize16(x, factors, q=None, s=None, stream=None):
    """16-element blocks with four factors per set [nT, 4, 2, 2]: returns
    (q [M, d/2] u8, s [M, d/16] u8)."""
    torch = _torch()
    M, d = _md(x)
    if q is None:
        q = torch.empty((M, d // 2), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty((M, d // 16), dtype=torch.uint8, device=x.device)
    st = _lib.kq_quantize16(_dev(x, _bf16_types(), "x"), M, d, _dev(factors, (torch.float32,), "factors"),
                            _nT16(factors), _dev(q, (torch.uint8,), "q"), _dev(s, (torch.uint8,), "s"),
                            _stream_handle(stream))
    _check(st, "kq_quantize16")
    return q, s


def kq_transform16_f32(x, factors, y=None, stream=None):
    """The transformed values of kq_quantize16 (fp32 [M, d])."""
    torch = _torch()
    M, d = _md(x)
    if y is None:
        y = torch.empty((M, d), dtype=torch.float32, device=x.device)
    st = _lib.kq_transform16_f32(_dev(x, _bf16_types(), "x"), M, d, _dev(factors, (torch.float32,), "factors"),
                                 _nT16(factors), _dev(y, (torch.float32,), "y"), _stream_handle(stream))
    _check(st, "kq_transform16_f32")
    return y


def _stats(h, M, stats):
    torch = _torch()
    if stats is None:
        stats = torch.empty((M, 2), dtype=torch.float64, device=h.device)
    return stats


def kq_adaln_quantize(h, shift, scale, tokens_per_sample, eps, factors, q=None, s=None, stats=None, stream=None,
                      tuning=None):
    """AdaLN front-end fused with the quantizer: x = LN(h) (1 + scale[b]) +
    shift[b] (b = row // tokens_per_sample) rounded to bf16, then the
    Kronecker transform and MXFP4.  `stats` is the [M, 2] float64 workspace
    (allocated here when not given).  Returns (q, s)."""
    torch = _torch()
    M, d = _md(h)
    q, s = _outputs(h, M, d, q, s)
    stats = _stats(h, M, stats)
    args = (_dev(h, _bf16_types(), "h"), M, d, _dev(shift, (torch.float32,), "shift"),
            _dev(scale, (torch.float32,), "scale"), int(tokens_per_sample), float(eps),
            _dev(factors, (torch.float32,), "factors"), _nT(factors), _dev(stats, (torch.float64,), "stats"),
            _dev(q, (torch.uint8,), "q"), _dev(s, (torch.uint8,), "s"))
    if tuning:
        st = _lib.kq_adaln_quantize_tuned(*args, _tuning(tuning), _stream_handle(stream))
    else:
        st = _lib.kq_adaln_quantize(*args, _stream_handle(stream))
    _check(st, "kq_adaln_quantize")
    return q, s


def kq_adaln_quantize_noalloc(h, shift, scale, tokens_per_sample, eps, factors, q, s, stream=None):
    """kq_adaln_quantize with the library's own fixed row-statistics array
    (at most KQ_NOALLOC_MAX_ROWS rows; calls overlapping in time on one GPU
    race on it): q and s are the caller's, nothing is allocated."""
    torch = _torch()
    M, d = _md(h)
    st = _lib.kq_adaln_quantize_noalloc(_dev(h, _bf16_types(), "h"), M, d, _dev(shift, (torch.float32,), "shift"),
                                        _dev(scale, (torch.float32,), "scale"), int(tokens_per_sample), float(eps),
                                        _dev(factors, (torch.float32,), "factors"), _nT(factors),
                                        _dev(q, (torch.uint8,), "q"), _dev(s, (torch.uint8,), "s"),
                                        _stream_handle(stream))
    _check(st, "kq_adaln_quantize_noalloc")
    return q, s


def adaln_modulate(h, shift, scale, tokens_per_sample, eps, x=None, stats=None, stream=None):
    """The AdaLN front-end alone: x (bf16 [M, d]) as kq_adaln_quantize computes it."""
    torch = _torch()
    M, d = _md(h)
    if x is None:
        x = torch.empty((M, d), dtype=torch.bfloat16, device=h.device)
    stats = _stats(h, M, stats)
    st = _lib.adaln_modulate(_dev(h, _bf16_types(), "h"), M, d, _dev(shift, (torch.float32,), "shift"),
                             _dev(scale, (torch.float32,), "scale"), int(tokens_per_sample), float(eps),
                             _dev(stats, (torch.float64,), "stats"), _dev(x, _bf16_types(), "x"),
                             _stream_handle(stream))
    _check(st, "adaln_modulate")
    return x


def measure_copy41(src, dst, form=0, stream=None):
    """Measurement only: a streaming copy with the quantizer's 4:1 footprint
    (reads all of src, writes src.nbytes / 4 bytes of dst), the benchmark's
    HBM ceiling; `form` picks one of the KQ_COPY_FORMS copy forms."""
    if not (src.is_cuda and dst.is_cuda and src.is_contiguous() and dst.is_contiguous()):
        raise ValueError("src and dst must be contiguous GPU tensors")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < nbytes // 4:
        raise ValueError("dst must hold src.nbytes / 4 bytes")
    _check(_lib.kq_measure_copy41(src.data_ptr(), nbytes, dst.data_ptr(), int(form), _stream_handle(stream)),
           "kq_measure_copy41")


# ---------------------------------------------------------------------------
# few-row products and the 4-bit key/value cache
# ---------------------------------------------------------------------------
MXCache = collections.namedtuple("MXCache", "kq ks vq vs")
MXCache.__doc__ = """The four uint8 buffers of a paged MXFP4 cache: codes kq, vq [pages, heads, page_size, dim/2] and
scales ks, vs [pages, heads, dim/32, page_size]."""


def mx_cache_new(pages, page_size, heads, dim, device="cuda"):
    """An MXCache of zeros (every position reads as 0)."""
    torch = _torch()
    if dim % 32:
        raise ValueError("dim must be a multiple of 32")
    q, s = (pages, heads, page_size, dim // 2), (pages, heads, dim // 32, page_size)
    return MXCache(*(torch.zeros(shape, dtype=torch.uint8, device=device) for shape in (q, s, q, s)))


# These calls are short enough on the GPU that the host side counts.  The usual
# call (the current stream, one visible GPU, tensors as documented) is checked
# and packed by the compiled module _serving; what it returns None for is done
# here: other streams and devices, bf16 given as bits, and every error that is
# found before the C ABI's own checks.
_usual = None
_raw_stream = None


def _serving():
    """The compiled module, or False where it has nothing to do."""
    global _usual, _raw_stream
    if _usual is None:
        torch = _torch()
        if not torch.cuda.is_available():
            return False
        _raw_stream = torch._C._cuda_getCurrentRawStream
        _usual = torch.cuda.device_count() == 1 and load_serving()
    return _usual


def load_serving():
    """_serving, bound to the library that is loaded (raises if it is not
    built, or not from the library's sources)."""
    _torch()
    from . import _serving as module
    if module.source_hash not in kq_build_info():
        raise ImportError("_serving.so and libkroquant.so are not built from the same sources; build again")
    module.bind(*(ctypes.cast(getattr(_lib, f), _P).value for f in (
        "mx_gemv", "mx_cache_write", "mx_cache_read", "mx_cache_attention", "mx_cache_attention_workspace")))
    return module


def _done(result, where):
    """The result of the compiled module, which returns a status for a call
    that was refused."""
    if type(result) is int:
        raise KQError(result, where)
    return result


def _gpu(t, dtype, name):
    """Address of a contiguous GPU tensor of the dtype."""
    if t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return _dev(t, (dtype,), name)


def _gpu_bf16(t, name):
    """Address of a contiguous GPU tensor of bf16 values (or their bits)."""
    if t.dtype in _bf16_types() and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return _dev(t, _bf16_types(), name)


_one_device = None


def _on_device(where, stream, tensors):
    """(the current device is the tensors' one, their device, stream handle)
    of tensors that have to share a device."""
    global _one_device
    torch = _torch_module
    if _one_device is None:
        _one_device = torch.cuda.device_count() == 1
    dev = 0
    if not _one_device:
        dev = tensors[0].get_device()
        for t in tensors:
            if t.get_device() != dev:
                raise ValueError(f"{where}: tensors lie on cuda:{dev} and {t.device}")
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"{where}: the stream belongs to {stream.device}, the tensors to cuda:{dev}")
    else:
        stream = stream.cuda_stream
    return _one_device or torch._C._cuda_getDevice() == dev, dev, stream


def _call(fn, where, stream, tensors, *args):
    """fn(*args, stream) with the tensors' device current."""
    here, dev, stream = _on_device(where, stream, tensors)
    if here:
        st = fn(*args, stream)
    else:
        with _torch_module.cuda.device(dev):
            st = fn(*args, stream)
    if st:
        raise KQError(st, where)


def _new(like, shape, dtype, stream):
    """An empty tensor on like's device that belongs to the call's stream: one
    of the current stream's could be given to that stream's next work, or still
    be in its earlier work's hands, while the call writes it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _torch_module.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _heads_view(t, name, heads, dim):
    """Address and row stride of a bf16 [rows, heads, dim] view whose rows are
    dense inside and any 16-byte multiple apart."""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a torch tensor on the GPU")
    if t.dtype not in _bf16_types():
        raise TypeError(f"{name} has dtype {t.dtype}, expected bfloat16")
    if t.dim() != 3 or t.shape[1:] != (heads, dim):
        raise ValueError(f"{name} must be [rows, {heads}, {dim}], is {list(t.shape)}")
    row, head, one = t.stride()
    if one != 1 or (heads > 1 and head != dim):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.data_ptr(), (row if t.shape[0] > 1 else heads * dim)


def _cache_arg(cache):
    """(mx_cache, heads, dim)"""
    u8 = _torch().uint8
    kq, ks, vq, vs = cache
    if kq.dim() != 4:
        raise ValueError("cache.kq must be [pages, heads, page_size, dim/2]")
    pages, heads, size, half = kq.shape
    if vq.shape != kq.shape or ks.shape != vs.shape or ks.shape != (pages, heads, half // 16, size):
        raise ValueError("the cache's buffers do not match: codes [pages, heads, page_size, dim/2], scales "
                         "[pages, heads, dim/32, page_size]")
    return _CACHE.pack(_gpu(kq, u8, "cache.kq"), _gpu(ks, u8, "cache.ks"), _gpu(vq, u8, "cache.vq"),
                       _gpu(vs, u8, "cache.vs"), pages, size, heads, half * 2), heads, half * 2


def _batch_arg(page_table, row_start, lengths, rows):
    """mx_batch"""
    i32 = _torch().int32
    seqs = lengths.numel()
    if page_table.dim() != 2 or page_table.shape[0] != seqs or row_start.numel() != seqs + 1:
        raise ValueError("a batch is page_table [seqs, width], row_start [seqs + 1], lengths [seqs]")
    return _BATCH.pack(_gpu(page_table, i32, "page_table"), _gpu(row_start, i32, "row_start"),
                       _gpu(lengths, i32, "lengths"), seqs, page_table.shape[1], rows)


def mx_gemv(x, qw, sw, out=None, out_dtype=None, stream=None):
    """out = x . W^T of at most KQ_GEMV_MAX_ROWS bf16 rows x [M, K] and an
    MXFP4 matrix W (codes [N, K/2], scales [N, K/32] u8), summed in fp32; out
    float32 (the default) or bfloat16 [M, N]."""
    torch = _torch()
    if stream is None and (fast := _serving()):
        dtype = out_dtype if out is None else out.dtype
        if (dtype is None or dtype is torch.bfloat16 or dtype is torch.float32) and (out is None or out_dtype is None):
            done = _done(fast.gemv(x, qw, sw, out, dtype is torch.bfloat16, _raw_stream(0)), "mx_gemv")
            if done is not None:
                return done
    M, K = _md(x)
    N = qw.shape[0]
    if qw.shape != (N, K // 2) or sw.shape != (N, K // 32):
        raise ValueError("operand shapes do not match")
    if out is None:
        dtype = out_dtype or torch.float32
        out = _new(x, (M, N), dtype, stream)
    else:
        dtype = out.dtype
        if out.shape != (M, N) or dtype is not (out_dtype or dtype):
            raise ValueError("out must be float32 or bfloat16 [M, N], as out_dtype says")
    bf16 = dtype is torch.bfloat16
    if not bf16 and dtype is not torch.float32:
        raise ValueError(f"out is {dtype}: float32 or bfloat16 is wanted")
    u8 = torch.uint8
    _call(_lib.mx_gemv, "mx_gemv", stream, (x, qw, sw, out), _gpu_bf16(x, "x"), M, _gpu(qw, u8, "qw"),
          _gpu(sw, u8, "sw"), N, K, _gpu(out, dtype, "out"), bf16)
    return out


def mx_cache_write(k, v, cache, page_table, row_start, lengths, factors=None, stream=None):
    """Quantizes the keys and values [rows, heads, dim] (bf16; row strides are
    free) of a step into their slots of the cache; `factors` [nT, 5, 2, 2]
    puts the keys through the Kronecker transform first.  Row r of sequence i
    is position lengths[i] - row_start[i + 1] + r."""
    if stream is None and (fast := _serving()):
        if _done(fast.write(k, v, cache, page_table, row_start, lengths, factors, _raw_stream(0)), "mx_cache_write"):
            return
    c, heads, dim = _cache_arg(cache)
    kp, kst = _heads_view(k, "k", heads, dim)
    vp, vst = _heads_view(v, "v", heads, dim)
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v must have the same rows")
    b = _batch_arg(page_table, row_start, lengths, k.shape[0])
    tensors = (k, v, *cache, page_table, row_start, lengths)
    fp, nT = None, 1
    if factors is not None:
        fp, nT = _gpu(factors, _torch().float32, "factors"), _nT(factors)
        tensors += (factors,)
    _call(_lib.mx_cache_write, "mx_cache_write", stream, tensors, kp, kst, vp, vst, fp, nT, c, b)


def mx_cache_read(cache, page_table, row_start, lengths, rows=None, k=None, v=None, stream=None):
    """Keys and values (bf16 [rows, heads, dim]) of a batch's rows, as the
    cache's codes stand for them.  `rows` sizes the outputs allocated here;
    rows of no sequence, or without a slot, are left as they were."""
    torch = _torch()
    if stream is None and k is None and v is None and (fast := _serving()):
        done = _done(fast.read(cache, page_table, row_start, lengths, rows, _raw_stream(0)), "mx_cache_read")
        if done is not None:
            return done
    c, heads, dim = _cache_arg(cache)
    if rows is None:
        if k is None:
            raise ValueError("give rows, or k and v")
        rows = k.shape[0]
    shape = (int(rows), heads, dim)
    if k is None:
        k = _new(cache.kq, shape, torch.bfloat16, stream)
    if v is None:
        v = _new(cache.kq, shape, torch.bfloat16, stream)
    if k.shape != shape or v.shape != shape:
        raise ValueError(f"k and v must be {list(shape)}")
    b = _batch_arg(page_table, row_start, lengths, shape[0])
    _call(_lib.mx_cache_read, "mx_cache_read", stream, (k, v, *cache, page_table, row_start, lengths),
          c, b, _gpu_bf16(k, "k"), _gpu_bf16(v, "v"))
    return k, v


def _attention_bytes(q_heads, c, b, window, sinks):
    need = _I64()
    st = _lib.mx_cache_attention_workspace(q_heads, c, b, window, sinks, ctypes.byref(need))
    if st:
        raise KQError(st, "mx_cache_attention")
    return need.value


def mx_cache_attention_workspace(rows, q_heads, cache, page_table, row_start, lengths, window=0, sinks=0):
    """Bytes of workspace that mx_cache_attention asks for (it depends on the
    sizes only, not on the lengths)."""
    with _torch().cuda.device(cache.kq.device):
        return _attention_bytes(int(q_heads), _cache_arg(cache)[0],
                                _batch_arg(page_table, row_start, lengths, int(rows)), int(window), int(sinks))


def mx_cache_attention(q, cache, page_table, row_start, lengths, softmax_scale=None, window=0, sinks=0, out=None,
                       workspace=None, stream=None):
    """Attention of the new rows q [rows, q_heads, dim] (bf16; the row stride
    is free) over the cache, which holds their keys and values already:
    causal, with window > 0 only the last `window` positions and the first
    `sinks`.  softmax_scale is 1 / sqrt(dim) by default.  Returns out (bf16,
    allocated here when not given; rows of no sequence are left as they were).
    `workspace` is a uint8 tensor of mx_cache_attention_workspace bytes
    (allocated here when not given)."""
    torch = _torch()
    if stream is None and workspace is None and (fast := _serving()):
        done = _done(fast.attention(q, cache, page_table, row_start, lengths, softmax_scale, window, sinks, out,
                                    _raw_stream(0)), "mx_cache_attention")
        if done is not None:
            return done
    if abs(window) >> 62 or abs(sinks) >> 62:
        raise ValueError("window and sinks are at most 2^30")  # ctypes would cut them to 64 bits
    c, _, dim = _cache_arg(cache)
    if q.dim() != 3:
        raise ValueError("q must be [rows, q_heads, dim]")
    rows, heads, _ = q.shape
    qp, qst = _heads_view(q, "q", heads, dim)
    if out is None:
        out = _new(q, (rows, heads, dim), torch.bfloat16, stream)
        op, ost = out.data_ptr(), heads * dim
    else:
        if out.shape[0] != rows:
            raise ValueError("out must have q's rows")
        op, ost = _heads_view(out, "out", heads, dim)
    b = _batch_arg(page_table, row_start, lengths, rows)
    tensors = (q, out, *cache, page_table, row_start, lengths)
    if workspace is None:
        # the size goes by the compute units of the current device: the tensors' one
        here, dev, _ = _on_device("mx_cache_attention", stream, tensors)
        if here:
            need = _attention_bytes(heads, c, b, window, sinks)
        else:
            with torch.cuda.device(dev):
                need = _attention_bytes(heads, c, b, window, sinks)
        wp = 0
        if need:
            workspace = _new(q, need, torch.uint8, stream)
    else:
        need = workspace.numel()
        tensors += (workspace,)
    if workspace is not None:
        wp = _gpu(workspace, torch.uint8, "workspace")
    _call(_lib.mx_cache_attention, "mx_cache_attention", stream, tensors, qp, qst, heads, c, b,
          dim ** -0.5 if softmax_scale is None else softmax_scale, window, sinks, op, ost, wp, need)
    return out


# ---------------------------------------------------------------------------
# host helpers (numpy arrays, synchronous)
# ---------------------------------------------------------------------------
def _host_f32(a, name):
    a = np.ascontiguousarray(a, dtype=np.float32)
    return a


def kq_lu_factors(lu):
    """2x2 factors [nT, 5, 2, 2] of LU scalars [nT, 5, 3], in the kernel's fp32 arithmetic."""
    f = _host_f32(lu, "lu")
    if f.size % 15:
        raise ValueError("lu must hold [nT, 5, 3] float32 values")
    nT = f.size // 15
    out = np.empty((nT, 5, 2, 2), np.float32)
    _check(_lib.kq_lu_factors(f.ctypes.data, nT, out.ctypes.data), "kq_lu_factors")
    return out


def kq_factor_inverse(factors):
    f = _host_f32(factors, "factors")
    nT = f.size // 20
    out = np.empty((nT, 5, 2, 2), np.float32)
    _check(_lib.kq_factor_inverse(f.ctypes.data, nT, out.ctypes.data), "kq_factor_inverse")
    return out


def kq_block_matrix(factors):
    f = _host_f32(factors, "factors")
    nT = f.size // 20
    out = np.empty((nT, 32, 32), np.float32)
    _check(_lib.kq_block_matrix(f.ctypes.data, nT, out.ctypes.data), "kq_block_matrix")
    return out


def kq_block_inverse(factors):
    f = _host_f32(factors, "factors")
    nT = f.size // 20
    out = np.empty((nT, 32, 32), np.float32)
    _check(_lib.kq_block_inverse(f.ctypes.data, nT, out.ctypes.data), "kq_block_inverse")
    return out


def kq_fold_weight(W, factors):
    """W_out = W . T^-T so that (X T) W_out^T = X W^T."""
    w = _host_f32(W, "W")
    f = _host_f32(factors, "factors")
    N, d = w.shape
    out = np.empty_like(w)
    _check(_lib.kq_fold_weight(w.ctypes.data, N, d, f.ctypes.data, f.size // 20, out.ctypes.data), "kq_fold_weight")
    return out
