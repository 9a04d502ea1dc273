"""Thin Python binding of libnvfp4.so (ctypes).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in include/nvfp4.h.  PyTorch supplies the
device memory (output tensors are allocated here with torch.empty) and the
current HIP stream.  The functions carry the C names.  If the library is not
built, or there is no GPU, they raise -- there is no CPU fallback.
"""
import collections
import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libnvfp4.so")

OUT_F32, OUT_BF16 = 0, 1
OUT_CLEAR_PADDING = 16
EPI_NONE, EPI_SILU_MUL = 0, 1
SEG_NONE, SEG_SIGMOID, SEG_GDN_DECAY = 0, 1, 2
MAX_SEGMENTS = 16
_SEG_NAMES = {"none": SEG_NONE, "sigmoid": SEG_SIGMOID, "gdn_decay": SEG_GDN_DECAY}
_EPI_NAMES = {"none": EPI_NONE, "silu_mul": EPI_SILU_MUL}

_lib = None

_c_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int

_SIGNATURES = {
    "nvfp4_quantize": (_int, [_c_p, _i64, _i64, _i64, _c_p, _int, _c_p, _c_p, _c_p]),
    "nvfp4_e2m1_encode": (_int, [_c_p, _i64, _c_p, _c_p]),
    "nvfp4_packed_weight_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "nvfp4_pack_weights": (_int, [_c_p, _i64, _i64, _int, _c_p, _c_p, _int, _c_p, ctypes.c_size_t, _c_p]),
    "nvfp4_unpack_weights_linear": (_int, [_c_p, _i64, _i64, _c_p, _c_p, _c_p]),
    "gemm_w4a4": (_int, [_c_p, _c_p, _c_p, _i64, _c_p, _c_p, _i64, _i64, _c_p, _int, _i64, _int, _c_p]),
    "nvfp4_linear": (_int, [_c_p, _i64, _i64, _i64, _c_p, _int, _c_p, _c_p, _c_p, _c_p, _i64, _c_p, _int, _i64,
                            _int, _c_p]),
    "gemm_w4a4_fused_segments": (_int, [_c_p, _c_p, _c_p, _i64, _c_p, _i64, _i64, _int, _c_p, _c_p, _c_p,
                                        _c_p, _c_p, _c_p, _int, _i64, _c_p]),
    "gemm_w4a4_silu_mul_quantize": (_int, [_c_p, _c_p, _c_p, _i64, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _c_p,
                                           _c_p, _c_p]),
    "nvfp4_silu_amax_parts": (_i64, [_i64, _i64]),
    "gemm_w4a4_silu_mul_amax": (_int, [_c_p, _c_p, _c_p, _i64, _c_p, _c_p, _i64, _i64, _c_p, _i64, _c_p, _i64,
                                       _c_p, _c_p]),
    "nvfp4_quantize_amax_parts": (_int, [_c_p, _i64, _i64, _i64, _c_p, _i64, _c_p, _c_p, _c_p, _c_p]),
    "gdn_recurrence": (_int, [_c_p, _i64, _c_p, _i64, _c_p, _i64, _c_p, _i64, _c_p, _i64, _i64, _int, _int, _int,
                              _c_p, _c_p, _c_p, _int, _i64, _c_p]),
    "nvfp4_weight_stream_read": (_int, [_c_p, _i64, _i64, _c_p, _c_p]),
    "paged_plan": (_int, [_c_p, _c_p, _i64, _int, _c_p, _i64, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _c_p, _c_p, _i64,
                          _c_p, _c_p]),
    "paged_kv_write": (_int, [_c_p, _i64, _c_p, _i64, _c_p, _i64, _c_p, _c_p, _int, _i64, _int, _int, _int, _i64, _i64,
                              _i64, _c_p, _c_p, _c_p]),
    "paged_attention_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _int, _int, _int, _i64, _i64]),
    "paged_attention": (_int, [_c_p, _i64, _i64, _c_p, _c_p, _i64, _i64, _i64, _int, _c_p, _c_p, _int, _i64, _int, _int,
                               _int, _i64, _i64, _i64, _c_p, _i64, _i64, ctypes.c_float, _i64, _c_p, _c_p, _c_p, _int,
                               _i64, _c_p, _c_p, ctypes.c_size_t, _c_p]),
    "verify_drafts_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64]),
    "verify_drafts": (_int, [_c_p, _int, _i64, _i64, _i64, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _i64, _c_p, _c_p, _c_p,
                             _i64, _c_p, _c_p, _c_p, _c_p, ctypes.c_size_t, _c_p]),
    "rotary_steps": (_int, [_int, ctypes.c_double, _int, ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                            _c_p, _c_p, _c_p]),
    "rotary": (_int, [_c_p, _i64, _i64, _int, _int, _c_p, _c_p, _int, _int, ctypes.c_double, _c_p, _i64, _c_p]),
    "paged_kv_append": (_int, [_c_p, _i64, _int, _c_p, _i64, _c_p, _i64, _c_p, _i64, _c_p, _c_p, _i64, _c_p, _int, _int,
                               ctypes.c_double, _c_p, _c_p, _int, _i64, _int, _int, _int, _i64, _i64, _i64, _c_p, _c_p, _c_p,
                               _c_p, _c_p]),
    "paged_attention_blocks": (_int, [_c_p, _i64, _i64, _c_p, _c_p, _i64, _i64, _i64, _int, _c_p, _c_p, _int, _i64, _int, _int,
                                      _int, _i64, _i64, _i64, _c_p, _c_p, _c_p, _i64, _i64, ctypes.c_float, _i64, _c_p, _int,
                                      _i64, _c_p, _c_p, ctypes.c_size_t, _c_p]),
    "int8_quantize": (_int, [_c_p, _i64, _i64, _i64, _c_p, _c_p, _c_p]),
    "gemm_w8a8_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64]),
    "gemm_w8a8": (_int, [_c_p, _c_p, _i64, _c_p, _c_p, _i64, _i64, _c_p, _int, _i64, _c_p, ctypes.c_size_t, _c_p]),
    "int8_linear": (_int, [_c_p, _i64, _i64, _i64, _c_p, _c_p, _c_p, _c_p, _i64, _c_p, _int, _i64, _c_p, ctypes.c_size_t, _c_p]),
    "nvfp4_status_string": (ctypes.c_char_p, [_int]),
    "nvfp4_last_hip_error": (_int, []),
}
EXPORTED = tuple(_SIGNATURES)


class NVFP4Error(RuntimeError):
    pass


def load(path=LIB_PATH):
    """Load the shared library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise NVFP4Error("libnvfp4.so not found at %s; build it with "
                         "`python -m nvfp4_w4a4_gemm_quantize_amd.build`" % path)
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(rc, what):
    if rc != 0:
        lib = load()
        msg = lib.nvfp4_status_string(rc).decode()
        if rc == -5:
            msg += " (hipError %d)" % lib.nvfp4_last_hip_error()
        raise NVFP4Error("%s failed: %s [%d]" % (what, msg, rc))


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev(t, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise NVFP4Error("%s must be a GPU tensor" % name)
    if t.dtype != dtype:
        raise NVFP4Error("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _i64_array(vals):
    arr = (ctypes.c_int64 * len(vals))(*[int(v) for v in vals])
    return arr


def nvfp4_quantize(x, global_scale=None, dynamic=True, codes=None, scales=None):
    """bf16 [rows, cols] (row stride allowed) -> (codes u8 [rows, cols/2], scales u8 [rows, cols/16], g).

    dynamic=True writes g = 2688/amax into ``global_scale`` (allocated if None);
    dynamic=False reads a calibrated g from it.
    """
    lib = load()
    _dev(x, torch.bfloat16, "x")
    if x.dim() != 2 or x.stride(1) != 1:
        raise NVFP4Error("x must be 2-D with unit column stride")
    rows, cols = x.shape
    if global_scale is None:
        if not dynamic:
            raise NVFP4Error("a static quantisation needs global_scale")
        global_scale = torch.empty(1, dtype=torch.float32, device=x.device)
    _dev(global_scale, torch.float32, "global_scale")
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
    _dev(codes, torch.uint8, "codes")
    _dev(scales, torch.uint8, "scales")
    if codes.numel() * 2 < rows * cols or scales.numel() * 16 < rows * cols or not codes.is_contiguous() \
            or not scales.is_contiguous():
        raise NVFP4Error("codes/scales must be contiguous [rows, cols/2] and [rows, cols/16]")
    ld = x.stride(0) if rows > 1 else cols          # a size-1 dimension's stride is arbitrary
    rc = lib.nvfp4_quantize(_ptr(x), rows, cols, ld, _ptr(global_scale), 1 if dynamic else 0,
                            _ptr(codes), _ptr(scales), _stream())
    _check(rc, "nvfp4_quantize")
    return codes, scales, global_scale


def nvfp4_e2m1_encode(q, codes=None):
    """fp32 [n] -> E2M1 codes u8 [n] (0..15), through the quantizer's device encoder."""
    lib = load()
    _dev(q, torch.float32, "q")
    if not q.is_contiguous():
        raise NVFP4Error("q must be contiguous")
    n = q.numel()
    if codes is None:
        codes = torch.empty(n, dtype=torch.uint8, device=q.device)
    _dev(codes, torch.uint8, "codes")
    if codes.numel() < n or not codes.is_contiguous():
        raise NVFP4Error("codes must be a contiguous uint8 buffer of at least n bytes")
    _check(lib.nvfp4_e2m1_encode(_ptr(q), n, _ptr(codes), _stream()), "nvfp4_e2m1_encode")
    return codes


def nvfp4_packed_weight_bytes(n, k):
    return int(load().nvfp4_packed_weight_bytes(int(n), int(k)))


def nvfp4_pack_weights(w, seg_offsets=None, seg_global=None, dynamic=True, packed=None):
    """bf16 [n, k] weight -> (opaque packed u8 buffer, per-segment global scales float32 [S])."""
    lib = load()
    _dev(w, torch.bfloat16, "w")
    if w.dim() != 2 or not w.is_contiguous():
        raise NVFP4Error("w must be a contiguous [n, k] tensor")
    n, k = w.shape
    offs = [0, n] if seg_offsets is None else [int(v) for v in seg_offsets]
    nseg = len(offs) - 1
    if seg_global is None:
        if not dynamic:
            raise NVFP4Error("a static pack needs seg_global")
        seg_global = torch.empty(max(nseg, 1), dtype=torch.float32, device=w.device)
    _dev(seg_global, torch.float32, "seg_global")
    nbytes = nvfp4_packed_weight_bytes(n, k)
    if packed is None:
        packed = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=w.device)
    _dev(packed, torch.uint8, "packed")
    rc = lib.nvfp4_pack_weights(_ptr(w), n, k, nseg, _i64_array(offs), _ptr(seg_global), 1 if dynamic else 0,
                                _ptr(packed), packed.numel(), _stream())
    _check(rc, "nvfp4_pack_weights")
    return packed, seg_global


def nvfp4_unpack_weights_linear(packed, n, k):
    lib = load()
    _dev(packed, torch.uint8, "packed")
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=packed.device)
    scales = torch.empty((n, k // 16), dtype=torch.uint8, device=packed.device)
    rc = lib.nvfp4_unpack_weights_linear(_ptr(packed), n, k, _ptr(codes), _ptr(scales), _stream())
    _check(rc, "nvfp4_unpack_weights_linear")
    return codes, scales


def _out(out, m, cols, out_dtype, device):
    dt = torch.bfloat16 if out_dtype in (OUT_BF16, torch.bfloat16) else torch.float32
    if out is None:
        out = torch.empty((m, cols), dtype=dt, device=device)
    _dev(out, dt, "out")
    if out.dim() != 2 or out.stride(1) != 1 or out.shape[0] != m or out.shape[1] != cols:
        raise NVFP4Error("out must be [%d, %d] with unit column stride" % (m, cols))
    return out, (OUT_BF16 if dt == torch.bfloat16 else OUT_F32)


def _ld(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def gemm_w4a4(a_codes, a_scales, a_global, w_packed, w_global, n, k, out_dtype=torch.bfloat16,
              epilogue="none", out=None):
    """y = A_q W_q^T / (g_a g_w), [m, n] (or [m, n/2] with epilogue='silu_mul')."""
    lib = load()
    _dev(a_codes, torch.uint8, "a_codes")
    _dev(a_scales, torch.uint8, "a_scales")
    _dev(a_global, torch.float32, "a_global")
    _dev(w_packed, torch.uint8, "w_packed")
    _dev(w_global, torch.float32, "w_global")
    epi = _EPI_NAMES[epilogue] if isinstance(epilogue, str) else int(epilogue)
    m = a_codes.shape[0]
    if a_codes.numel() != m * (k // 2) or a_scales.numel() != m * (k // 16):
        raise NVFP4Error("a_codes/a_scales do not match [m, k] with k=%d" % k)
    if w_packed.numel() < nvfp4_packed_weight_bytes(n, k):
        raise NVFP4Error("w_packed is smaller than the packed size of [%d, %d]" % (n, k))
    out, od = _out(out, m, n // 2 if epi == EPI_SILU_MUL else n, out_dtype, a_codes.device)
    rc = lib.gemm_w4a4(_ptr(a_codes), _ptr(a_scales), _ptr(a_global), m, _ptr(w_packed), _ptr(w_global), n, k,
                       _ptr(out), od, _ld(out), epi, _stream())
    _check(rc, "gemm_w4a4")
    return out


def nvfp4_linear(x, w_packed, w_global, n, out_dtype=torch.bfloat16, epilogue="none", out=None,
                 a_global=None, dynamic=True, a_codes=None, a_scales=None):
    """The W4A4 layer on a bf16 activation x [m, k]: quantise x (as nvfp4_quantize) and multiply.
    Returns (out, a_codes, a_scales, a_global)."""
    lib = load()
    _dev(x, torch.bfloat16, "x")
    if x.dim() != 2 or x.stride(1) != 1:
        raise NVFP4Error("x must be 2-D with unit column stride")
    m, k = x.shape
    _dev(w_packed, torch.uint8, "w_packed")
    _dev(w_global, torch.float32, "w_global")
    if a_global is None:
        if not dynamic:
            raise NVFP4Error("a static quantisation needs a_global")
        a_global = torch.empty(1, dtype=torch.float32, device=x.device)
    _dev(a_global, torch.float32, "a_global")
    if a_codes is None:
        a_codes = torch.empty((m, k // 2), dtype=torch.uint8, device=x.device)
    if a_scales is None:
        a_scales = torch.empty((m, k // 16), dtype=torch.uint8, device=x.device)
    _dev(a_codes, torch.uint8, "a_codes")
    _dev(a_scales, torch.uint8, "a_scales")
    if a_codes.numel() != m * (k // 2) or a_scales.numel() != m * (k // 16) or not a_codes.is_contiguous() \
            or not a_scales.is_contiguous():
        raise NVFP4Error("a_codes/a_scales must be contiguous [m, k/2] and [m, k/16]")
    if w_packed.numel() < nvfp4_packed_weight_bytes(n, k):
        raise NVFP4Error("w_packed is smaller than the packed size of [%d, %d]" % (n, k))
    epi = _EPI_NAMES[epilogue] if isinstance(epilogue, str) else int(epilogue)
    out, od = _out(out, m, n // 2 if epi == EPI_SILU_MUL else n, out_dtype, x.device)
    ld_x = x.stride(0) if m > 1 else k
    rc = lib.nvfp4_linear(_ptr(x), m, k, ld_x, _ptr(a_global), 1 if dynamic else 0, _ptr(a_codes), _ptr(a_scales),
                          _ptr(w_packed), _ptr(w_global), n, _ptr(out), od, _ld(out), epi, _stream())
    _check(rc, "nvfp4_linear")
    return out, a_codes, a_scales, a_global


def gemm_w4a4_fused_segments(a_codes, a_scales, a_global, w_packed, n, k, seg_offsets, seg_w_global,
                             seg_epilogue=None, a_log=None, dt_bias=None, out_dtype=torch.bfloat16, out=None):
    """One GEMM over a fused weight; column segment s gets alpha_s = 1/(g_a g_w[s]) and its epilogue."""
    lib = load()
    _dev(a_codes, torch.uint8, "a_codes")
    _dev(a_scales, torch.uint8, "a_scales")
    _dev(a_global, torch.float32, "a_global")
    _dev(w_packed, torch.uint8, "w_packed")
    _dev(seg_w_global, torch.float32, "seg_w_global")
    offs = [int(v) for v in seg_offsets]
    nseg = len(offs) - 1
    epis = [SEG_NONE] * nseg if seg_epilogue is None else \
        [_SEG_NAMES[e] if isinstance(e, str) else int(e) for e in seg_epilogue]
    if len(epis) != nseg:
        raise NVFP4Error("one epilogue per segment")
    if a_log is not None:
        _dev(a_log, torch.float32, "a_log")
    if dt_bias is not None:
        _dev(dt_bias, torch.float32, "dt_bias")
    m = a_codes.shape[0]
    if a_codes.numel() != m * (k // 2) or a_scales.numel() != m * (k // 16):
        raise NVFP4Error("a_codes/a_scales do not match [m, k] with k=%d" % k)
    if w_packed.numel() < nvfp4_packed_weight_bytes(n, k):
        raise NVFP4Error("w_packed is smaller than the packed size of [%d, %d]" % (n, k))
    out, od = _out(out, m, n, out_dtype, a_codes.device)
    ep = (ctypes.c_int * max(nseg, 1))(*epis)
    rc = lib.gemm_w4a4_fused_segments(_ptr(a_codes), _ptr(a_scales), _ptr(a_global), m, _ptr(w_packed), n, k,
                                      nseg, _i64_array(offs), _ptr(seg_w_global), ep, _ptr(a_log), _ptr(dt_bias),
                                      _ptr(out), od, _ld(out), _stream())
    _check(rc, "gemm_w4a4_fused_segments")
    return out


def nvfp4_silu_amax_parts(m, n):
    """Entries of the partial-maxima buffer gemm_w4a4_silu_mul_amax needs for an m x n gate/up projection."""
    return int(load().nvfp4_silu_amax_parts(int(m), int(n)))


def gemm_w4a4_silu_mul_amax(a_codes, a_scales, a_global, w_packed, w_global, n, k, h=None, parts=None):
    """Gate/up GEMM into bf16 h [m, n/2] (silu(gate) * up) that also leaves partial maxima of |h|.
    Returns (h, parts, n_parts); parts (uint32, allocated if None, at least nvfp4_silu_amax_parts(m, n)
    entries) may be a view of the codes buffer h is quantised into next (nvfp4_quantize_amax_parts)."""
    lib = load()
    _dev(a_codes, torch.uint8, "a_codes")
    _dev(a_scales, torch.uint8, "a_scales")
    _dev(a_global, torch.float32, "a_global")
    _dev(w_packed, torch.uint8, "w_packed")
    _dev(w_global, torch.float32, "w_global")
    m = a_codes.shape[0]
    if a_codes.numel() != m * (k // 2) or a_scales.numel() != m * (k // 16):
        raise NVFP4Error("a_codes/a_scales do not match [m, k] with k=%d" % k)
    if w_packed.numel() < nvfp4_packed_weight_bytes(n, k):
        raise NVFP4Error("w_packed is smaller than the packed size of [%d, %d]" % (n, k))
    h, _ = _out(h, m, n // 2, torch.bfloat16, a_codes.device)
    need = nvfp4_silu_amax_parts(m, n)
    if parts is None:
        parts = torch.empty(max(need, 1), dtype=torch.int32, device=a_codes.device)
    if not isinstance(parts, torch.Tensor) or not parts.is_cuda or parts.dtype not in (torch.int32, torch.uint32) \
            or not parts.is_contiguous():
        raise NVFP4Error("parts must be a contiguous 32-bit GPU tensor")
    written = ctypes.c_int64(0)
    rc = lib.gemm_w4a4_silu_mul_amax(_ptr(a_codes), _ptr(a_scales), _ptr(a_global), m, _ptr(w_packed),
                                     _ptr(w_global), n, k, _ptr(h), _ld(h), _ptr(parts), parts.numel(),
                                     ctypes.byref(written), _stream())
    _check(rc, "gemm_w4a4_silu_mul_amax")
    return h, parts, int(written.value)


def nvfp4_quantize_amax_parts(x, parts, n_parts, global_scale=None, codes=None, scales=None):
    """nvfp4_quantize with a dynamic global scale whose amax is the largest of n_parts partial maxima
    (from gemm_w4a4_silu_mul_amax over x).  Returns (codes, scales, g)."""
    lib = load()
    _dev(x, torch.bfloat16, "x")
    if x.dim() != 2 or x.stride(1) != 1:
        raise NVFP4Error("x must be 2-D with unit column stride")
    rows, cols = x.shape
    if global_scale is None:
        global_scale = torch.empty(1, dtype=torch.float32, device=x.device)
    _dev(global_scale, torch.float32, "global_scale")
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
    _dev(codes, torch.uint8, "codes")
    _dev(scales, torch.uint8, "scales")
    if not isinstance(parts, torch.Tensor) or not parts.is_cuda or parts.numel() < n_parts:
        raise NVFP4Error("parts must be a GPU tensor of at least n_parts entries")
    ld = x.stride(0) if rows > 1 else cols
    rc = lib.nvfp4_quantize_amax_parts(_ptr(x), rows, cols, ld, _ptr(parts), int(n_parts), _ptr(global_scale),
                                       _ptr(codes), _ptr(scales), _stream())
    _check(rc, "nvfp4_quantize_amax_parts")
    return codes, scales, global_scale


def gemm_w4a4_silu_mul_quantize(a_codes, a_scales, a_global, w_packed, w_global, n, k, h_global,
                                h_codes=None, h_scales=None, return_h=False):
    """Gate/up GEMM with h = silu(gate)*up quantised to NVFP4 in the epilogue with the static scale h_global.

    Returns (h_codes u8 [m, n/4], h_scales u8 [m, n/32]) and, with return_h, also the bf16 h [m, n/2]
    that was quantised.
    """
    lib = load()
    _dev(a_codes, torch.uint8, "a_codes")
    _dev(a_scales, torch.uint8, "a_scales")
    _dev(a_global, torch.float32, "a_global")
    _dev(w_packed, torch.uint8, "w_packed")
    _dev(w_global, torch.float32, "w_global")
    _dev(h_global, torch.float32, "h_global")
    m = a_codes.shape[0]
    if a_codes.numel() != m * (k // 2) or a_scales.numel() != m * (k // 16):
        raise NVFP4Error("a_codes/a_scales do not match [m, k] with k=%d" % k)
    if w_packed.numel() < nvfp4_packed_weight_bytes(n, k):
        raise NVFP4Error("w_packed is smaller than the packed size of [%d, %d]" % (n, k))
    dev = a_codes.device
    if h_codes is None:
        h_codes = torch.empty((m, n // 4), dtype=torch.uint8, device=dev)
    if h_scales is None:
        h_scales = torch.empty((m, n // 32), dtype=torch.uint8, device=dev)
    _dev(h_codes, torch.uint8, "h_codes")
    _dev(h_scales, torch.uint8, "h_scales")
    if h_codes.numel() != m * (n // 4) or h_scales.numel() != m * (n // 32) or not h_codes.is_contiguous() \
            or not h_scales.is_contiguous():
        raise NVFP4Error("h_codes/h_scales must be contiguous [m, n/4] and [m, n/32]")
    h = torch.empty((m, n // 2), dtype=torch.bfloat16, device=dev) if return_h else None
    rc = lib.gemm_w4a4_silu_mul_quantize(_ptr(a_codes), _ptr(a_scales), _ptr(a_global), m, _ptr(w_packed),
                                         _ptr(w_global), n, k, _ptr(h_global), _ptr(h_codes), _ptr(h_scales),
                                         _ptr(h), _stream())
    _check(rc, "gemm_w4a4_silu_mul_quantize")
    return (h_codes, h_scales, h) if return_h else (h_codes, h_scales)


def nvfp4_weight_stream_read(w_packed, n, k, sink=None):
    """Read a packed weight exactly as the decode GEMM streams it, without arithmetic (roofline reference)."""
    lib = load()
    _dev(w_packed, torch.uint8, "w_packed")
    if w_packed.numel() < nvfp4_packed_weight_bytes(n, k):
        raise NVFP4Error("w_packed is smaller than the packed size of [%d, %d]" % (n, k))
    if sink is None:
        sink = torch.zeros(1, dtype=torch.int32, device=w_packed.device)
    _check(lib.nvfp4_weight_stream_read(_ptr(w_packed), n, k, _ptr(sink), _stream()), "nvfp4_weight_stream_read")
    return sink


def _ld2(t, name):
    """Row stride (elements) of a 2-D bf16 view with unit column stride."""
    _dev(t, torch.bfloat16, name)
    if t.dim() != 2 or t.stride(1) != 1:
        raise NVFP4Error("%s must be a 2-D view with unit column stride" % name)
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def gdn_recurrence(q, k, v, beta, g, hk, hv, s_init=None, return_state=False, out_dtype=torch.float32, out=None):
    """Gated delta rule over T steps.  q, k [T, hk*128], v [T, hv*128], beta, g [T, hv]: bf16 2-D views
    (they may be column slices of the fused in-projection output).  Returns o [T, hv*128] (and the final
    fp32 state [hv, 128, 128] with return_state)."""
    lib = load()
    T = q.shape[0]
    lds = [_ld2(x, n) for x, n in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta"), (g, "g"))]
    if any(x.shape[0] != T for x in (k, v, beta, g)):
        raise NVFP4Error("q, k, v, beta, g must have the same number of rows")
    if q.shape[1] != hk * 128 or k.shape[1] != hk * 128 or v.shape[1] != hv * 128 or beta.shape[1] != hv \
            or g.shape[1] != hv:
        raise NVFP4Error("shapes must be q, k [T, hk*128], v [T, hv*128], beta, g [T, hv]")
    if s_init is not None:
        _dev(s_init, torch.float32, "s_init")
        if s_init.shape != (hv, 128, 128) or not s_init.is_contiguous():
            raise NVFP4Error("s_init must be contiguous fp32 [hv, 128, 128]")
    s_final = torch.empty((hv, 128, 128), dtype=torch.float32, device=q.device) if return_state else None
    out, od = _out(out, T, hv * 128, out_dtype, q.device)
    rc = lib.gdn_recurrence(_ptr(q), lds[0], _ptr(k), lds[1], _ptr(v), lds[2], _ptr(beta), lds[3], _ptr(g), lds[4],
                            T, hk, hv, 128, _ptr(s_init), _ptr(s_final), _ptr(out), od, _ld(out), _stream())
    _check(rc, "gdn_recurrence")
    return (out, s_final) if return_state else out


# ------------------------------------------------- the paged serving step ----

CACHE_BF16, CACHE_E4M3 = 0, 1
LOGITS_F32, LOGITS_BF16 = 0, 1

PagedPlan = collections.namedtuple("PagedPlan", "q_start seq_lens positions slots counts")

# A step of the serving loop makes these calls for every layer, and its smallest ones take the GPU a few microseconds:
# the checks below read each tensor once, and addresses go to ctypes as plain integers.
_Tensor, _i32, _i64t, _f32, _bf16, _u8 = torch.Tensor, torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.uint8
_e4m3 = torch.float8_e4m3fn
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _refuse(t, dtype, name, shape):
    _dev(t, dtype, name)
    raise NVFP4Error("%s must be %s, got %s with strides %s" % (name, shape, tuple(t.shape), t.stride()))


def _vec(t, dtype, n, name):
    """The address of a contiguous GPU tensor of n elements."""
    if not isinstance(t, _Tensor) or not t.is_cuda or t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        _refuse(t, dtype, name, "contiguous with %d elements" % n)
    return t.data_ptr()


def _rows(t, dtype, rows, cols, name):
    """(address, row stride, columns) of a 2-D GPU view with unit column stride; rows and cols None: any."""
    if not isinstance(t, _Tensor) or not t.is_cuda or t.dtype is not dtype or t.dim() != 2:
        _refuse(t, dtype, name, "a 2-D view")
    r, c = t.shape
    ld, unit = t.stride()
    if (unit != 1 and c > 1) or (rows is not None and r != rows) or (cols is not None and c != cols):
        _refuse(t, dtype, name, "[%s, %s] with unit column stride" % (rows, cols))
    return t.data_ptr(), (ld if r > 1 else c), c    # a size-1 dimension's stride is arbitrary


def _cache(k_cache, v_cache, k_scale, v_scale):
    """The C arguments that describe a pair of [pages, heads, page size, head dim] views, and (heads, head dim)."""
    kind = k_cache.dtype if isinstance(k_cache, _Tensor) else None
    if kind is not _bf16 and kind is not _e4m3:
        raise NVFP4Error("k_cache must be a bfloat16 or float8_e4m3fn tensor")
    if not isinstance(v_cache, _Tensor) or not k_cache.is_cuda or not v_cache.is_cuda or v_cache.dtype is not kind:
        raise NVFP4Error("k_cache and v_cache must be GPU tensors of one type")
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or not k_cache.numel():
        raise NVFP4Error("k_cache and v_cache must be [pages, heads, page size, head dim] views of one shape")
    pages, heads, page_size, dim = k_cache.shape
    ps, hs, ts, unit = k_cache.stride()
    vp, vh, vt, vu = v_cache.stride()
    if unit != 1 or vu != 1 or ts != vt or (ps != vp and pages > 1) or (hs != vh and heads > 1):
        raise NVFP4Error("k_cache and v_cache need the same strides, the last of them 1")
    ks = None if k_scale is None else _vec(k_scale, _f32, heads, "k_scale")
    vs = None if v_scale is None else _vec(v_scale, _f32, heads, "v_scale")
    return (k_cache.data_ptr(), v_cache.data_ptr(), CACHE_BF16 if kind is _bf16 else CACHE_E4M3, pages, page_size, heads,
            dim, ps if pages > 1 else 0, hs if heads > 1 else 0, ts), ks, vs, heads, dim


def _plan_apart(ctx, new, free, cursor, outs):
    """Refuse inputs inside a plan's outputs ((address, bytes) each), but for the two that are carried in place."""
    low, high = min(o for o, _ in outs), max(o + n for o, n in outs)
    for x in (ctx, new, free, cursor):
        if x[0] >= high or x[0] + x[1] <= low or not x[1]:
            continue
        for out in outs:
            carried = (x is ctx and out is outs[1] and x == out) or (x is cursor and out is outs[4])
            if out[1] and x[0] < out[0] + out[1] and out[0] < x[0] + x[1] and not carried:
                raise NVFP4Error("ctx_lens, new_lens, free_pages or free_cursor shares memory with an output of the plan")


def paged_plan(ctx_lens, new_lens, free_pages, block_table, page_size, max_tokens, free_cursor=None, plan=None):
    """Block tables and slot maps of a step from the requests' lengths, on the device.

    ctx_lens, new_lens int32 [R]; free_pages int32 [F]; block_table int32 [R, max_pages] (written in place for the
    new pages); free_cursor int32 [1] or None.  Returns PagedPlan(q_start int32 [R + 1], seq_lens int32 [R],
    positions int32 [max_tokens], slots int64 [max_tokens], counts int32 [4]: new tokens, pages taken, pages missing,
    cursor after the step); ``plan`` reuses the tensors of an earlier one, whose seq_lens may be this step's ctx_lens and
    whose counts[3:] its free_cursor (no other input may share memory with an output).
    """
    lib = _lib or load()
    if not isinstance(ctx_lens, _Tensor) or not isinstance(free_pages, _Tensor):
        raise NVFP4Error("ctx_lens and free_pages must be GPU tensors")
    R, F = ctx_lens.numel(), free_pages.numel()
    ctx, new, free = _vec(ctx_lens, _i32, R, "ctx_lens"), _vec(new_lens, _i32, R, "new_lens"), _vec(free_pages, _i32, F, "free_pages")
    table, ld, cols = _rows(block_table, _i32, R, None, "block_table")
    cursor = None if free_cursor is None else _vec(free_cursor, _i32, 1, "free_cursor")
    if max_tokens < 0:
        raise NVFP4Error("max_tokens must not be negative")
    if plan is None:
        q_start, seq_lens, positions, counts = ctx_lens.new_empty(2 * R + 5 + max_tokens).split((R + 1, R, max_tokens, 4))
        plan = PagedPlan(q_start, seq_lens, positions, ctx_lens.new_empty(max_tokens, dtype=_i64t), counts)
        p0 = q_start.data_ptr()
        p1, p2, p3, p4 = p0 + 4 * (R + 1), p0 + 4 * (2 * R + 1), plan.slots.data_ptr(), p0 + 4 * (2 * R + 1 + max_tokens)
    else:
        p0, p1 = _vec(plan.q_start, _i32, R + 1, "q_start"), _vec(plan.seq_lens, _i32, R, "seq_lens")
        p2, p3 = _vec(plan.positions, _i32, max_tokens, "positions"), _vec(plan.slots, _i64t, max_tokens, "slots")
        p4 = _vec(plan.counts, _i32, 4, "counts")
        _plan_apart((ctx, 4 * R), (new, 4 * R), (free, 4 * F), (cursor or 0, 4 if cursor else 0),
                    ((p0, 4 * R + 4), (p1, 4 * R), (p2, 4 * max_tokens), (p3, 8 * max_tokens), (p4, 16)))
    rc = lib.paged_plan(ctx, new, R, page_size, free, F, cursor, table, cols, ld, p0, p1, p2, p3, max_tokens, p4,
                        _raw_stream(ctx_lens.get_device()))
    if rc:
        _check(rc, "paged_plan")
    return plan


def paged_kv_write(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None):
    """Write the rows of k, v (bf16 2-D views [T, heads * head_dim]) into the caches at slots (int64 [T]; -1: skip).

    k_cache, v_cache: [pages, heads, page size, head dim] views, bfloat16 or float8_e4m3fn (then x / scale[head],
    rounded to nearest even and clamped to +-448, is stored)."""
    lib = _lib or load()
    (kc, vc, kind, pages, page_size, heads, dim, ps, hs, ts), ks, vs, _, _ = _cache(k_cache, v_cache, k_scale, v_scale)
    kp, ld_k, _ = _rows(k, _bf16, None, heads * dim, "k")
    T = k.shape[0]
    vp, ld_v, _ = _rows(v, _bf16, T, heads * dim, "v")
    rc = lib.paged_kv_write(kp, ld_k, vp, ld_v, _vec(slots, _i64t, T, "slots"), T, kc, vc, kind, pages, page_size, heads, dim,
                            ps, hs, ts, ks, vs, _raw_stream(k.get_device()))
    if rc:
        _check(rc, "paged_kv_write")


def paged_attention_workspace(tokens, num_requests, num_heads, num_kv_heads, head_dim, max_new, max_seq, device="cuda"):
    """A workspace for paged_attention calls of these sizes (zero where the first call needs it)."""
    n = load().paged_attention_workspace_bytes(tokens, num_requests, num_heads, num_kv_heads, head_dim, max_new, max_seq)
    if n == 0:
        raise NVFP4Error("paged_attention does not take these sizes")
    workspace = torch.empty(n, dtype=_u8, device=device)
    workspace[:2048].zero_()
    return workspace


def paged_attention(q, k_cache, v_cache, block_table, q_start, seq_lens, max_new, max_seq, scale=None, window=0,
                    k_scale=None, v_scale=None, out_dtype=torch.bfloat16, out=None, lse=None, return_lse=False,
                    workspace=None, clear_padding=None):
    """Attention of every request's new tokens over its cached keys (causal, optionally a sliding window).

    q: bf16 [T, num_heads * head_dim] view, rows of request r from q_start[r] to q_start[r + 1]; caches as in
    paged_kv_write; block_table int32 [R, max_pages]; max_new and max_seq bound the requests' new tokens and lengths.
    Rows of q from q_start[R] on are padding: with clear_padding they get 0 (lse -inf), without they are left as they
    are (None: cleared where out is allocated here).
    Returns out [T, num_heads * head_dim] (and lse fp32 [T, num_heads] with return_lse)."""
    lib = _lib or load()
    cache, ks, vs, heads, dim = _cache(k_cache, v_cache, k_scale, v_scale)
    qp, ld_q, cols = _rows(q, _bf16, None, None, "q")
    T = q.shape[0]
    num_heads = cols // dim
    if cols == 0 or cols % dim or num_heads % heads:
        raise NVFP4Error("q must be [T, num_heads * %d] with num_heads a multiple of %d" % (dim, heads))
    if not isinstance(seq_lens, _Tensor):
        raise NVFP4Error("seq_lens must be a GPU tensor")
    R = seq_lens.numel()
    table, ld_t, max_pages = _rows(block_table, _i32, R, None, "block_table")
    if clear_padding is None:
        clear_padding = out is None
    if out is None:
        out = q.new_empty((T, cols), dtype=_bf16 if out_dtype in (OUT_BF16, _bf16) else _f32)
        op, ld_o = out.data_ptr(), cols
    else:
        op, ld_o, _ = _rows(out, _bf16 if out_dtype in (OUT_BF16, _bf16) else _f32, T, cols, "out")
    if lse is None and return_lse:
        lse = q.new_empty((T, num_heads), dtype=_f32)
    if workspace is None:
        workspace = paged_attention_workspace(T, R, num_heads, heads, dim, max_new, max_seq, q.device)
    bytes_ = workspace.numel()
    rc = lib.paged_attention(qp, ld_q, T, _vec(q_start, _i32, R + 1, "q_start"), _vec(seq_lens, _i32, R, "seq_lens"), R,
                             max_new, max_seq, num_heads, *cache, table, max_pages, ld_t,
                             dim ** -0.5 if scale is None else scale, window, ks, vs, op,
                             (OUT_BF16 if out.dtype is _bf16 else OUT_F32) + (OUT_CLEAR_PADDING if clear_padding else 0), ld_o,
                             None if lse is None else _vec(lse, _f32, T * num_heads, "lse"),
                             _vec(workspace, _u8, bytes_, "workspace"), bytes_, _raw_stream(q.get_device()))
    if rc:
        _check(rc, "paged_attention")
    return (out, lse) if return_lse else out


def verify_drafts_workspace(num_requests, max_drafts, vocab, device="cuda"):
    """A workspace for verify_drafts calls of these sizes (zero where the first call needs it)."""
    n = load().verify_drafts_workspace_bytes(num_requests, max_drafts, vocab)
    if n == 0:
        raise NVFP4Error("verify_drafts does not take these sizes")
    workspace = torch.empty(n, dtype=_u8, device=device)
    workspace[:1 << 18].zero_()
    return workspace


def verify_drafts(logits, row_start, num_drafts, draft_tokens, uniform, noise, draft_probs=None, temperature=None,
                  workspace=None):
    """Keep or refuse drafted tokens and draw the next one, from given random numbers.

    logits bf16 or fp32 [N, V] view: row row_start[r] + i is the target's after i kept drafts of request r;
    row_start, num_drafts int32 [R]; draft_tokens int32 [R, K]; uniform fp32 [R, K]; noise fp32 [R, V] (standard
    exponential); draft_probs fp32 [R, K, V] or None; temperature fp32 [R] or None (0: greedy).
    logits, noise and draft_probs begin 16-byte aligned: rows further on go by row_start, not by a slice of logits.
    Returns (tokens int32 [R, K + 1], accepted int32 [R], logprobs fp32 [R, K + 1])."""
    lib = _lib or load()
    kind = logits.dtype if isinstance(logits, _Tensor) else None
    if kind is not _bf16 and kind is not _f32:
        raise NVFP4Error("logits must be a bfloat16 or float32 tensor")
    lp, ld, V = _rows(logits, kind, None, None, "logits")
    if not isinstance(draft_tokens, _Tensor) or draft_tokens.dim() != 2:
        raise NVFP4Error("draft_tokens must be [requests, max drafts]")
    R, K = draft_tokens.shape
    np_, ld_noise, _ = _rows(noise, _f32, R, V, "noise")
    probs, ld_probs = None, V
    if draft_probs is not None:
        _dev(draft_probs, _f32, "draft_probs")
        sr, sk, sv = draft_probs.stride() if draft_probs.dim() == 3 else (0, 0, 0)
        if draft_probs.shape != (R, K, V) or (V > 1 and sv != 1) or (R > 1 and K > 1 and sr != K * sk):
            raise NVFP4Error("draft_probs must be [requests, max drafts, vocab] with evenly spaced rows")
        probs, ld_probs = draft_probs.data_ptr(), sk if K > 1 else sr if R > 1 else V
    if workspace is None:
        workspace = verify_drafts_workspace(R, K, V, logits.device)
    bytes_ = workspace.numel()
    tokens = draft_tokens.new_empty((R, K + 1))
    accepted = draft_tokens.new_empty(R)
    logprobs = noise.new_empty((R, K + 1))
    rc = lib.verify_drafts(lp, LOGITS_F32 if kind is _f32 else LOGITS_BF16, ld, logits.shape[0], V,
                           _vec(row_start, _i32, R, "row_start"), _vec(num_drafts, _i32, R, "num_drafts"), R, K,
                           _vec(draft_tokens, _i32, R * K, "draft_tokens"), probs, ld_probs,
                           None if temperature is None else _vec(temperature, _f32, R, "temperature"),
                           _vec(uniform, _f32, R * K, "uniform"), np_, ld_noise, tokens.data_ptr(), accepted.data_ptr(),
                           logprobs.data_ptr(), _vec(workspace, _u8, bytes_, "workspace"), bytes_,
                           _raw_stream(logits.get_device()))
    if rc:
        _check(rc, "verify_drafts")
    return tokens, accepted, logprobs


# ------------------------------------------- the attention layer in 8 bits ----

CACHE_E4M3_BLOCKS, CACHE_INT8_BLOCKS = 2, 3
ROTARY_HALF, ROTARY_INTERLEAVED = 0, 1
_LAYOUTS = {"half": ROTARY_HALF, "interleaved": ROTARY_INTERLEAVED}
_ROPE = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "wavelength": 4}
_e8m0, _int8 = torch.float8_e8m0fnu, torch.int8

RotaryTable = collections.namedtuple("RotaryTable", "steps rotary_dim layout amplitude")


def rotary_table(rotary_dim, base=10000.0, layout="half", scaling="none", factor=1.0, original_length=8192, slow_turns=1.0,
                 fast_turns=None, pair_factors=None, amplitude=None, device="cuda"):
    """A rotation of heads' first rotary_dim columns, for rotary and paged_kv_append; made once a model.

    layout: "half" turns columns (i, i + rotary_dim / 2), "interleaved" (2 i, 2 i + 1).  scaling for long contexts:
    "none", "linear", "ntk", "yarn" (pairs that make fewer than slow_turns turns over original_length are stretched by
    factor, those that make more than fast_turns, 32, are not; amplitude 0.1 ln factor + 1), "wavelength" (likewise by
    wavelength, fast_turns 4).  pair_factors (rotary_dim / 2 numbers) divide the frequencies one by one; amplitude
    replaces the scaling's."""
    if layout not in _LAYOUTS or scaling not in _ROPE:
        raise NVFP4Error("layout is one of %s, scaling one of %s" % (", ".join(_LAYOUTS), ", ".join(_ROPE)))
    n = max(int(rotary_dim), 0) // 2
    steps, amp = (ctypes.c_uint64 * max(n, 1))(), ctypes.c_double()
    factors = None
    if pair_factors is not None:
        factors = [float(x) for x in pair_factors]
        if len(factors) != n:
            raise NVFP4Error("pair_factors must hold %d numbers" % n)
        factors = (ctypes.c_double * max(n, 1))(*factors)
    if fast_turns is None:
        fast_turns = 32.0 if scaling == "yarn" else 4.0
    rc = load().rotary_steps(rotary_dim, base, _ROPE[scaling], factor, original_length, slow_turns, fast_turns, factors, steps,
                             ctypes.byref(amp))
    if rc:
        _check(rc, "rotary_steps")
    host = torch.tensor([x - (1 << 64) if x >> 63 else x for x in steps], dtype=_i64t)   # the 64 bits, as torch has them
    return RotaryTable(host.to(device), rotary_dim, layout, amp.value if amplitude is None else float(amplitude))


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _gpu_of(t):
    """The GPU of a call's first tensor; refused if it is not the current one, on whose default stream the call would run.
    The other tensors' devices are compared with it, which finds host tensors too (-1)."""
    device = t.get_device() if isinstance(t, _Tensor) else -1
    if device < 0:
        return -2       # no tensor's
    if device != _current_device():
        raise NVFP4Error("the tensors of a call must be on one GPU, the current one")
    return device


def _misplaced(t, dtype, name, shape):
    if isinstance(t, _Tensor) and t.is_cuda and t.get_device() != _current_device():
        raise NVFP4Error("the tensors of a call must be on one GPU, the current one")
    _refuse(t, dtype, name, shape)


def _rows_on(device, t, dtype, rows, cols, name):
    """_rows of a tensor on that GPU."""
    if not isinstance(t, _Tensor) or t.get_device() != device or t.dtype is not dtype or t.dim() != 2:
        _misplaced(t, dtype, name, "a 2-D view")
    r, c = t.shape
    ld, unit = t.stride()
    if (unit != 1 and c > 1) or (rows is not None and r != rows) or (cols is not None and c != cols):
        _refuse(t, dtype, name, "[%s, %s] with unit column stride" % (rows, cols))
    return t.data_ptr(), (ld if r > 1 else c), c    # a size-1 dimension's stride is arbitrary


def _vec_on(device, t, dtype, n, name):
    """_vec of a tensor on that GPU."""
    if not isinstance(t, _Tensor) or t.get_device() != device or t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        _misplaced(t, dtype, name, "contiguous with %d elements" % n)
    return t.data_ptr()


def _rotation(device, table, positions, tokens):
    """The C arguments (positions, steps, rotary dim, layout, amplitude)."""
    if not isinstance(table, RotaryTable) or table.layout not in _LAYOUTS:
        raise NVFP4Error("the rotation must come from rotary_table")
    steps, dim, layout, amplitude = table
    return (_vec_on(device, positions, _i32, tokens, "positions"), _vec_on(device, steps, _i64t, dim // 2, "steps"), dim,
            _LAYOUTS[layout], amplitude)


def rotary(x, positions, table, head_dim, out=None):
    """Rows of heads (bf16 view [T, heads * head_dim]) rotated to their positions (int32 [T]; negative: copied).

    table: from rotary_table.  out may be x (in place).  Returns out."""
    lib, device = _lib or load(), _gpu_of(x)
    xp, ld_x, cols = _rows_on(device, x, _bf16, None, None, "x")
    T = x.shape[0]
    if head_dim <= 0 or cols == 0 or cols % head_dim:
        raise NVFP4Error("x must be [T, heads * %d]" % head_dim)
    pos, steps, dim, layout, amplitude = _rotation(device, table, positions, T)
    if out is None:
        out = x.new_empty((T, cols))
        op, ld_o = out.data_ptr(), cols
    else:
        op, ld_o, _ = _rows_on(device, out, _bf16, T, cols, "out")
        _apart(x, out, same=True)
    rc = lib.rotary(xp, ld_x, T, cols // head_dim, head_dim, pos, steps, dim, layout, amplitude, op, ld_o, _raw_stream(device))
    if rc:
        _check(rc, "rotary")
    return out


def _apart(x, out, same=False):
    """Refuse an output that shares memory with an input (same: but for the input's own rows)."""
    a, b = x.data_ptr(), out.data_ptr()
    T, cols = x.shape
    if not T or (same and a == b):
        return
    ex, eo = x.element_size(), out.element_size()
    lx, lo, wide, cols = x.stride(0) * ex, out.stride(0) * eo, out.shape[1] * eo, cols * ex
    if a < b + (T - 1) * lo + wide and b < a + (T - 1) * lx + cols:
        # column slices of one matrix interleave without sharing an element
        at = (a - b) % lo if lx == lo and lo > 0 else 0
        if at < wide or at + cols > lo:
            raise NVFP4Error("an output overlaps an input")


def _apart_from(t, others):
    """Refuse a 2-D view of which a row shares memory with one of others ((address, bytes) each)."""
    rows, cols = t.shape
    if not rows:
        return
    p, size = t.data_ptr(), t.element_size()
    ld, cols = t.stride(0) * size, cols * size
    end = p + (rows - 1) * ld + cols
    for q, n in others:
        if n and q < end and p < q + n:
            at = (q - p) % ld if rows > 1 and q > p and ld >= cols else 0     # of the row that q lies in or behind
            if at < cols or at + n > ld:
                raise NVFP4Error("a tensor that the call writes overlaps another one")


def _meet(*ranges):
    """Whether any of (address, end) ranges meet: what most calls have to look at."""
    end = 0
    for p, e in sorted(ranges):
        if p < end:
            return True
        end = e
    return False


def _apart_all(written, read):
    """Refuse written ranges ((address, bytes) each) that meet each other or one that is read."""
    for i, (p, n) in enumerate(written):
        for q, o in written[i + 1:] + read:
            if n and o and p < q + o and q < p + n:
                raise NVFP4Error("a tensor that the call writes overlaps another one")


def _block_cache(device, k_cache, v_cache, k_scales, v_scales):
    """_cache for block-scaled caches: the C arguments, the scales' addresses and (heads, head dim)."""
    if not isinstance(k_cache, _Tensor) or k_cache.dtype is not _e4m3 and k_cache.dtype is not _int8:
        raise NVFP4Error("a block-scaled k_cache must be a float8_e4m3fn or int8 tensor")
    kind = k_cache.dtype
    if not isinstance(v_cache, _Tensor) or v_cache.dtype is not kind:
        raise NVFP4Error("k_cache and v_cache must be GPU tensors of one type")
    shape = k_cache.shape
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.get_device() != device or t.dim() != 4 or t.shape != shape:
            _misplaced(t, kind, name, "[pages, heads, page size, head dim], as the other cache")
    pages, heads, page_size, dim = shape
    ps, hs, ts, unit = k_cache.stride()
    vp, vh, vt, vu = v_cache.stride()
    if not pages * heads * page_size * dim or unit != 1 or vu != 1 or ts != vt or (ps != vp and pages > 1) \
            or (hs != vh and heads > 1):
        raise NVFP4Error("k_cache and v_cache need elements and the same strides, the last of them 1")
    scales = (pages, heads, page_size // 16)
    for name, t in (("k_scale", k_scales), ("v_scale", v_scales)):
        if not isinstance(t, _Tensor) or t.get_device() != device or t.dtype is not _e8m0 or t.shape != scales \
                or not t.is_contiguous():
            _misplaced(t, _e8m0, name, "[%d, %d, %d] contiguous" % scales)
    return ((k_cache.data_ptr(), v_cache.data_ptr(), CACHE_E4M3_BLOCKS if kind is _e4m3 else CACHE_INT8_BLOCKS, pages, page_size,
             heads, dim, ps if pages > 1 else 0, hs if heads > 1 else 0, ts), k_scales.data_ptr(), v_scales.data_ptr(), heads, dim)


def paged_kv_append(k, v, positions, slots, k_cache, v_cache, rotation=None, k_scale=None, v_scale=None, q=None, q_out=None):
    """Rotate the rows of k (bf16 2-D views [T, heads * head_dim]) and write them and those of v into the caches at slots.

    positions int32 [T], slots int64 [T] as from paged_plan (slots -1: skip); rotation: from rotary_table (None: none).
    Caches as in paged_kv_write, with its float scales a head, or block-scaled: float8_e4m3fn or int8 caches with k_scale,
    v_scale float8_e8m0fnu [pages, heads, page size / 16], which follow the values (a block's first token begins it anew;
    a block's rows of one call are neighbours, as paged_plan lays them).  q (bf16 view [T, num_heads * head_dim]) is
    rotated into q_out (allocated if None; may be q).  Returns q_out, or None without q."""
    lib, device = _lib or load(), _gpu_of(k)
    if isinstance(k_scale, _Tensor) and k_scale.dtype is _e8m0 or isinstance(k_cache, _Tensor) and k_cache.dtype is _int8:
        cache, kb, vb, heads, dim = _block_cache(device, k_cache, v_cache, k_scale, v_scale)
        ks = vs = None
    else:
        cache, ks, vs, heads, dim = _cache(k_cache, v_cache, k_scale, v_scale)
        kb = vb = None
        for t in (k_cache, v_cache, k_scale, v_scale):
            if t is not None and t.get_device() != device:
                _misplaced(t, t.dtype, "a cache", "on the current GPU")
    kp, ld_k, _ = _rows_on(device, k, _bf16, None, heads * dim, "k")
    T = k.shape[0]
    vp, ld_v, _ = _rows_on(device, v, _bf16, T, heads * dim, "v")
    pos, steps, rdim, layout, amplitude = (None, None, 0, ROTARY_HALF, 1.0) if rotation is None else \
        _rotation(device, rotation, positions, T)
    qp = op = None
    ld_q = ld_o = num_heads = 0
    if q is not None:
        qp, ld_q, cols = _rows_on(device, q, _bf16, T, None, "q")
        if cols == 0 or cols % dim:
            raise NVFP4Error("q must be [T, num_heads * %d]" % dim)
        num_heads = cols // dim
        if q_out is None:
            q_out = q.new_empty((T, cols))
            op, ld_o = q_out.data_ptr(), cols
        else:
            op, ld_o, _ = _rows_on(device, q_out, _bf16, T, cols, "q_out")
            _apart(q, q_out, same=True)
            _apart(k, q_out)
            _apart(v, q_out)
    elif q_out is not None:
        raise NVFP4Error("q_out needs q")
    rc = lib.paged_kv_append(qp, ld_q, num_heads, op, ld_o, kp, ld_k, vp, ld_v, pos, _vec_on(device, slots, _i64t, T, "slots"), T,
                             steps, rdim, layout, amplitude, *cache, ks, vs, kb, vb, _raw_stream(device))
    if rc:
        _check(rc, "paged_kv_append")
    return q_out


def paged_attention_blocks(q, k_cache, v_cache, k_scale, v_scale, block_table, q_start, seq_lens, max_new, max_seq, scale=None,
                           window=0, out_dtype=torch.bfloat16, out=None, lse=None, return_lse=False, workspace=None,
                           clear_padding=None):
    """paged_attention over a block-scaled cache: float8_e4m3fn or int8 caches with scales float8_e8m0fnu
    [pages, heads, page size / 16], as paged_kv_append leaves them.  Everything else, the workspace too, as there."""
    lib, device = _lib or load(), _gpu_of(q)
    cache, kb, vb, heads, dim = _block_cache(device, k_cache, v_cache, k_scale, v_scale)
    qp, ld_q, cols = _rows_on(device, q, _bf16, None, None, "q")
    T = q.shape[0]
    num_heads = cols // dim
    if cols == 0 or cols % dim or num_heads % heads:
        raise NVFP4Error("q must be [T, num_heads * %d] with num_heads a multiple of %d" % (dim, heads))
    if not isinstance(seq_lens, _Tensor):
        raise NVFP4Error("seq_lens must be a GPU tensor")
    R = seq_lens.numel()
    table, ld_t, max_pages = _rows_on(device, block_table, _i32, R, None, "block_table")
    if clear_padding is None:
        clear_padding = out is None
    if out is None:
        out = q.new_empty((T, cols), dtype=_bf16 if out_dtype in (OUT_BF16, _bf16) else _f32)
        op, ld_o = out.data_ptr(), cols
    else:
        op, ld_o, _ = _rows_on(device, out, _bf16 if out_dtype in (OUT_BF16, _bf16) else _f32, T, cols, "out")
    if lse is None and return_lse:
        lse = q.new_empty((T, num_heads), dtype=_f32)
    if workspace is None:
        workspace = paged_attention_workspace(T, R, num_heads, heads, dim, max_new, max_seq, q.device)
    bytes_ = workspace.numel()
    rc = lib.paged_attention_blocks(qp, ld_q, T, _vec_on(device, q_start, _i32, R + 1, "q_start"),
                                    _vec_on(device, seq_lens, _i32, R, "seq_lens"), R, max_new, max_seq, num_heads, *cache, kb, vb,
                                    table, max_pages, ld_t,
                                    dim ** -0.5 if scale is None else scale, window, op,
                                    (OUT_BF16 if out.dtype is _bf16 else OUT_F32) + (OUT_CLEAR_PADDING if clear_padding else 0),
                                    ld_o, None if lse is None else _vec_on(device, lse, _f32, T * num_heads, "lse"),
                                    _vec_on(device, workspace, _u8, bytes_, "workspace"), bytes_, _raw_stream(device))
    if rc:
        _check(rc, "paged_attention_blocks")
    return (out, lse) if return_lse else out


def _codes8(device, t, rows, cols, name):
    """(address, rows, columns) of a contiguous int8 matrix."""
    if not isinstance(t, _Tensor) or t.get_device() != device or t.dtype is not _int8 or t.dim() != 2 or not t.is_contiguous() \
            or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        _misplaced(t, _int8, name, "[%s, %s] contiguous" % (rows, cols))
    return t.data_ptr(), t.shape[0], t.shape[1]


def _int8_out(device, x, m, n, out_dtype, out):
    dtype = _bf16 if out_dtype in (OUT_BF16, _bf16) else _f32
    if out is None:
        out = x.new_empty((m, n), dtype=dtype)
        return out, out.data_ptr(), n, OUT_BF16 if dtype is _bf16 else OUT_F32
    op, ld, _ = _rows_on(device, out, dtype, m, n, "out")
    _apart(x, out)
    return out, op, ld, OUT_BF16 if dtype is _bf16 else OUT_F32


def int8_quantize(x, codes=None, scales=None):
    """bf16 [rows, cols] (row stride allowed) -> (codes int8 [rows, cols], scales fp32 [rows]): a scale amax / 127 for each
    row, a token's or an output channel's.  codes and scales share no memory with x or each other."""
    lib, device = _lib or load(), _gpu_of(x)
    xp, ld, cols = _rows_on(device, x, _bf16, None, None, "x")
    rows, given = x.shape[0], codes is not None or scales is not None
    if codes is None:
        codes = x.new_empty((rows, cols), dtype=_int8)
    if scales is None:
        scales = x.new_empty(rows, dtype=_f32)
    cp, sp = _codes8(device, codes, rows, cols, "codes")[0], _vec_on(device, scales, _f32, rows, "scales")
    if given and _meet((xp, xp + 2 * ((rows - 1) * ld + cols)), (cp, cp + rows * cols), (sp, sp + 4 * rows)):
        written = [(cp, rows * cols), (sp, 4 * rows)]
        _apart_all(written, [])
        _apart_from(x, written)
    rc = lib.int8_quantize(xp, rows, cols, ld, cp, sp, _raw_stream(device))
    if rc:
        _check(rc, "int8_quantize")
    return codes, scales


def gemm_w8a8_workspace(tokens, n, k, device="cuda"):
    """A workspace for gemm_w8a8 and int8_linear calls of up to these tokens, n channels and k columns; for several layers
    the largest of theirs serves all.  Without an element where no such product is split."""
    lib = load()
    rc = lib.gemm_w8a8(None, None, tokens, None, None, n, k, None, OUT_BF16, n, None, 0, None)     # sizes come first
    if rc not in (0, -1):
        _check(rc, "gemm_w8a8")
    return torch.empty(lib.gemm_w8a8_workspace_bytes(tokens, n, k), dtype=_u8, device=device)


def _int8_workspace(device, lib, like, m, n, k, workspace):
    """(workspace or None, its address, its bytes): one that products of few rows are split with, allocated if None."""
    if workspace is None:
        need = lib.gemm_w8a8_workspace_bytes(m, n, k)
        if not need:
            return None, None, 0
        workspace = like.new_empty(need, dtype=_u8)
        return workspace, workspace.data_ptr(), need
    bytes_ = workspace.numel() if isinstance(workspace, _Tensor) else 0
    return workspace, _vec_on(device, workspace, _u8, bytes_, "workspace"), bytes_


def gemm_w8a8(a, a_scale, w, w_scale, out_dtype=torch.bfloat16, out=None, workspace=None):
    """out [m, n] = a_scale[m] * (a [m, k] . w [n, k]^T) * w_scale[n]: int8 codes with a scale for each row, as
    int8_quantize gives them.  workspace: from gemm_w8a8_workspace, of as many tokens or more (allocated if None; without an
    element: k is not split)."""
    lib, device = _lib or load(), _gpu_of(a)
    ap, m, k = _codes8(device, a, None, None, "a")
    wp, n, _ = _codes8(device, w, None, k, "w")
    made = out is not None
    out, op, ld, kind = _int8_out(device, a, m, n, out_dtype, out)
    sp, tp = _vec_on(device, a_scale, _f32, m, "a_scale"), _vec_on(device, w_scale, _f32, n, "w_scale")
    given = workspace is not None
    workspace, wsp, bytes_ = _int8_workspace(device, lib, a, m, n, k, workspace)
    if (given or made) and _meet((ap, ap + m * k), (sp, sp + 4 * m), (wp, wp + n * k), (tp, tp + 4 * n), (wsp or 0, (wsp or 0) + bytes_),
                                 (op, op + ((m - 1) * ld + n) * out.element_size())):
        read = [(ap, m * k), (sp, 4 * m), (wp, n * k), (tp, 4 * n)]
        if given:
            _apart_all([(wsp, bytes_)], read)
            read.append((wsp, bytes_))
        if made:
            _apart_from(out, read)
    rc = lib.gemm_w8a8(ap, sp, m, wp, tp, n, k, op, kind, ld, wsp, bytes_, _raw_stream(device))
    if rc:
        _check(rc, "gemm_w8a8")
    return out


def int8_linear(x, w, w_scale, out_dtype=torch.bfloat16, out=None, codes=None, scales=None, workspace=None):
    """x bf16 [m, k] (row stride allowed), quantised to int8 with a scale for each token, times w (int8 [n, k], w_scale
    fp32 [n]; from int8_quantize of the weight).  codes, scales: where x's are left (allocated if None); workspace as in
    gemm_w8a8.  What the call writes shares no memory with anything else of it (out may be other columns of x's matrix)."""
    lib, device = _lib or load(), _gpu_of(x)
    xp, ld_x, k = _rows_on(device, x, _bf16, None, None, "x")
    m = x.shape[0]
    wp, n, _ = _codes8(device, w, None, k, "w")
    tp = _vec_on(device, w_scale, _f32, n, "w_scale")
    need = lib.gemm_w8a8_workspace_bytes(m, n, k) if workspace is None else 0
    written = []
    if codes is None and scales is None and workspace is None:
        # one allocation for all three, alive until the call has been enqueued
        at, ws_at = m * k, (m * (k + 4) + 255) // 256 * 256
        held = x.new_empty(ws_at + need, dtype=_u8)
        cp = held.data_ptr()
        sp, wsp, bytes_ = cp + at, cp + ws_at if need else None, need
    else:
        if codes is None:
            codes = x.new_empty((m, k), dtype=_int8)
        if scales is None:
            scales = x.new_empty(m, dtype=_f32)
        if workspace is None and need:
            workspace = x.new_empty(need, dtype=_u8)
        cp, sp = _codes8(device, codes, m, k, "codes")[0], _vec_on(device, scales, _f32, m, "scales")
        bytes_ = workspace.numel() if isinstance(workspace, _Tensor) else 0
        wsp = None if workspace is None else _vec_on(device, workspace, _u8, bytes_, "workspace")
        written = [(cp, m * k), (sp, 4 * m), (wsp or 0, bytes_)]
    made = out is not None
    out, op, ld, kind = _int8_out(device, x, m, n, out_dtype, out)
    if (made or written) and _meet((xp, xp + 2 * ((m - 1) * ld_x + k)), (wp, wp + n * k), (tp, tp + 4 * n),
                                   (op, op + ((m - 1) * ld + n) * out.element_size()), *((p, p + size) for p, size in written)):
        _apart_all(written, [(wp, n * k), (tp, 4 * n)])
        _apart_from(x, written)
        _apart_from(out, written + [(wp, n * k), (tp, 4 * n)])
    rc = lib.int8_linear(xp, m, k, ld_x, cp, sp, wp, tp, n, op, kind, ld, wsp, bytes_, _raw_stream(device))
    if rc:
        _check(rc, "int8_linear")
    return out
