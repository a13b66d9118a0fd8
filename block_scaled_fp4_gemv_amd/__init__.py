"""Python binding of the MI355X NVFP4 block-scaled batched GEMV (libnvfp4gemv.so).

Argument marshalling only: every step of the GEMV runs in the HIP library. The
names mirror the C ABI in include/nvfp4_gemv.h. torch provides device memory and
the stream; tensors are passed as raw device pointers.

    nvfp4_gemv(a, b, sfa, sfb, c, M, K, L, sf_layout, stream=None)
    nvfp4_gemv_scaled(..., sf_layout, alpha, workspace=None, stream=None)
    nvfp4_scales_to_blocked(plain, blocked, rows, K, L, stream=None)

FP4 linear layers and routed experts (last part of the header):

    nvfp4_global_scale(x, scale, rows, K, L, workspace)
    nvfp4_quantize(x, codes, scales, rows, K, L, sf_layout, global_scale=None)
    nvfp4_dequantize(codes, scales, out, rows, K, L, sf_layout, global_scale=None)
    nvfp4_gemm(a, b, sfa, sfb, c, M, N, K, L, sf_layout, workspace=None)
    nvfp4_moe_route(logits, ids, weights, offsets, order, T, E, k, workspace=...)
    nvfp4_gemm_experts(a, b, sfa, sfb, c, M, K, E, rows, slots_per_row, sf_layout, offsets, order)
    nvfp4_moe_combine(y, ids, weights, out, T, k, M)

Attention over a paged NVFP4 key/value cache:

    nvfp4_rope_frequencies(R, base, method="unscaled", ...)
    nvfp4_rope(x, out, positions, frequencies, T, H, D, R, layout="half")
    Nvfp4Cache(k_codes, k_scales, v_codes, v_scales, pages, page_size, heads, head_size)
    nvfp4_cache_write(cache, k, v, slots, T)
    nvfp4_cache_read(cache, k, v, slots, T)
    nvfp4_cache_attention(cache, q, out, offsets, lengths, table, T, H, B, max_q, max_length, workspace=...)

    a   uint8 [L, M, K/2]   packed E2M1, low nibble = even k
    b   uint8 [L, K/2]
    sfa uint8 plain [L, M, K/16] or blocked [L, ceil(M/128)*ceil(K/64)*512]
    sfb uint8 plain [L, K/16]    or blocked [L, ceil(K/64)*512]
    c   float16 [L, M]          written

There is no fallback: if the library is missing the import fails.
"""
from __future__ import annotations

import ctypes
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libnvfp4gemv.so")

NVFP4_SF_PLAIN = 0
NVFP4_SF_BLOCKED = 1
NVFP4_OK = 0
NVFP4_ERR_NULL_POINTER = 1
NVFP4_ERR_INVALID_SHAPE = 2
NVFP4_ERR_MISALIGNED = 3
NVFP4_ERR_INVALID_LAYOUT = 4
NVFP4_ERR_WORKSPACE = 5
NVFP4_ERR_HIP = 6
NVFP4_ERR_INVALID_SCALE = 7
NVFP4_ERR_INVALID_STRIDE = 8
NVFP4_ERR_INVALID_TYPE = 9
NVFP4_ERR_INVALID_ROUTING = 10
NVFP4_ERR_INVALID_ROTATION = 11
NVFP4_ERR_INVALID_CACHE = 12
NVFP4_F16 = 0
NVFP4_BF16 = 1
NVFP4_F32 = 2
NVFP4_SCORE_SOFTMAX = 0
NVFP4_SCORE_SIGMOID = 1
NVFP4_ROPE_HALF = 0
NVFP4_ROPE_INTERLEAVED = 1
NVFP4_ROPE_UNSCALED = 0
NVFP4_ROPE_LINEAR = 1
NVFP4_ROPE_BASE = 2
NVFP4_ROPE_BANDS = 3
NVFP4_ROPE_RAMP = 4
NVFP4_WORKSPACE_MAX_BYTES = 67174400        # serves any call that takes one of the layers', experts' and attention's

EXPORTED_SYMBOLS = (
    "nvfp4_gemv",
    "nvfp4_gemv_noalloc",
    "nvfp4_gemv_noalloc_scratch_bytes",
    "nvfp4_gemv_workspace_bytes",
    "nvfp4_gemv_ex",
    "nvfp4_gemv_scaled",
    "nvfp4_gemv_strided",
    "nvfp4_gemv_dense_strides",
    "nvfp4_gemv_plan",
    "nvfp4_gemv_two_vectors_plan",
    "nvfp4_gemm_small_n",
    "nvfp4_gemm_small_n_plan",
    "nvfp4_scales_to_blocked",
    "nvfp4_blocked_scales_bytes",
    "nvfp4_global_scale",
    "nvfp4_global_scale_workspace_bytes",
    "nvfp4_quantize",
    "nvfp4_dequantize",
    "nvfp4_gemm",
    "nvfp4_gemm_workspace_bytes",
    "nvfp4_gemm_plan",
    "nvfp4_moe_route",
    "nvfp4_moe_route_workspace_bytes",
    "nvfp4_gemm_experts",
    "nvfp4_gemm_experts_workspace_bytes",
    "nvfp4_moe_combine",
    "nvfp4_rope",
    "nvfp4_rope_frequencies",
    "nvfp4_cache_write",
    "nvfp4_cache_read",
    "nvfp4_cache_attention",
    "nvfp4_cache_attention_workspace_bytes",
    "nvfp4_status_string",
    "nvfp4_last_hip_error",
)


class Nvfp4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = status_string(status)
        if status == NVFP4_ERR_HIP:
            msg += f" (hipError_t {lib().nvfp4_last_hip_error()})"
        super().__init__(f"{where}: {msg} [status {status}]")


class Strides(ctypes.Structure):
    """nvfp4_strides_t: byte strides (c_batch in float16 elements)."""
    _fields_ = [("a_row", ctypes.c_int64), ("a_batch", ctypes.c_int64),
                ("b_batch", ctypes.c_int64),
                ("sfa_row", ctypes.c_int64), ("sfa_batch", ctypes.c_int64),
                ("sfb_batch", ctypes.c_int64),
                ("c_batch", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class Plan(ctypes.Structure):
    _fields_ = [("lanes_per_row", ctypes.c_int32),
                ("rows_per_wg", ctypes.c_int32),
                ("k_splits", ctypes.c_int32),
                ("k_per_split", ctypes.c_int32),
                ("workgroups", ctypes.c_int64),
                ("threads_per_wg", ctypes.c_int32),
                ("lds_bytes", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class GemmPlan(ctypes.Structure):
    """nvfp4_gemm_plan_t."""
    _fields_ = [("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("k_splits", ctypes.c_int32), ("k_per_split", ctypes.c_int32),
                ("workgroups", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class Routing(ctypes.Structure):
    """nvfp4_routing_t."""
    _fields_ = [("score", ctypes.c_int32), ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scaling", ctypes.c_float)]


class RopeScaling(ctypes.Structure):
    """nvfp4_rope_scaling_t."""
    _fields_ = [("method", ctypes.c_int32), ("factor", ctypes.c_double), ("length", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double)]


class CacheStruct(ctypes.Structure):
    """nvfp4_cache_t."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("head_size", ctypes.c_int64), ("code_page_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64)]


class Attention(ctypes.Structure):
    """nvfp4_attention_t."""
    _fields_ = [("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("max_q", ctypes.c_int64),
                ("max_length", ctypes.c_int64), ("window", ctypes.c_int64), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int32)]


_lib = None


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m block_scaled_fp4_gemv_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.nvfp4_gemv.restype = i32
    L.nvfp4_gemv.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp]
    L.nvfp4_gemv_ex.restype = i32
    L.nvfp4_gemv_noalloc.restype = i32
    L.nvfp4_gemv_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp]
    L.nvfp4_gemv_noalloc_scratch_bytes.restype = ctypes.c_size_t
    L.nvfp4_gemv_noalloc_scratch_bytes.argtypes = []
    L.nvfp4_gemv_ex.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, ctypes.c_size_t, vp]
    L.nvfp4_gemv_scaled.restype = i32
    L.nvfp4_gemv_scaled.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, ctypes.c_float, vp,
                                    ctypes.c_size_t, vp]
    L.nvfp4_gemv_strided.restype = i32
    L.nvfp4_gemv_strided.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, ctypes.POINTER(Strides),
                                     ctypes.c_float, vp, ctypes.c_size_t, vp]
    L.nvfp4_gemv_dense_strides.restype = None
    L.nvfp4_gemv_dense_strides.argtypes = [i64, i64, i64, i32, ctypes.POINTER(Strides)]
    L.nvfp4_gemv_workspace_bytes.restype = ctypes.c_size_t
    L.nvfp4_gemv_workspace_bytes.argtypes = [i64, i64, i64]
    L.nvfp4_gemv_plan.restype = i32
    L.nvfp4_gemv_plan.argtypes = [i64, i64, i64, ctypes.POINTER(Plan)]
    L.nvfp4_gemv_two_vectors_plan.restype = i32
    L.nvfp4_gemv_two_vectors_plan.argtypes = [i64, i64, i64, ctypes.POINTER(Plan)]
    L.nvfp4_gemm_small_n.restype = i32
    L.nvfp4_gemm_small_n.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, ctypes.c_float, vp]
    L.nvfp4_gemm_small_n_plan.restype = i32
    L.nvfp4_gemm_small_n_plan.argtypes = [i64, i64, i64, i64, i32, ctypes.POINTER(ctypes.c_int32),
                                          ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int32)]
    L.nvfp4_scales_to_blocked.restype = i32
    L.nvfp4_scales_to_blocked.argtypes = [vp, vp, i64, i64, i64, vp]
    L.nvfp4_blocked_scales_bytes.restype = ctypes.c_size_t
    L.nvfp4_blocked_scales_bytes.argtypes = [i64, i64, i64]
    f32, size = ctypes.c_float, ctypes.c_size_t
    L.nvfp4_global_scale.restype = i32
    L.nvfp4_global_scale.argtypes = [vp, i32, vp, i64, i64, i64, i64, i64, vp, size, vp]
    L.nvfp4_global_scale_workspace_bytes.restype = size
    L.nvfp4_global_scale_workspace_bytes.argtypes = []
    L.nvfp4_quantize.restype = i32
    L.nvfp4_quantize.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, i64, i64, i32, vp]
    L.nvfp4_dequantize.restype = i32
    L.nvfp4_dequantize.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, i32, vp]
    L.nvfp4_gemm.restype = i32
    L.nvfp4_gemm.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, i64, i32, f32, vp, vp, vp, size, vp]
    L.nvfp4_gemm_workspace_bytes.restype = size
    L.nvfp4_gemm_workspace_bytes.argtypes = [i64, i64, i64, i64]
    L.nvfp4_gemm_plan.restype = i32
    L.nvfp4_gemm_plan.argtypes = [i64, i64, i64, i64, ctypes.POINTER(GemmPlan)]
    L.nvfp4_moe_route.restype = i32
    L.nvfp4_moe_route.argtypes = [vp, i32, vp, vp, vp, vp, vp, i64, i64, i64, ctypes.POINTER(Routing), vp, size, vp]
    L.nvfp4_moe_route_workspace_bytes.restype = size
    L.nvfp4_moe_route_workspace_bytes.argtypes = [i64, i64, i64]
    L.nvfp4_gemm_experts.restype = i32
    L.nvfp4_gemm_experts.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, i64, i64, i64, i32, vp, vp, f32, vp, vp, vp,
                                     size, vp]
    L.nvfp4_gemm_experts_workspace_bytes.restype = size
    L.nvfp4_gemm_experts_workspace_bytes.argtypes = [i64, i64, i64, i64]
    L.nvfp4_moe_combine.restype = i32
    L.nvfp4_moe_combine.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, vp]
    L.nvfp4_rope.restype = i32
    L.nvfp4_rope.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64, i32, f32, i32, vp]
    L.nvfp4_rope_frequencies.restype = i32
    L.nvfp4_rope_frequencies.argtypes = [ctypes.POINTER(ctypes.c_double), i64, ctypes.c_double,
                                         ctypes.POINTER(RopeScaling)]
    cache, att = ctypes.POINTER(CacheStruct), ctypes.POINTER(Attention)
    L.nvfp4_cache_write.restype = i32
    L.nvfp4_cache_write.argtypes = [cache, vp, vp, i32, vp, i64, i64, i64, i64, i64, vp]
    L.nvfp4_cache_read.restype = i32
    L.nvfp4_cache_read.argtypes = [cache, vp, vp, i32, vp, i64, vp]
    L.nvfp4_cache_attention.restype = i32
    L.nvfp4_cache_attention.argtypes = [cache, vp, i32, vp, vp, vp, vp, vp, i64, i64, i64, i64, att, vp, size, vp]
    L.nvfp4_cache_attention_workspace_bytes.restype = size
    L.nvfp4_cache_attention_workspace_bytes.argtypes = [cache, i32, i64, i64, i64, att]
    L.nvfp4_status_string.restype = ctypes.c_char_p
    L.nvfp4_status_string.argtypes = [i32]
    L.nvfp4_last_hip_error.restype = i32
    L.nvfp4_last_hip_error.argtypes = []
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().nvfp4_status_string(status).decode()


def layout_id(layout) -> int:
    if layout in (NVFP4_SF_PLAIN, "plain"):
        return NVFP4_SF_PLAIN
    if layout in (NVFP4_SF_BLOCKED, "blocked"):
        return NVFP4_SF_BLOCKED
    return int(layout)   # passed through; the library rejects unknown values


def cdiv(a: int, b: int) -> int:
    return (a + b - 1) // b


def operand_bytes(M: int, K: int, L: int, layout) -> dict:
    """Bytes each operand must hold for a shape."""
    lay = layout_id(layout)
    nkb = K // 16
    if lay == NVFP4_SF_BLOCKED:
        sfa = L * cdiv(M, 128) * cdiv(nkb, 4) * 512
        sfb = L * cdiv(nkb, 4) * 512
    else:
        sfa, sfb = L * M * nkb, L * nkb
    return {"a": L * M * K // 2, "b": L * K // 2, "sfa": sfa, "sfb": sfb, "c": 2 * L * M}


def _ptr_and_bytes(x):
    """(device pointer, byte size) of a torch tensor, or (x, None) for a raw int."""
    if x is None:
        return None, None
    if isinstance(x, int):
        return x, None
    if not x.is_cuda:
        raise ValueError("operands must be device tensors")
    if not x.is_contiguous():
        raise ValueError("operands must be contiguous")
    return x.data_ptr(), x.numel() * x.element_size()


_raw_stream = None


def _stream_handle(stream):
    if stream is None:
        # the current stream's handle without a Stream object (that takes 2.8 us, this 0.2)
        global _raw_stream
        if _raw_stream is None:
            import torch
            get, dev = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
            if get is None or dev is None:
                return torch.cuda.current_stream().cuda_stream
            torch.cuda.current_stream()                     # initialises torch's device state
            _raw_stream = lambda: get(dev())  # noqa: E731
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_sizes(M, K, L, layout, **ops):
    if M < 1 or K < 1 or L < 1 or K % 32:
        return   # the library reports shape errors itself
    need = operand_bytes(M, K, L, layout)
    for name, nbytes in ops.items():
        if nbytes is not None and nbytes < need[name]:
            raise ValueError(f"{name} holds {nbytes} bytes, the shape needs {need[name]}")


def nvfp4_gemv(a, b, sfa, sfb, c, M: int, K: int, L: int, sf_layout, stream=None) -> None:
    """Enqueue c = GEMV(a, b, sfa, sfb) on ``stream`` (default: torch's current stream)."""
    (pa, na), (pb, nb), (psa, nsa), (psb, nsb), (pc, nc) = map(_ptr_and_bytes, (a, b, sfa, sfb, c))
    lay = layout_id(sf_layout)
    _check_sizes(M, K, L, lay, a=na, b=nb, sfa=nsa, sfb=nsb, c=nc)
    st = lib().nvfp4_gemv(pa, pb, psa, psb, pc, M, K, L, lay, _stream_handle(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_gemv")


def nvfp4_gemv_noalloc(a, b, sfa, sfb, c, M: int, K: int, L: int, sf_layout, stream=None) -> None:
    """As nvfp4_gemv, with the split-K workspace taken from the library's fixed
    per-device scratch array (no allocation; calls on one GPU must not overlap)."""
    (pa, na), (pb, nb), (psa, nsa), (psb, nsb), (pc, nc) = map(_ptr_and_bytes, (a, b, sfa, sfb, c))
    lay = layout_id(sf_layout)
    _check_sizes(M, K, L, lay, a=na, b=nb, sfa=nsa, sfb=nsb, c=nc)
    st = lib().nvfp4_gemv_noalloc(pa, pb, psa, psb, pc, M, K, L, lay, _stream_handle(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_gemv_noalloc")


def nvfp4_gemv_noalloc_scratch_bytes() -> int:
    return int(lib().nvfp4_gemv_noalloc_scratch_bytes())


def nvfp4_gemv_workspace_bytes(M: int, K: int, L: int) -> int:
    return int(lib().nvfp4_gemv_workspace_bytes(M, K, L))


def nvfp4_gemv_ex(a, b, sfa, sfb, c, M: int, K: int, L: int, sf_layout, workspace,
                  workspace_bytes: int | None = None, stream=None) -> None:
    """As nvfp4_gemv with a caller-owned (zero-initialised) workspace."""
    (pa, na), (pb, nb), (psa, nsa), (psb, nsb), (pc, nc) = map(_ptr_and_bytes, (a, b, sfa, sfb, c))
    pw, nw = _ptr_and_bytes(workspace)
    if workspace_bytes is None:
        workspace_bytes = nw or 0
    lay = layout_id(sf_layout)
    _check_sizes(M, K, L, lay, a=na, b=nb, sfa=nsa, sfb=nsb, c=nc)
    st = lib().nvfp4_gemv_ex(pa, pb, psa, psb, pc, M, K, L, lay, pw, workspace_bytes,
                             _stream_handle(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_gemv_ex")


def nvfp4_gemv_scaled(a, b, sfa, sfb, c, M: int, K: int, L: int, sf_layout, alpha: float,
                      workspace=None, workspace_bytes: int | None = None, stream=None) -> None:
    """Enqueue c = fp16(alpha * GEMV(a, b, sfa, sfb)); ``workspace`` None uses
    the library-owned one, else a caller-owned (zero-initialised) workspace."""
    (pa, na), (pb, nb), (psa, nsa), (psb, nsb), (pc, nc) = map(_ptr_and_bytes, (a, b, sfa, sfb, c))
    pw, nw = _ptr_and_bytes(workspace)
    if workspace_bytes is None:
        workspace_bytes = nw or 0
    lay = layout_id(sf_layout)
    _check_sizes(M, K, L, lay, a=na, b=nb, sfa=nsa, sfb=nsb, c=nc)
    st = lib().nvfp4_gemv_scaled(pa, pb, psa, psb, pc, M, K, L, lay, float(alpha), pw,
                                 workspace_bytes, _stream_handle(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_gemv_scaled")


def nvfp4_gemv_dense_strides(M: int, K: int, L: int, sf_layout) -> dict:
    st = Strides()
    lib().nvfp4_gemv_dense_strides(M, K, L, layout_id(sf_layout), ctypes.byref(st))
    return st.as_dict()


def _raw_ptr(x):
    """Device pointer of a torch tensor (any strides: the library reads through
    the strides it is given), or a raw int."""
    if x is None or isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("operands must be device tensors")
    return x.data_ptr()


def nvfp4_gemv_strided(a, b, sfa, sfb, c, M: int, K: int, L: int, sf_layout, strides: dict,
                       alpha: float = 1.0, workspace=None, workspace_bytes: int | None = None,
                       stream=None) -> None:
    """Enqueue c = fp16(alpha * GEMV) over strided operands: ``strides`` holds
    the fields of nvfp4_strides_t (bytes; c_batch in elements). The tensors
    are passed by base pointer: the library reads and writes through the
    strides, so each tensor must cover what they address."""
    st = Strides(**strides)
    pw, nw = _ptr_and_bytes(workspace)
    if workspace_bytes is None:
        workspace_bytes = nw or 0
    rc = lib().nvfp4_gemv_strided(_raw_ptr(a), _raw_ptr(b), _raw_ptr(sfa), _raw_ptr(sfb), _raw_ptr(c),
                                  M, K, L, layout_id(sf_layout), ctypes.byref(st), float(alpha), pw,
                                  workspace_bytes, _stream_handle(stream))
    if rc != NVFP4_OK:
        raise Nvfp4Error(rc, "nvfp4_gemv_strided")


def nvfp4_gemv_plan(M: int, K: int, L: int) -> dict:
    plan = Plan()
    st = lib().nvfp4_gemv_plan(M, K, L, ctypes.byref(plan))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_gemv_plan")
    return plan.as_dict()


def nvfp4_gemv_two_vectors_plan(M: int, K: int, L: int) -> dict:
    plan = Plan()
    st = lib().nvfp4_gemv_two_vectors_plan(M, K, L, ctypes.byref(plan))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_gemv_two_vectors_plan")
    return plan.as_dict()


def nvfp4_gemm_small_n_plan(M: int, N: int, K: int, L: int, layout="blocked") -> dict:
    r, wg, lds = ctypes.c_int32(), ctypes.c_int64(), ctypes.c_int32()
    st = lib().nvfp4_gemm_small_n_plan(M, N, K, L, layout_id(layout), ctypes.byref(r), ctypes.byref(wg),
                                       ctypes.byref(lds))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_gemm_small_n_plan")
    return {"rows_per_wg": r.value, "workgroups": wg.value, "lds_bytes": lds.value}


def small_n_operand_bytes(M: int, N: int, K: int, L: int, layout) -> dict:
    """Bytes each operand of nvfp4_gemm_small_n must hold."""
    lay = layout_id(layout)
    nkb = K // 16
    if lay == NVFP4_SF_BLOCKED:
        sfa, sfb = L * cdiv(M, 128) * cdiv(nkb, 4) * 512, L * cdiv(N, 128) * cdiv(nkb, 4) * 512
    else:
        sfa, sfb = L * M * nkb, L * N * nkb
    return {"a": L * M * K // 2, "b": L * N * K // 2, "sfa": sfa, "sfb": sfb, "c": 2 * L * N * M}


def nvfp4_gemm_small_n(a, b, sfa, sfb, c, M: int, N: int, K: int, L: int, sf_layout,
                       alpha: float = 1.0, stream=None) -> None:
    """Enqueue c[l][n][m] = fp16(alpha * sum_k A*SFA*B_n*SFB_n) for N = 1..8 vectors."""
    (pa, na), (pb, nb), (psa, nsa), (psb, nsb), (pc, nc) = map(_ptr_and_bytes, (a, b, sfa, sfb, c))
    lay = layout_id(sf_layout)
    if M >= 1 and K >= 32 and K % 32 == 0 and L >= 1 and 1 <= N <= 8:
        need = small_n_operand_bytes(M, N, K, L, lay)
        for name, nbytes in dict(a=na, b=nb, sfa=nsa, sfb=nsb, c=nc).items():
            if nbytes is not None and nbytes < need[name]:
                raise ValueError(f"{name} holds {nbytes} bytes, the shape needs {need[name]}")
    st = lib().nvfp4_gemm_small_n(pa, pb, psa, psb, pc, M, N, K, L, lay, float(alpha), _stream_handle(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_gemm_small_n")


def nvfp4_blocked_scales_bytes(rows: int, K: int, L: int) -> int:
    return int(lib().nvfp4_blocked_scales_bytes(rows, K, L))


def nvfp4_scales_to_blocked(plain, blocked, rows: int, K: int, L: int, stream=None) -> None:
    """Enqueue the plain -> 128x4 blocked reblock of a scale tensor.
    plain uint8 [L, rows, K/16]; blocked uint8 of nvfp4_blocked_scales_bytes bytes."""
    (pp, npb), (pb, nbb) = _ptr_and_bytes(plain), _ptr_and_bytes(blocked)
    need = nvfp4_blocked_scales_bytes(rows, K, L)
    if need and npb is not None and npb < L * rows * (K // 16):
        raise ValueError(f"plain holds {npb} bytes, the shape needs {L * rows * (K // 16)}")
    if need and nbb is not None and nbb < need:
        raise ValueError(f"blocked holds {nbb} bytes, the shape needs {need}")
    st = lib().nvfp4_scales_to_blocked(pp, pb, rows, K, L, _stream_handle(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_scales_to_blocked")


# ---------------------------------------------------------------- FP4 linear layers, routed experts

_DTYPES = {"torch.float16": (NVFP4_F16, 2), "torch.bfloat16": (NVFP4_BF16, 2), "torch.float32": (NVFP4_F32, 4)}


def _dtype_id(x, dtype):
    """nvfp4_dtype_t of a tensor (or of ``dtype``, needed for raw pointers)."""
    if dtype is None:
        if x is None or isinstance(x, int):
            raise ValueError("raw pointers need dtype=")
        dtype = x.dtype
    if isinstance(dtype, int):
        return dtype                        # passed through; the library rejects unknown values
    known = _DTYPES.get(str(dtype))
    if known is None:
        raise ValueError(f"{dtype} is none of float16, bfloat16, float32")
    return known[0]


def _op(x, need, name, dtype=None):
    """Device pointer of a dense tensor that holds at least ``need`` bytes and,
    where ``dtype`` is given, has that type; raw pointers and None pass."""
    if x is None or isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("operands must be device tensors")
    if not x.is_contiguous():
        raise ValueError("operands must be contiguous")
    if dtype is not None and str(x.dtype) != dtype:
        raise ValueError(f"{name} is {x.dtype}, not {dtype.replace('torch.', '')}")
    held = x.numel() * x.element_size()
    if held < need:
        raise ValueError(f"{name} holds {held} bytes, the shape needs {need}")
    return x.data_ptr()


_F32, _I32 = "torch.float32", "torch.int32"


def _workspace(x, nbytes):
    """(pointer, bytes) of a workspace, its own size by default."""
    if nbytes is None:
        nbytes = 0 if x is None or isinstance(x, int) else x.numel() * x.element_size()
    if nbytes < 0:
        raise ValueError(f"workspace_bytes is {nbytes}")
    return _op(x, nbytes, "workspace"), nbytes


def _strided(x, name, dt, rows, K, L, row_stride, batch_stride):
    """Pointer of an [L][rows][K] tensor of type ``dt`` and its strides in elements,
    checked against what the tensor's memory holds behind its first element."""
    given = row_stride is not None or batch_stride is not None
    if row_stride is None:
        row_stride = K
    if batch_stride is None:
        batch_stride = rows * row_stride
    if x is None or isinstance(x, int):
        return x, row_stride, batch_stride
    if not x.is_cuda:
        raise ValueError("operands must be device tensors")
    if not given and not x.is_contiguous():
        raise ValueError(f"{name} is not contiguous: give its strides")
    size = 4 if dt == NVFP4_F32 else 2                       # of the elements that are read, whatever x's type
    if row_stride == K and batch_stride == rows * K and x.is_contiguous():
        held = x.numel() * x.element_size() // size
        if rows * K * L > held:
            raise ValueError(f"{name} holds {held} elements, the shape needs {rows * K * L}")
    elif min(rows, K, L) >= 1 and min(row_stride, batch_stride) >= 0:
        held = (x.untyped_storage().nbytes() - x.storage_offset() * x.element_size()) // size
        need = (L - 1) * batch_stride + (rows - 1) * row_stride + K
        if held < need:
            raise ValueError(f"{name} holds {held} elements, the shape needs {need}")
    return x.data_ptr(), row_stride, batch_stride


def _scale_bytes(rows, K, L, lay):
    return L * (cdiv(rows, 128) * cdiv(K, 64) * 512 if lay == NVFP4_SF_BLOCKED else rows * (K // 16))


def _done(status, where) -> None:
    if status != NVFP4_OK:
        raise Nvfp4Error(status, where)


def nvfp4_global_scale_workspace_bytes() -> int:
    return int(lib().nvfp4_global_scale_workspace_bytes())


def nvfp4_global_scale(x, scale, rows: int, K: int, L: int, workspace, workspace_bytes: int | None = None,
                       row_stride: int | None = None, batch_stride: int | None = None, dtype=None,
                       stream=None) -> None:
    """Enqueue scale[0] = max finite |x| * (1 / 2688) (strides in elements; dense by default)."""
    dt = _dtype_id(x, dtype)
    px, rs, bs = _strided(x, "x", dt, rows, K, L, row_stride, batch_stride)
    pw, nw = _workspace(workspace, workspace_bytes)
    _done(lib().nvfp4_global_scale(px, dt, _op(scale, 4, "scale", _F32), rows, K, L, rs, bs, pw, nw,
                                   _stream_handle(stream)), "nvfp4_global_scale")


def nvfp4_quantize(x, codes, scales, rows: int, K: int, L: int, sf_layout, global_scale=None,
                   row_stride: int | None = None, batch_stride: int | None = None, dtype=None,
                   stream=None) -> None:
    """Enqueue the quantisation of x [L][rows][K] (strides in elements; dense by
    default) to NVFP4 codes and scales; global_scale: float32 on the device."""
    dt = _dtype_id(x, dtype)
    px, rs, bs = _strided(x, "x", dt, rows, K, L, row_stride, batch_stride)
    lay = layout_id(sf_layout)
    on = 1 if min(rows, K, L) >= 1 else 0                   # the library reports shape errors itself
    _done(lib().nvfp4_quantize(px, dt, _op(global_scale, 4, "global_scale", _F32),
                               _op(codes, on * L * rows * K // 2, "codes"),
                               _op(scales, on * _scale_bytes(rows, K, L, lay), "scales"), rows, K, L, rs, bs, lay,
                               _stream_handle(stream)), "nvfp4_quantize")


def nvfp4_dequantize(codes, scales, out, rows: int, K: int, L: int, sf_layout, global_scale=None, dtype=None,
                     stream=None) -> None:
    """Enqueue out [L][rows][K] = the values that codes and scales stand for."""
    lay, dt = layout_id(sf_layout), _dtype_id(out, dtype)
    n = L * rows * K if min(rows, K, L) >= 1 else 0
    _done(lib().nvfp4_dequantize(_op(codes, n // 2, "codes"),
                                 _op(scales, _scale_bytes(rows, K, L, lay) if n else 0, "scales"),
                                 _op(global_scale, 4, "global_scale", _F32),
                                 _op(out, n * (4 if dt == NVFP4_F32 else 2), "out"), dt, rows, K, L, lay,
                                 _stream_handle(stream)), "nvfp4_dequantize")


def nvfp4_gemm_workspace_bytes(M: int, N: int, K: int, L: int) -> int:
    return int(lib().nvfp4_gemm_workspace_bytes(M, N, K, L))


def nvfp4_gemm_plan(M: int, N: int, K: int, L: int) -> dict:
    plan = GemmPlan()
    _done(lib().nvfp4_gemm_plan(M, N, K, L, ctypes.byref(plan)), "nvfp4_gemm_plan")
    return plan.as_dict()


def nvfp4_gemm(a, b, sfa, sfb, c, M: int, N: int, K: int, L: int, sf_layout, alpha: float = 1.0, scale_a=None,
               scale_b=None, workspace=None, workspace_bytes: int | None = None, dtype=None, stream=None) -> None:
    """Enqueue c[l][n][m] = alpha * ga * gb * sum_k A*SFA*B_n*SFB_n for any N; c
    float16, bfloat16 or float32; scale_a, scale_b: float32 on the device; a
    (zero-initialised) workspace of nvfp4_gemm_workspace_bytes, which fewer rows
    may raise, or of NVFP4_WORKSPACE_MAX_BYTES."""
    lay, dt = layout_id(sf_layout), _dtype_id(c, dtype)
    pw, nw = _workspace(workspace, workspace_bytes)
    on = 1 if min(M, N, K, L) >= 1 else 0
    _done(lib().nvfp4_gemm(_op(a, on * L * M * K // 2, "a"), _op(b, on * L * N * K // 2, "b"),
                           _op(sfa, on * _scale_bytes(M, K, L, lay), "sfa"),
                           _op(sfb, on * _scale_bytes(N, K, L, lay), "sfb"),
                           _op(c, on * L * N * M * (4 if dt == NVFP4_F32 else 2), "c"), dt, M, N, K, L, lay,
                           alpha, _op(scale_a, 4, "scale_a", _F32), _op(scale_b, 4, "scale_b", _F32), pw, nw,
                           _stream_handle(stream)), "nvfp4_gemm")


def nvfp4_moe_route_workspace_bytes(T: int, E: int, k: int) -> int:
    return int(lib().nvfp4_moe_route_workspace_bytes(T, E, k))


_SCORES = {"softmax": NVFP4_SCORE_SOFTMAX, "sigmoid": NVFP4_SCORE_SIGMOID}


def nvfp4_moe_route(logits, ids, weights, offsets, order, T: int, E: int, k: int, score="softmax", bias=None,
                    n_group: int = 1, topk_group: int = 1, group_top: int = 1, renormalize: bool = True,
                    scaling: float = 1.0, workspace=None, workspace_bytes: int | None = None, dtype=None,
                    stream=None) -> None:
    """Enqueue the routing of T tokens to k of E experts: ids and weights [T][k],
    and the experts' lists (offsets [E + 1], order [T * k])."""
    dt = _dtype_id(logits, dtype)
    pw, nw = _workspace(workspace, workspace_bytes)
    on = 1 if min(T, E, k) >= 1 else 0
    slots = on * 4 * T * k
    opts = Routing(_SCORES.get(score, score), n_group, topk_group, group_top, int(renormalize), scaling)
    _done(lib().nvfp4_moe_route(_op(logits, on * T * E * (4 if dt == NVFP4_F32 else 2), "logits"), dt,
                                _op(bias, on * 4 * E, "bias", _F32), _op(ids, slots, "ids", _I32),
                                _op(weights, slots, "weights", _F32), _op(offsets, on * 4 * (E + 1), "offsets", _I32),
                                _op(order, slots, "order", _I32), T, E, k, ctypes.byref(opts), pw, nw,
                                _stream_handle(stream)), "nvfp4_moe_route")


def nvfp4_gemm_experts_workspace_bytes(M: int, K: int, E: int, S: int) -> int:
    return int(lib().nvfp4_gemm_experts_workspace_bytes(M, K, E, S))


def nvfp4_gemm_experts(a, b, sfa, sfb, c, M: int, K: int, E: int, rows: int, slots_per_row: int, sf_layout, offsets,
                       order, alpha: float = 1.0, scale_a=None, scale_b=None, workspace=None,
                       workspace_bytes: int | None = None, dtype=None, stream=None) -> None:
    """Enqueue c[s][m] for every slot s of the experts' lists: the row
    s // slots_per_row of b times the weights a[e] of the slot's expert e."""
    lay, dt = layout_id(sf_layout), _dtype_id(c, dtype)
    pw, nw = _workspace(workspace, workspace_bytes)
    on = 1 if min(M, K, E, rows, slots_per_row) >= 1 else 0
    S = on * rows * slots_per_row
    _done(lib().nvfp4_gemm_experts(_op(a, on * E * M * K // 2, "a"), _op(b, on * rows * K // 2, "b"),
                                   _op(sfa, on * _scale_bytes(M, K, E, lay), "sfa"),
                                   _op(sfb, on * _scale_bytes(rows, K, 1, lay), "sfb"),
                                   _op(c, S * M * (4 if dt == NVFP4_F32 else 2), "c"), dt, M, K, E, rows,
                                   slots_per_row, lay, _op(offsets, on * 4 * (E + 1), "offsets", _I32),
                                   _op(order, 4 * S, "order", _I32), alpha, _op(scale_a, on * 4 * E, "scale_a", _F32),
                                   _op(scale_b, 4, "scale_b", _F32), pw, nw, _stream_handle(stream)),
          "nvfp4_gemm_experts")


def nvfp4_moe_combine(y, ids, weights, out, T: int, k: int, M: int, dtype=None, stream=None) -> None:
    """Enqueue out[t] = sum_j weights[t][j] * y[t * k + j] over ids[t][j] >= 0."""
    dt = _dtype_id(y, dtype)
    if dt != _dtype_id(out, dtype):
        raise ValueError("y and out have different types")
    n = T * M * (4 if dt == NVFP4_F32 else 2) if min(T, k, M) >= 1 else 0
    slots = 4 * T * k if n else 0
    _done(lib().nvfp4_moe_combine(_op(y, k * n, "y"), dt, _op(ids, slots, "ids", _I32),
                                  _op(weights, slots, "weights", _F32), _op(out, n, "out"), T, k, M,
                                  _stream_handle(stream)), "nvfp4_moe_combine")


# ---------------------------------------------------------------- attention over a paged cache

_LAYOUTS = {"half": NVFP4_ROPE_HALF, "interleaved": NVFP4_ROPE_INTERLEAVED}
_METHODS = {"unscaled": NVFP4_ROPE_UNSCALED, "linear": NVFP4_ROPE_LINEAR, "base": NVFP4_ROPE_BASE,
            "bands": NVFP4_ROPE_BANDS, "ramp": NVFP4_ROPE_RAMP}
# What a call costs on the host is as long as a small kernel: types are compared as
# objects here, not as text (0.4 us each), and each tensor is asked once for what is needed.
_torch = None


class _Torch:
    """torch's types and device query, looked up once (torch is imported with the first call)."""

    def __init__(self):
        import torch
        self.kinds = {torch.float16: NVFP4_F16, torch.bfloat16: NVFP4_BF16, torch.float32: NVFP4_F32}
        self.f32, self.f64, self.i32, self.i64, self.u8 = (torch.float32, torch.float64, torch.int32, torch.int64,
                                                           torch.uint8)
        self.current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _types() -> _Torch:
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _kind(x, dtype, t):
    """nvfp4_dtype_t of a tensor (or of ``dtype``, needed for raw pointers)."""
    if dtype is None and x is not None and not isinstance(x, int):
        kind = t.kinds.get(x.dtype)
        if kind is not None:
            return kind
    return _dtype_id(x, dtype)


def _here(x, name, t):
    """Kernels are launched on the current device: a tensor of another is refused."""
    device = x.get_device()
    if device < 0:
        raise ValueError("operands must be device tensors")
    if device != t.current_device():
        raise ValueError(f"{name} is on {x.device}, not on the current device")


def _at(x, need, name, dtype, t):
    """Device pointer of a dense tensor of type ``dtype`` that holds at least ``need`` bytes;
    raw pointers and None pass."""
    if x is None or isinstance(x, int):
        return x
    _here(x, name, t)
    if not x.is_contiguous():
        raise ValueError("operands must be contiguous")
    if x.dtype is not dtype and dtype is not None:
        raise ValueError(f"{name} is {x.dtype}, not {str(dtype).replace('torch.', '')}")
    if x.nbytes < need:
        raise ValueError(f"{name} holds {x.nbytes} bytes, the shape needs {need}")
    return x.data_ptr()


def _rows(x, name, dt, T, H, D, token_stride, head_stride, t):
    """Pointer of a [T][H][D] tensor of type ``dt`` and its strides in elements (dense
    by default), checked against what its memory holds behind its first element."""
    given = token_stride is not None or head_stride is not None
    if head_stride is None:
        head_stride = D
    if token_stride is None:
        token_stride = H * head_stride
    if x is None or isinstance(x, int):
        return x, token_stride, head_stride
    _here(x, name, t)
    if t.kinds.get(x.dtype) != dt:
        raise ValueError(f"{name} is {x.dtype}, not of the call's type")
    if not given:
        if not x.is_contiguous():
            raise ValueError(f"{name} is not contiguous: give its strides")
        held = x.numel()
    else:
        if x.dim() and x.stride(-1) != 1 and x.shape[-1] > 1:
            raise ValueError(f"rows of {name} are not contiguous")
        held = x.untyped_storage().nbytes() // x.element_size() - x.storage_offset()
    if T >= 1 and H >= 1 and D >= 1 and token_stride >= 0 and head_stride >= 0:
        need = (T - 1) * token_stride + (H - 1) * head_stride + D
        if held < need:
            raise ValueError(f"{name} holds {held} elements, the shape needs {need}")
    return x.data_ptr(), token_stride, head_stride


def nvfp4_rope_frequencies(R: int, base: float, method="unscaled", factor: float = 1.0, length: float = 0.0,
                           low: float = 0.0, high: float = 0.0) -> list:
    """The R / 2 frequencies of the pairs, as a list of floats (float64 on the device for nvfp4_rope)."""
    f = (ctypes.c_double * max(1, R // 2))()
    opts = RopeScaling(_METHODS.get(method, method), factor, length, low, high)
    _done(lib().nvfp4_rope_frequencies(f, R, base, ctypes.byref(opts)), "nvfp4_rope_frequencies")
    return list(f)


def nvfp4_rope(x, out, positions, frequencies, T: int, H: int, D: int, R: int, layout="half", factor: float = 1.0,
               transpose: bool = False, token_stride: int | None = None, head_stride: int | None = None,
               out_token_stride: int | None = None, out_head_stride: int | None = None, dtype=None, stream=None) -> None:
    """Enqueue out = x [T][H][D] with the pairs of each head's first R values turned by
    positions[t] * frequencies[j] (``transpose``: back, the gradient). Strides in
    elements, dense by default; out may be x (with x's strides then)."""
    t = _torch or _types()
    dt = _kind(x, dtype, t)
    px, ts, hs = _rows(x, "x", dt, T, H, D, token_stride, head_stride, t)
    if out is x and out_token_stride is None and out_head_stride is None:
        out_token_stride, out_head_stride = ts, hs
    po, ots, ohs = _rows(out, "out", dt, T, H, D, out_token_stride, out_head_stride, t)
    # (the library reports shape errors itself: a negative size needs nothing here)
    _done(lib().nvfp4_rope(px, dt, po, _at(positions, 8 * T, "positions", t.i64, t),
                           _at(frequencies, 4 * R, "frequencies", t.f64, t), T, H, D, R, ts, hs, ots, ohs,
                           _LAYOUTS.get(layout, layout), factor, int(transpose), _stream_handle(stream)), "nvfp4_rope")


class Nvfp4Cache:
    """nvfp4_cache_t of device tensors (which it keeps alive): codes uint8 [pages][heads][page_size]
    [head_size / 2] and scales uint8 [..][head_size / 16] of keys and of values, k_scale and v_scale
    float32 on the device (None: 1). Page strides in bytes, dense by default; with them the tensors
    may be views whose pages are dense."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, pages: int, page_size: int, heads: int, head_size: int,
                 k_scale=None, v_scale=None, code_page_stride: int | None = None, scale_page_stride: int | None = None):
        self.pages, self.page_size, self.heads, self.head_size = pages, page_size, heads, head_size
        self.tensors = (k_codes, k_scales, v_codes, v_scales, k_scale, v_scale)
        row = heads * page_size
        strides, pointers = [], []
        for given, each in ((code_page_stride, row * head_size // 2), (scale_page_stride, row * head_size // 16)):
            strides.append(each if given is None else given)
        t = _types()
        for name, x, stride, given, each in (
                ("k_codes", k_codes, strides[0], code_page_stride, row * head_size // 2),
                ("k_scales", k_scales, strides[1], scale_page_stride, row * head_size // 16),
                ("v_codes", v_codes, strides[0], code_page_stride, row * head_size // 2),
                ("v_scales", v_scales, strides[1], scale_page_stride, row * head_size // 16)):
            if given is None or x is None or isinstance(x, int):
                pointers.append(_at(x, max(0, pages * each), name, t.u8, t))
                continue
            _here(x, name, t)
            if x.dtype is not t.u8:
                raise ValueError(f"{name} is {x.dtype}, not uint8")
            need, held = (pages - 1) * stride + each, x.untyped_storage().nbytes() - x.storage_offset()
            if min(pages, stride) >= 1 and held < need:
                raise ValueError(f"{name} holds {held} bytes, the shape needs {need}")
            pointers.append(x.data_ptr())
        self.struct = CacheStruct(*pointers, _at(k_scale, 4, "k_scale", t.f32, t), _at(v_scale, 4, "v_scale", t.f32, t),
                                  pages, page_size, heads, head_size, *strides)
        self._ref = ctypes.byref(self.struct)


_DENSE = (None, None)


def nvfp4_cache_write(cache, k, v, slots, T: int, k_strides=None, v_strides=None, dtype=None, stream=None) -> None:
    """Enqueue the quantisation of k, v [T][heads][head_size] (strides: (token, head) in elements,
    dense by default) into the cache's rows ``slots`` (int64 [T]; outside the cache: not written)."""
    t = _torch or _types()
    dt, H, D = _kind(k, dtype, t), cache.heads, cache.head_size
    pk, kt, kh = _rows(k, "k", dt, T, H, D, *(k_strides or _DENSE), t)
    pv, vt, vh = _rows(v, "v", dt, T, H, D, *(v_strides or _DENSE), t)
    _done(lib().nvfp4_cache_write(cache._ref, pk, pv, dt, _at(slots, 8 * T, "slots", t.i64, t), T, kt, kh, vt, vh,
                                  _stream_handle(stream)), "nvfp4_cache_write")


def nvfp4_cache_read(cache, k, v, slots, T: int, dtype=None, stream=None) -> None:
    """Enqueue k, v [T][heads][head_size] = the values of the cache's rows ``slots`` (int64 [T];
    outside the cache: zeros)."""
    t = _torch or _types()
    dt, H, D = _kind(k, dtype, t), cache.heads, cache.head_size
    pk, _, _ = _rows(k, "k", dt, T, H, D, None, None, t)
    pv, _, _ = _rows(v, "v", dt, T, H, D, None, None, t)
    _done(lib().nvfp4_cache_read(cache._ref, pk, pv, dt, _at(slots, 8 * T, "slots", t.i64, t), T,
                                 _stream_handle(stream)), "nvfp4_cache_read")


def nvfp4_cache_attention_workspace_bytes(cache, dtype, T: int, H: int, B: int, max_q: int, max_length: int,
                                          window: int = 0) -> int:
    """Bytes of a workspace for such a call (0: none needed, or a call that is refused); ``dtype`` as q's."""
    opts = Attention(0, 0, max_q, max_length, window, 1.0, 1)
    return int(lib().nvfp4_cache_attention_workspace_bytes(cache._ref, _dtype_id(None, dtype), T, H, B,
                                                           ctypes.byref(opts)))


def nvfp4_cache_attention(cache, q, out, offsets, lengths, table, T: int, H: int, B: int, max_q: int, max_length: int,
                          scale: float | None = None, causal: bool = True, window: int = 0, lse=None, workspace=None,
                          workspace_bytes: int | None = None, token_stride: int | None = None,
                          head_stride: int | None = None, table_width: int | None = None, dtype=None,
                          stream=None) -> None:
    """Enqueue the attention of q [T][H][head_size] (strides in elements, dense by default): rows
    offsets[b] .. offsets[b + 1] are the last of the lengths[b] positions of sequence b, which are in
    the pages table[b] (int32 [B][table_width]; its last dimension by default). scale None:
    head_size ** -0.5; lse: float32 [T][H]; a (zero-initialised) workspace of
    nvfp4_cache_attention_workspace_bytes or of NVFP4_WORKSPACE_MAX_BYTES."""
    t = _torch or _types()
    D, dt = cache.head_size, _kind(q, dtype, t)
    pq, ts, hs = _rows(q, "q", dt, T, H, D, token_stride, head_stride, t)
    po, _, _ = _rows(out, "out", dt, T, H, D, None, None, t)
    if table_width is None:
        if isinstance(table, int) or table is None:
            raise ValueError("raw pointers need table_width=")
        table_width = table.shape[-1]
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or isinstance(workspace, int) else workspace.nbytes
    elif workspace_bytes < 0:
        raise ValueError(f"workspace_bytes is {workspace_bytes}")
    opts = Attention(ts, hs, max_q, max_length, window, max(D, 1) ** -0.5 if scale is None else scale, causal)
    # (the library reports shape errors itself: a negative size needs nothing here)
    _done(lib().nvfp4_cache_attention(cache._ref, pq, dt, po, _at(lse, 4 * T * H, "lse", t.f32, t),
                                      _at(offsets, 4 * (B + 1), "offsets", t.i32, t), _at(lengths, 4 * B, "lengths", t.i32, t),
                                      _at(table, 4 * B * table_width, "table", t.i32, t), T, H, B, table_width,
                                      ctypes.byref(opts), _at(workspace, workspace_bytes, "workspace", None, t),
                                      workspace_bytes, _stream_handle(stream)), "nvfp4_cache_attention")


def nvfp4_status_string(status: int) -> str:
    return status_string(status)


def nvfp4_last_hip_error() -> int:
    return int(lib().nvfp4_last_hip_error())
