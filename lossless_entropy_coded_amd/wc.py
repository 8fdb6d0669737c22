"""Thin ctypes binding of libwc (include/wc.h).

Argument marshalling only: every step of encoding, planning and decoding runs
in the native library (host C++ and gfx950 HIP kernels).  Importing this
module loads ``libwc.so`` from this package directory and fails loudly if it
has not been built (``python -m lossless_entropy_coded_amd.build``); there is
no Python or CPU fallback for any entry point.

PyTorch is used only as the owner of device memory and streams: callers pass
tensors (or raw integer device pointers) and the binding forwards
``data_ptr()`` and ``torch.cuda.current_stream().cuda_stream``.

The C entry points receive bare pointers without sizes, so before forwarding
a tensor the binding checks what the kernels will touch: the tensor must be a
CUDA tensor on the plan's device, contiguous, and at least as large as the
bytes the call reads or writes.  A failed check raises ``WCError`` with
``WC_ERR_INVALID_ARG`` and nothing is launched.  Raw integer pointers are
forwarded unchecked (the C side checks their alignment only).
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libwc.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libwc.so is not built at {LIB_PATH}; run `python -m lossless_entropy_coded_amd.build`")

_lib = ctypes.CDLL(LIB_PATH)

_u8p = ctypes.POINTER(ctypes.c_uint8)
_u16p = ctypes.POINTER(ctypes.c_uint16)
_u64p = ctypes.POINTER(ctypes.c_uint64)
_u32p = ctypes.POINTER(ctypes.c_uint32)


class EncodeOpts(ctypes.Structure):
    _fields_ = [("max_code_len", ctypes.c_uint32), ("chunk_bytes", ctypes.c_uint32),
                ("chunks_per_group", ctypes.c_uint32), ("n_threads", ctypes.c_uint32),
                ("group_align", ctypes.c_uint32), ("group_max_elems", ctypes.c_uint32),
                ("layout", ctypes.c_uint32), ("seg_max_bits", ctypes.c_uint32), ("coder", ctypes.c_uint32),
                ("gap_bits", ctypes.c_uint32)]


_lib.wc_encode_host.argtypes = [ctypes.POINTER(_u16p), _u64p, ctypes.c_uint32, ctypes.POINTER(EncodeOpts),
                                ctypes.POINTER(_u8p), _u64p]
_lib.wc_encode_host.restype = ctypes.c_int
_lib.wc_encode_u8_host.argtypes = [ctypes.POINTER(_u8p), _u64p, ctypes.c_uint32, ctypes.POINTER(EncodeOpts),
                                   ctypes.POINTER(_u8p), _u64p]
_lib.wc_encode_u8_host.restype = ctypes.c_int
_lib.wc_free_host.argtypes = [_u8p]
_lib.wc_free_host.restype = None
_lib.wc_plan.argtypes = [_u8p, ctypes.c_uint64, ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)]
_lib.wc_plan.restype = ctypes.c_int
_lib.wc_plan_info.argtypes = [ctypes.c_void_p, _u64p, _u32p, _u64p, _u64p]
_lib.wc_plan_info.restype = ctypes.c_int
_lib.wc_plan_stats.argtypes = [ctypes.c_void_p, _u64p, _u64p, _u64p, _u32p, _u32p, _u32p, _u32p]
_lib.wc_plan_stats.restype = ctypes.c_int
_lib.wc_decode_async.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
_lib.wc_decode_async.restype = ctypes.c_int
_lib.wc_decode_u8_async.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
_lib.wc_decode_u8_async.restype = ctypes.c_int
_lib.wc_plan_format.argtypes = [ctypes.c_void_p, _u32p, _u32p, _u32p]
_lib.wc_plan_format.restype = ctypes.c_int
_lib.wc_plan_decode_shape.argtypes = [ctypes.c_void_p, _u32p, _u32p, _u32p]
_lib.wc_plan_decode_shape.restype = ctypes.c_int
_lib.wc_gemv_bf16_async.argtypes = [ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p]
_lib.wc_gemv_bf16_async.restype = ctypes.c_int


class GemvOperand(ctypes.Structure):
    _fields_ = [("tensor", ctypes.c_uint32), ("cols", ctypes.c_uint32), ("x", ctypes.c_void_p),
                ("y", ctypes.c_void_p)]


_lib.wc_decode_gemv_work_bytes.argtypes = [ctypes.c_void_p, ctypes.POINTER(GemvOperand), ctypes.c_uint32, _u64p]
_lib.wc_decode_gemv_work_bytes.restype = ctypes.c_int
_lib.wc_decode_gemv_async.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(GemvOperand),
                                      ctypes.c_uint32, ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]
_lib.wc_decode_gemv_async.restype = ctypes.c_int
_lib.wc_decode_gemv_noalloc_async.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(GemvOperand),
                                              ctypes.c_uint32, ctypes.c_void_p]
_lib.wc_decode_gemv_noalloc_async.restype = ctypes.c_int


class _Q4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("rows", ctypes.c_uint32), ("cols", ctypes.c_uint32), ("group", ctypes.c_uint32)]


class _Fp8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_uint32),
                ("cols", ctypes.c_uint32)]


class _Grad(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_uint64),
                ("kind", ctypes.c_uint32)]


_void_p, _u32, _u64, _int, _float = (ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int, ctypes.c_float)
for _name, _args in {
        "wc_q4_check": [_void_p],
        "wc_gemv_q4_async": [_void_p, _void_p, _u32, _void_p, _void_p],
        "wc_embed_async": [_void_p, _u32, _u32, _void_p, _u32, _u64, _float, _void_p, _void_p],
        "wc_embed_q4_async": [_void_p, _void_p, _u32, _u64, _float, _void_p, _void_p],
        "wc_embed_grad_work_bytes": [_u64, _u32, _u64p],
        "wc_embed_grad_async": [_void_p, _void_p, _u32, _u64, _float, _void_p, _u32, _u32, _u32, _int, _void_p, _u64,
                                _void_p],
        "wc_ce_work_bytes": [_u64, _u32, _u32, _int, _u64p],
        "wc_ce_loss_async": [_void_p, _void_p, _void_p, _u32, _u64, _u32, _u32, _void_p, _void_p, _void_p, _u64,
                             _void_p],
        "wc_ce_grad_async": [_void_p, _void_p, _void_p, _u32, _u64, _u32, _u32, _void_p, _void_p, _void_p, _void_p,
                             _void_p, _u64, _void_p],
        "wc_quant_fp8_async": [_void_p, _u64, _u32, _int, _void_p, _void_p, _void_p],
        "wc_rms_norm_async": [_void_p, _void_p, _void_p, _u64, _u32, _float, _void_p, _void_p, _void_p, _void_p, _void_p,
                              _void_p],
        "wc_rms_norm_grad_work_bytes": [_u64, _u32, _u64p],
        "wc_rms_norm_grad_async": [_void_p, _void_p, _void_p, _void_p, _void_p, _u64, _u32, _void_p, _void_p, _int,
                                   _void_p, _u64, _void_p],
        "wc_fp8_check": [_void_p],
        "wc_gemm_fp8_work_bytes": [_void_p, _u64, _u64p],
        "wc_gemm_fp8_async": [_void_p, _void_p, _void_p, _u64, _void_p, _u32, _void_p, _u64, _void_p],
        "wc_clip_grads_work_bytes": [_void_p, _u32, _u64p],
        "wc_clip_grads_async": [_void_p, _u32, _float, _void_p, _void_p, _u64, _void_p]}.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = ctypes.c_int
_lib.wc_stream_reference_async.argtypes = [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_uint64,
                                           ctypes.c_void_p]
_lib.wc_stream_reference_async.restype = ctypes.c_int
_lib.wc_plan_debug_status.argtypes = [ctypes.c_void_p, _u32p, ctypes.c_int]
_lib.wc_plan_debug_status.restype = ctypes.c_int
_lib.wc_plan_destroy.argtypes = [ctypes.c_void_p]
_lib.wc_plan_destroy.restype = None
_lib.wc_status_str.argtypes = [ctypes.c_int]
_lib.wc_status_str.restype = ctypes.c_char_p

# status codes (include/wc.h)
WC_OK = 0
WC_ERR_INVALID_ARG = -1
WC_ERR_NOMEM = -2
WC_ERR_HIP = -3
WC_ERR_UNSUPPORTED = -4
WC_ERR_SCRATCH = -5
# the no-allocation fused product's static work array (include/wc.h)
NOALLOC_SCRATCH_BYTES = 8 << 20
WC_ERR_BAD_MAGIC = -10
WC_ERR_TRUNCATED = -11
WC_ERR_SECTION_BOUNDS = -12
WC_ERR_CODE_LENGTHS = -13
WC_ERR_KRAFT = -14
WC_ERR_GAP = -15
WC_ERR_GROUP_START = -16
WC_ERR_STREAM_BITS = -17
WC_ERR_TENSOR_TABLE = -18
# bits of a debug plan's status word (plans made with WC_DEBUG=1)
WC_DEBUG_GROUP_COUNT = 1
WC_DEBUG_LANE_BITS = 2

# Group table defaults (wc_encode_opts): G = chunks per group, what one wave64
# decodes in one pass (two 64-bit chunks per lane; wider groups take several
# passes); A = elements per block, so that every group's output starts on a
# 256-byte boundary; M = elements per group at most (eight 8-element merge
# steps per lane).  The writer takes any G, A a positive multiple of 8 and
# M <= 4096, the range the GPU decoder takes.
GROUP_CHUNKS = 128
GROUP_ALIGN = 128
GROUP_MAX_ELEMS = 4096
# Interleaved-lane layout (container v3): stream bits per segment at most; the
# GPU decoder stages a segment's stream (at most 1984 bytes) in LDS.
SEG_MAX_BITS = 15872
LAYOUTS = {"lanes": 0, "chunks": 1}
# Entropy coders of the interleaved-lane layout: canonical Huffman, or rANS
# (12-bit frequencies, 32-bit state, 16-bit words; lanes layout only).
CODERS = {"huffman": 0, "rans": 1}

EXPORTED = ("wc_encode_host", "wc_encode_u8_host", "wc_free_host", "wc_plan", "wc_plan_info", "wc_plan_stats",
            "wc_plan_format", "wc_plan_decode_shape", "wc_decode_u8_async",
            "wc_decode_async", "wc_gemv_bf16_async", "wc_decode_gemv_work_bytes", "wc_decode_gemv_async",
            "wc_decode_gemv_noalloc_async", "wc_stream_reference_async", "wc_plan_debug_status",
            "wc_q4_check", "wc_gemv_q4_async", "wc_embed_async", "wc_embed_q4_async", "wc_embed_grad_work_bytes",
            "wc_embed_grad_async", "wc_ce_work_bytes", "wc_ce_loss_async", "wc_ce_grad_async",
            "wc_quant_fp8_async", "wc_rms_norm_async", "wc_rms_norm_grad_work_bytes", "wc_rms_norm_grad_async",
            "wc_fp8_check", "wc_gemm_fp8_work_bytes", "wc_gemm_fp8_async", "wc_clip_grads_work_bytes",
            "wc_clip_grads_async",
            "wc_plan_destroy", "wc_status_str")


class WCError(RuntimeError):
    def __init__(self, status: int, call: str, detail: str = ""):
        self.status = status
        super().__init__(f"{call} failed: {status_str(status)} ({status})" + (f": {detail}" if detail else ""))


def status_str(status: int) -> str:
    return _lib.wc_status_str(int(status)).decode()


def _check(status: int, call: str):
    if status != WC_OK:
        raise WCError(status, call)


def _as_u16(t) -> np.ndarray:
    if hasattr(t, "numpy"):                    # torch CPU tensor (bf16/int16/uint16)
        import torch
        t = t.detach()
        if t.dtype == torch.bfloat16:
            t = t.view(torch.int16)
        t = t.contiguous().numpy()
    a = np.ascontiguousarray(t).reshape(-1)
    if a.dtype != np.uint16:
        a = a.view(np.uint16)
    return a


def encode_host(tensors, max_code_len: int = 24, chunks_per_group: int = GROUP_CHUNKS,
                n_threads: int = 0, group_align: int = GROUP_ALIGN,
                group_max_elems: int = GROUP_MAX_ELEMS, layout: str = "lanes",
                seg_max_bits: int = SEG_MAX_BITS, coder: str = "huffman", gap_bits: int = 8) -> np.ndarray:
    """wc_encode_host over a list of bf16 tensors (numpy uint16 or torch CPU).

    layout: "lanes" (the default: container v3, interleaved lanes;
    seg_max_bits caps a segment's stream bits) or "chunks" (container v2,
    per-chunk gaps; chunks_per_group applies).  coder: "huffman" or "rans"
    (lanes only; max_code_len is then ignored).  gap_bits: 8, or 5 for packed
    gaps (chunks only).
    Returns the container as a numpy uint8 array (a copy of the library buffer)."""
    arrs = [_as_u16(t) for t in tensors]
    nt = len(arrs)
    ptrs = (_u16p * max(nt, 1))(*[a.ctypes.data_as(_u16p) for a in arrs])
    numels = (ctypes.c_uint64 * max(nt, 1))(*[a.size for a in arrs])
    opts = EncodeOpts(max_code_len, 8, chunks_per_group, n_threads, group_align, group_max_elems,
                      LAYOUTS[layout], seg_max_bits, CODERS[coder], gap_bits)
    out = _u8p()
    nbytes = ctypes.c_uint64(0)
    _check(_lib.wc_encode_host(ptrs, numels, nt, ctypes.byref(opts), ctypes.byref(out), ctypes.byref(nbytes)),
           "wc_encode_host")
    try:
        blob = np.empty(nbytes.value, np.uint8)
        ctypes.memmove(blob.ctypes.data, out, nbytes.value)
    finally:
        _lib.wc_free_host(out)
    return blob


def encode_u8_host(tensors, max_code_len: int = 0, n_threads: int = 0, group_align: int = GROUP_ALIGN,
                   group_max_elems: int = GROUP_MAX_ELEMS, seg_max_bits: int = SEG_MAX_BITS,
                   coder: str = "huffman") -> np.ndarray:
    """wc_encode_u8_host over a list of uint8 code planes (numpy or torch CPU): a u8-kind
    interleaved-lane container (each byte one symbol, no raw plane), Huffman or rANS.
    max_code_len 0 selects the library's default for code planes (11 bits)."""
    arrs = [np.ascontiguousarray(t.numpy() if hasattr(t, "numpy") else t).reshape(-1).view(np.uint8)
            for t in tensors]
    nt = len(arrs)
    ptrs = (_u8p * max(nt, 1))(*[a.ctypes.data_as(_u8p) for a in arrs])
    numels = (ctypes.c_uint64 * max(nt, 1))(*[a.size for a in arrs])
    opts = EncodeOpts(max_code_len, 8, 0, n_threads, group_align, group_max_elems, LAYOUTS["lanes"], seg_max_bits,
                      CODERS[coder])
    out = _u8p()
    nbytes = ctypes.c_uint64(0)
    _check(_lib.wc_encode_u8_host(ptrs, numels, nt, ctypes.byref(opts), ctypes.byref(out), ctypes.byref(nbytes)),
           "wc_encode_u8_host")
    try:
        blob = np.empty(nbytes.value, np.uint8)
        ctypes.memmove(blob.ctypes.data, out, nbytes.value)
    finally:
        _lib.wc_free_host(out)
    return blob


class Plan:
    """wc_plan over a host container; owns the native plan until close()."""

    def __init__(self, blob_host: np.ndarray, device: int = 0):
        self._blob = np.ascontiguousarray(blob_host, dtype=np.uint8)
        h = ctypes.c_void_p()
        _check(_lib.wc_plan(self._blob.ctypes.data_as(_u8p), self._blob.size, int(device), ctypes.byref(h)),
               "wc_plan")
        self._h = h
        self.device = int(device)
        n = ctypes.c_uint64(0)
        nt = ctypes.c_uint32(0)
        _check(_lib.wc_plan_info(self._h, ctypes.byref(n), ctypes.byref(nt), None, None), "wc_plan_info")
        offs = (ctypes.c_uint64 * max(nt.value, 1))()
        nums = (ctypes.c_uint64 * max(nt.value, 1))()
        _check(_lib.wc_plan_info(self._h, None, None, offs, nums), "wc_plan_info")
        self.n_elems = n.value
        self.n_tensors = nt.value
        self.container_bytes = self.stats()["container_bytes"]
        self.tensor_offsets = [offs[i] for i in range(nt.value)]
        self.tensor_numels = [nums[i] for i in range(nt.value)]

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("plan is closed")
        return self._h

    def format(self):
        """wc_plan_format: (container version, element kind: 0 bf16, 1 u8, coder: 0 Huffman, 1 rANS)."""
        v, k, c = ctypes.c_uint32(), ctypes.c_uint32(), ctypes.c_uint32()
        _check(_lib.wc_plan_format(self.handle, ctypes.byref(v), ctypes.byref(k), ctypes.byref(c)),
               "wc_plan_format")
        return v.value, k.value, c.value

    def decode_shape(self) -> dict:
        """wc_plan_decode_shape: waves per workgroup, grid and launches per call of the decode entry point."""
        w, g, n = ctypes.c_uint32(), ctypes.c_uint32(), ctypes.c_uint32()
        _check(_lib.wc_plan_decode_shape(self.handle, ctypes.byref(w), ctypes.byref(g), ctypes.byref(n)),
               "wc_plan_decode_shape")
        return {"waves_per_group": w.value, "grid": g.value, "launches": n.value}

    def stats(self) -> dict:
        cb, sb, ng = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_uint64()
        kc, kd, gr, lds = ctypes.c_uint32(), ctypes.c_uint32(), ctypes.c_uint32(), ctypes.c_uint32()
        _check(_lib.wc_plan_stats(self.handle, ctypes.byref(cb), ctypes.byref(sb), ctypes.byref(ng),
                                  ctypes.byref(kc), ctypes.byref(kd), ctypes.byref(gr), ctypes.byref(lds)),
               "wc_plan_stats")
        return {"container_bytes": cb.value, "stream_bits": sb.value, "n_groups": ng.value,
                "count_bits": kc.value, "decode_bits": kd.value, "grid": gr.value, "lds_bytes": lds.value}

    def close(self):
        if self._h is not None:
            _lib.wc_plan_destroy(self._h)
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def plan_debug_status(plan: Plan, reset: bool = False) -> int:
    """wc_plan_debug_status: the status word of a plan made with WC_DEBUG=1 in
    the environment (0: no invariant failed; WC_DEBUG_GROUP_COUNT: a group of
    the chunks layout decoded a codeword count other than its element count;
    WC_DEBUG_LANE_BITS: a lane of the lanes layout's decode or fused product
    did not end its string where the next lane's begins).  Waits for the
    plan's device; reset clears the word after reading it."""
    word = ctypes.c_uint32(0)
    _check(_lib.wc_plan_debug_status(plan.handle, ctypes.byref(word), 1 if reset else 0), "wc_plan_debug_status")
    return word.value


def _ptr(x) -> int:
    return int(x.data_ptr()) if hasattr(x, "data_ptr") else int(x)


def _require(t, nbytes: int, device, what: str, call: str) -> None:
    """Check a tensor argument before its pointer goes to C: a CUDA tensor on
    `device` (None: any), contiguous, holding at least `nbytes` bytes.  Raw
    integer pointers are not checked."""
    if not hasattr(t, "data_ptr"):
        return
    problem = None
    if not getattr(t, "is_cuda", False):
        problem = "is not a CUDA tensor"
    elif device is not None and t.device.index is not None and t.device.index != device:
        problem = f"is on cuda:{t.device.index}, not on cuda:{device}"
    elif not t.is_contiguous():
        problem = "is not contiguous"
    elif t.numel() * t.element_size() < nbytes:
        problem = f"holds {t.numel() * t.element_size()} bytes, fewer than the {nbytes} the call touches"
    if problem:
        raise WCError(WC_ERR_INVALID_ARG, call, f"{what} {problem}")


def decode_async(plan: Plan, blob_dev, out_dev, stream=None) -> None:
    """wc_decode_async: one launch decoding the whole container into out_dev.

    blob_dev / out_dev: torch device tensors (or raw device pointers).  stream:
    a torch.cuda.Stream, a raw hipStream_t integer, or None for torch's current
    stream."""
    _require(blob_dev, plan.container_bytes, plan.device, "blob_dev", "wc_decode_async")
    _require(out_dev, 2 * plan.n_elems, plan.device, "out_dev", "wc_decode_async")
    _check(_lib.wc_decode_async(plan.handle, ctypes.c_void_p(_ptr(blob_dev)), ctypes.c_void_p(_ptr(out_dev)),
                                ctypes.c_void_p(_stream_handle(stream))), "wc_decode_async")


def decode_u8_async(plan: Plan, blob_dev, out_dev, stream=None) -> None:
    """wc_decode_u8_async: one launch decoding a u8-kind container into out_dev (n bytes)."""
    _require(blob_dev, plan.container_bytes, plan.device, "blob_dev", "wc_decode_u8_async")
    _require(out_dev, plan.n_elems, plan.device, "out_dev", "wc_decode_u8_async")
    _check(_lib.wc_decode_u8_async(plan.handle, ctypes.c_void_p(_ptr(blob_dev)), ctypes.c_void_p(_ptr(out_dev)),
                                   ctypes.c_void_p(_stream_handle(stream))), "wc_decode_u8_async")


_lookups_found = None   # what _lookups returns, once torch has a device in use


def _lookups():
    """(current device, handle of its current stream), two functions, once torch has a device in use (None before).
    A Stream object costs 3 us, much of a call of a token, so the handle itself is asked for where torch has it."""
    global _lookups_found
    if _lookups_found is None:
        import torch
        if not torch.cuda.is_initialized():
            return None
        device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _lookups_found = device, (lambda: raw_stream(device())) if raw_stream else _current_stream
    return _lookups_found


def _current_stream() -> int:
    import torch
    return int(torch.cuda.current_stream().cuda_stream)


def _stream_handle(stream) -> int:
    if stream is None:
        found = _lookups_found or _lookups()
        return found[1]() if found else _current_stream()
    if hasattr(stream, "cuda_stream"):
        return int(stream.cuda_stream)
    return int(stream)


def gemv_bf16_async(W_dev, rows: int, cols: int, x_dev, y_dev, stream=None) -> None:
    """wc_gemv_bf16_async: y = W x (bf16 W rows x cols row-major, bf16 x, fp32 y), one launch.

    W_dev / x_dev / y_dev: torch device tensors (or raw device pointers)."""
    if rows > 0:
        dev = _current_device()
        _require(W_dev, 2 * int(rows) * int(cols), dev, "W", "wc_gemv_bf16_async")
        _require(x_dev, 2 * int(cols), dev, "x", "wc_gemv_bf16_async")
        _require(y_dev, 4 * int(rows), dev, "y", "wc_gemv_bf16_async")
    _check(_lib.wc_gemv_bf16_async(ctypes.c_void_p(_ptr(W_dev)), int(rows), int(cols), ctypes.c_void_p(_ptr(x_dev)),
                                   ctypes.c_void_p(_ptr(y_dev)), ctypes.c_void_p(_stream_handle(stream))),
           "wc_gemv_bf16_async")


def stream_reference_async(src_dev, src_bytes: int, dst_dev, dst_bytes: int, stream=None) -> None:
    """wc_stream_reference_async: the streaming yardstick (reads src_bytes once,
    writes dst_bytes; 16-byte output item j = NOT input item
    min(floor(j r / 2^32), ns - 1), r = ceil(ns 2^32 / nd)), one launch."""
    if src_bytes or dst_bytes:
        dev = _current_device()
        _require(src_dev, int(src_bytes), dev, "src", "wc_stream_reference_async")
        _require(dst_dev, int(dst_bytes), dev, "dst", "wc_stream_reference_async")
    _check(_lib.wc_stream_reference_async(ctypes.c_void_p(_ptr(src_dev)), int(src_bytes), ctypes.c_void_p(_ptr(dst_dev)),
                                          int(dst_bytes), ctypes.c_void_p(_stream_handle(stream))),
           "wc_stream_reference_async")


def _current_device():
    found = _lookups_found or _lookups()
    if found:
        return found[0]()
    import torch
    return torch.cuda.current_device() if torch.cuda.is_available() else None


def _require_operands(plan: Plan, ops, call: str) -> None:
    """x and y of every operand over a non-empty tensor: cols bf16 and
    numel / cols float32 (bad tensor indexes and shapes are left to C)."""
    for i, (t, c, x, y) in enumerate(ops):
        t, c = int(t), int(c)
        if not (0 <= t < plan.n_tensors) or c <= 0 or plan.tensor_numels[t] == 0:
            continue
        _require(x, 2 * c, plan.device, f"ops[{i}].x", call)
        _require(y, 4 * (plan.tensor_numels[t] // c), plan.device, f"ops[{i}].y", call)


def _operands(ops):
    """(tensor, cols, x, y) tuples -> a ctypes array of wc_gemv_operand (x, y: device tensors or pointers)."""
    arr = (GemvOperand * max(len(ops), 1))()
    for i, (t, c, x, y) in enumerate(ops):
        arr[i] = GemvOperand(int(t), int(c), _ptr(x) if x is not None else 0, _ptr(y) if y is not None else 0)
    return arr


def decode_gemv_work_bytes(plan: Plan, ops) -> int:
    """wc_decode_gemv_work_bytes for operands [(tensor, cols, x, y), ...]."""
    _require_operands(plan, ops, "wc_decode_gemv_work_bytes")
    n = ctypes.c_uint64(0)
    _check(_lib.wc_decode_gemv_work_bytes(plan.handle, _operands(ops), len(ops), ctypes.byref(n)),
           "wc_decode_gemv_work_bytes")
    return n.value


def decode_gemv_async(plan: Plan, blob_dev, ops, work_dev, work_bytes: int, stream=None) -> None:
    """wc_decode_gemv_async: y = W x for each operand (tensor, cols, x, y) -- consecutive tensors of the
    container, decoded on chip and never written out -- in one decode launch and one row-sum launch.
    work_dev: device scratch of work_bytes >= decode_gemv_work_bytes(plan, ops), 256-byte aligned."""
    _require(blob_dev, plan.container_bytes, plan.device, "blob_dev", "wc_decode_gemv_async")
    _require_operands(plan, ops, "wc_decode_gemv_async")
    _require(work_dev, int(work_bytes), plan.device, "work_dev", "wc_decode_gemv_async")
    _check(_lib.wc_decode_gemv_async(plan.handle, ctypes.c_void_p(_ptr(blob_dev)), _operands(ops), len(ops),
                                     ctypes.c_void_p(_ptr(work_dev)), int(work_bytes),
                                     ctypes.c_void_p(_stream_handle(stream))),
           "wc_decode_gemv_async")


def decode_gemv_noalloc_async(plan: Plan, blob_dev, ops, stream=None) -> None:
    """wc_decode_gemv_noalloc_async: decode_gemv_async with the library's static device work
    array (NOALLOC_SCRATCH_BYTES) instead of a caller's buffer; allocates nothing.  Calls that
    overlap on one GPU race on that array."""
    _require(blob_dev, plan.container_bytes, plan.device, "blob_dev", "wc_decode_gemv_noalloc_async")
    _require_operands(plan, ops, "wc_decode_gemv_noalloc_async")
    _check(_lib.wc_decode_gemv_noalloc_async(plan.handle, ctypes.c_void_p(_ptr(blob_dev)), _operands(ops), len(ops),
                                             ctypes.c_void_p(_stream_handle(stream))),
           "wc_decode_gemv_noalloc_async")


# ---- operators on decoded tensors ------------------------------------------------

# limits (include/wc.h)
MAX_VOCAB = 1 << 22
MAX_DIM = 1 << 16
MAX_TOKENS = 1 << 20
MAX_LOGITS = 1 << 38   # tokens times vocabulary of one cross entropy call
GEMV_Q4_MAX_VECS = 16
OUT_KINDS = {"f32": 0, "bf16": 1}


_KINDS = {}   # dtype -> "bf16", "f32", "words" (whole numbers) or its own name, of the types seen


def _kind_of(dtype) -> str:
    kind = _KINDS.get(dtype)
    if kind is None:
        name = str(dtype).rsplit(".", 1)[-1]
        kind = _KINDS[dtype] = {"bfloat16": "bf16", "float32": "f32"}.get(
            name, "words" if name.startswith(("int", "uint", "bool")) else name)
    return kind


def _bytes_ok(t, nbytes: int, device, what: str, call: str, kind: str = "") -> int:
    """The device pointer of a tensor that _require accepts (or of a raw integer pointer).  kind: the floating type
    that the call reads or writes ("bf16", "f32"), or "words" for whole numbers alone; a tensor of whole numbers is
    taken as the words that it holds in any case.  Empty: any type."""
    try:   # what every call of a good tensor takes, without a further look
        found = _KINDS[t.dtype]
        if ((found == kind or found == "words" or not kind) and t.is_cuda and t.get_device() == device and
                t.nbytes >= nbytes and t.is_contiguous()):
            return t.data_ptr()
    except (AttributeError, KeyError):
        pass
    if kind and hasattr(t, "dtype"):
        found = _kind_of(t.dtype)
        if found != kind and found != "words":
            raise WCError(WC_ERR_INVALID_ARG, call, f"{what} is {t.dtype}, where {kind} is read or written")
    _require(t, nbytes, device, what, call)
    return _ptr(t)


def _sizes(call: str, **sizes) -> None:
    """Sizes must be whole numbers that the C types hold; C checks the rest."""
    for what, v in sizes.items():
        if not 0 <= v <= 0xFFFFFFFF:
            raise WCError(WC_ERR_INVALID_ARG, call, f"{what} is {v}")


def _workspace(work_dev, work_bytes: int, device, call: str):
    """The pointer and the size of a workspace; a size that C's 64 bits do not hold would arrive there as another."""
    size = int(work_bytes)
    if not 0 <= size < 1 << 64:
        raise WCError(WC_ERR_INVALID_ARG, call, f"work_bytes is {size}")
    return _bytes_ok(work_dev, size, device, "work", call), size


_INDEX_BYTES = {}   # dtype -> bytes, of the id types seen


def _index_bytes(ids, what: str, call: str) -> int:
    """4 for int32 ids, 8 for int64 ids (raw pointers are taken as int64)."""
    if not hasattr(ids, "dtype"):
        return 8
    width = _INDEX_BYTES.get(ids.dtype)
    if width is None:
        name = str(ids.dtype)
        if name not in ("torch.int32", "torch.int64"):
            raise WCError(WC_ERR_INVALID_ARG, call, f"{what} is {name}, not int32 or int64")
        width = _INDEX_BYTES[ids.dtype] = 4 if name == "torch.int32" else 8
    return width


class Q4Matrix:
    """A wc_q4_matrix over device tensors (kept alive by this handle): 4-bit codes, two per byte and the first in
    the low nibble (an int4 plane as decode_u8_async leaves it), bf16 scales and optional uint8 zero points
    (8 without them), rows x ceil(cols / group) each."""

    def __init__(self, codes, scales, rows: int, cols: int, group: int, zeros=None):
        _sizes("wc_q4_check", rows=rows, cols=cols, group=group)
        self.rows, self.cols, self.group = int(rows), int(cols), int(group)
        self._tensors = (codes, scales, zeros)
        self.device = _current_device()
        n = self.rows * -(-self.cols // max(self.group, 1))
        c = _bytes_ok(codes, self.rows * self.cols // 2, self.device, "codes", "wc_q4_check", "words")
        s = _bytes_ok(scales, 2 * n, self.device, "scales", "wc_q4_check", "bf16")
        z = _bytes_ok(zeros, n, self.device, "zeros", "wc_q4_check", "words") if zeros is not None else 0
        self._struct = _Q4(c, s, z, self.rows, self.cols, self.group)
        self._ref = ctypes.addressof(self._struct)
        _check(_lib.wc_q4_check(self._ref), "wc_q4_check")


def _on_device(W: Q4Matrix, call: str):
    dev = _current_device()
    if W.device != dev:
        raise WCError(WC_ERR_INVALID_ARG, call, f"the matrix is on cuda:{W.device}, not on cuda:{dev}")
    return dev


def gemv_q4_async(W: Q4Matrix, x_dev, n_vecs: int, y_dev, stream=None) -> None:
    """wc_gemv_q4_async: y[t] = W x[t] for n_vecs (at most GEMV_Q4_MAX_VECS) bf16 vectors, fp32 y, one launch.

    x_dev: n_vecs x cols bf16; y_dev: n_vecs x rows float32."""
    call = "wc_gemv_q4_async"
    dev = _on_device(W, call)
    if n_vecs >> 32:
        _sizes(call, n_vecs=n_vecs)
    x = _bytes_ok(x_dev, 2 * n_vecs * W.cols, dev, "x", call, "bf16")
    y = _bytes_ok(y_dev, 4 * n_vecs * W.rows, dev, "y", call, "f32")
    _check(_lib.wc_gemv_q4_async(W._ref, x, n_vecs, y, _stream_handle(stream)), call)


def embed_async(table_dev, vocab: int, dim: int, ids_dev, n: int, out_dev, scale: float = 1.0, stream=None) -> None:
    """wc_embed_async: out[t] = scale * table[ids[t]] (bf16), zero where ids[t] is outside [0, vocab); one launch."""
    call = "wc_embed_async"
    dev = _current_device()
    if (vocab | dim | n) >> 32:
        _sizes(call, vocab=vocab, dim=dim, n=n)
    width = _index_bytes(ids_dev, "ids", call)
    table = _bytes_ok(table_dev, 2 * vocab * dim, dev, "table", call, "bf16")
    ids = _bytes_ok(ids_dev, width * n, dev, "ids", call)
    out = _bytes_ok(out_dev, 2 * n * dim, dev, "out", call, "bf16")
    _check(_lib.wc_embed_async(table, vocab, dim, ids, width, n, scale, out, _stream_handle(stream)), call)


def embed_q4_async(W: Q4Matrix, ids_dev, n: int, out_dev, scale: float = 1.0, stream=None) -> None:
    """wc_embed_q4_async: embed_async from a 4-bit table of W.rows entries."""
    call = "wc_embed_q4_async"
    dev = _on_device(W, call)
    if n >> 32:
        _sizes(call, n=n)
    width = _index_bytes(ids_dev, "ids", call)
    ids = _bytes_ok(ids_dev, width * n, dev, "ids", call)
    out = _bytes_ok(out_dev, 2 * n * W.cols, dev, "out", call, "bf16")
    _check(_lib.wc_embed_q4_async(W._ref, ids, width, n, scale, out, _stream_handle(stream)), call)


def embed_grad_work_bytes(n: int, dim: int) -> int:
    """wc_embed_grad_work_bytes: device scratch of embed_grad_async for n tokens."""
    _sizes("wc_embed_grad_work_bytes", n=n, dim=dim)
    b = ctypes.c_uint64(0)
    _check(_lib.wc_embed_grad_work_bytes(n, dim, ctypes.byref(b)), "wc_embed_grad_work_bytes")
    return b.value


def embed_grad_async(dout_dev, ids_dev, n: int, dtable_dev, vocab: int, dim: int, work_dev, work_bytes: int,
                     out: str = "f32", scale: float = 1.0, accumulate: bool = False, stream=None) -> None:
    """wc_embed_grad_async: dtable[v] = scale * sum of dout[t] over the t with ids[t] = v, in fp32 and a fixed order.

    out: "f32" or "bf16", dtable's type.  accumulate: add to dtable instead of writing every row."""
    call = "wc_embed_grad_async"
    dev = _current_device()
    if (vocab | dim | n) >> 32:
        _sizes(call, n=n, vocab=vocab, dim=dim)
    if out not in OUT_KINDS:
        raise WCError(WC_ERR_INVALID_ARG, call, f"out is {out!r}, not one of {sorted(OUT_KINDS)}")
    width = _index_bytes(ids_dev, "ids", call)
    dout = _bytes_ok(dout_dev, 2 * n * dim, dev, "dout", call, "bf16")
    ids = _bytes_ok(ids_dev, width * n, dev, "ids", call)
    dtable = _bytes_ok(dtable_dev, (4 if out == "f32" else 2) * vocab * dim, dev, "dtable", call, out)
    work, work_bytes = _workspace(work_dev, work_bytes, dev, call)
    _check(_lib.wc_embed_grad_async(dout, ids, width, n, scale, dtable, OUT_KINDS[out], vocab, dim, bool(accumulate),
                                    work, work_bytes, _stream_handle(stream)), call)


def ce_work_bytes(tokens: int, vocab: int, dim: int, grad: bool = True) -> int:
    """wc_ce_work_bytes: device scratch of ce_loss_async (grad False) or of both ce_loss_async and ce_grad_async."""
    _sizes("wc_ce_work_bytes", tokens=tokens, vocab=vocab, dim=dim)
    b = ctypes.c_uint64(0)
    _check(_lib.wc_ce_work_bytes(tokens, vocab, dim, bool(grad), ctypes.byref(b)), "wc_ce_work_bytes")
    return b.value


def ce_loss_async(h_dev, W_dev, targets_dev, tokens: int, vocab: int, dim: int, loss_dev, lse_dev, work_dev,
                  work_bytes: int, stream=None) -> None:
    """wc_ce_loss_async: loss[t] = lse[t] - z[t][target[t]], lse[t] = log sum exp z[t] for z = h W^T (bf16 h, W)."""
    call = "wc_ce_loss_async"
    dev = _current_device()
    if (tokens | vocab | dim) >> 32:
        _sizes(call, tokens=tokens, vocab=vocab, dim=dim)
    width = _index_bytes(targets_dev, "targets", call)
    h = _bytes_ok(h_dev, 2 * tokens * dim, dev, "h", call, "bf16")
    W = _bytes_ok(W_dev, 2 * vocab * dim, dev, "W", call, "bf16")
    targets = _bytes_ok(targets_dev, width * tokens, dev, "targets", call)
    loss = _bytes_ok(loss_dev, 4 * tokens, dev, "loss", call, "f32")
    lse = _bytes_ok(lse_dev, 4 * tokens, dev, "lse", call, "f32")
    work, work_bytes = _workspace(work_dev, work_bytes, dev, call)
    _check(_lib.wc_ce_loss_async(h, W, targets, width, tokens, vocab, dim, loss, lse, work, work_bytes,
                                 _stream_handle(stream)), call)


def ce_grad_async(h_dev, W_dev, targets_dev, tokens: int, vocab: int, dim: int, lse_dev, dloss_dev, dh_dev, dW_dev,
                  work_dev, work_bytes: int, stream=None) -> None:
    """wc_ce_grad_async: dh and dW (bf16; either may be None) of sum dloss[t] * loss[t], with ce_loss_async's lse."""
    call = "wc_ce_grad_async"
    dev = _current_device()
    if (tokens | vocab | dim) >> 32:
        _sizes(call, tokens=tokens, vocab=vocab, dim=dim)
    width = _index_bytes(targets_dev, "targets", call)
    h = _bytes_ok(h_dev, 2 * tokens * dim, dev, "h", call, "bf16")
    W = _bytes_ok(W_dev, 2 * vocab * dim, dev, "W", call, "bf16")
    targets = _bytes_ok(targets_dev, width * tokens, dev, "targets", call)
    lse = _bytes_ok(lse_dev, 4 * tokens, dev, "lse", call, "f32")
    dloss = _bytes_ok(dloss_dev, 4 * tokens, dev, "dloss", call, "f32")
    dh = _bytes_ok(dh_dev, 2 * tokens * dim, dev, "dh", call, "bf16") if dh_dev is not None else 0
    dW = _bytes_ok(dW_dev, 2 * vocab * dim, dev, "dW", call, "bf16") if dW_dev is not None else 0
    work, work_bytes = _workspace(work_dev, work_bytes, dev, call)
    _check(_lib.wc_ce_grad_async(h, W, targets, width, tokens, vocab, dim, lse, dloss, dh, dW, work, work_bytes,
                                 _stream_handle(stream)), call)


# ---- 8-bit floating point, norms and gradients -------------------------------------

FP8_BLOCK = 128   # columns (and rows of a matrix) that share a scale
MAX_GRADS = 1 << 20
MAX_GRAD_NUMEL = 1 << 34
_CODE_KIND = "float8_e4m3fn"


def quant_fp8_async(x_dev, n: int, dim: int, codes_dev, scales_dev, gated: bool = False, stream=None) -> None:
    """wc_quant_fp8_async: rows of bf16 activations (gated: silu(gate) * up of rows gate, up) to e4m3 codes with an
    fp32 scale per FP8_BLOCK columns; one launch.

    x_dev: n x dim bf16 (gated: n x 2 dim); codes_dev: n x dim float8_e4m3fn (or bytes); scales_dev: n x
    ceil(dim / FP8_BLOCK) float32."""
    call = "wc_quant_fp8_async"
    dev = _current_device()
    if (n | dim) >> 32:
        _sizes(call, n=n, dim=dim)
    gated = bool(gated)
    x = _bytes_ok(x_dev, (4 if gated else 2) * n * dim, dev, "x", call, "bf16")
    codes = _bytes_ok(codes_dev, n * dim, dev, "codes", call, _CODE_KIND)
    scales = _bytes_ok(scales_dev, 4 * n * -(-dim // FP8_BLOCK), dev, "scales", call, "f32")
    _check(_lib.wc_quant_fp8_async(x, n, dim, gated, codes, scales, _stream_handle(stream)), call)


def rms_norm_async(x_dev, weight_dev, n: int, dim: int, eps: float, y_dev=None, codes_dev=None, scales_dev=None,
                   residual_dev=None, sum_dev=None, rstd_dev=None, stream=None) -> None:
    """wc_rms_norm_async: y = h * rstd * weight, rstd = 1 / sqrt(mean(h^2) + eps), of h = x or h = bf16(x + residual),
    which goes to sum_dev; one launch.

    y goes to y_dev (bf16), to codes_dev and scales_dev (as quant_fp8_async writes them), or to both; rstd_dev (n
    float32), if given, keeps rstd for the gradient.  sum_dev may be x_dev or residual_dev, and y_dev may be x_dev, but
    not both the same tensor."""
    call = "wc_rms_norm_async"
    dev = _current_device()
    if y_dev is not None and y_dev is sum_dev:
        raise WCError(WC_ERR_INVALID_ARG, call, "y and sum are the same tensor")
    if (n | dim) >> 32:
        _sizes(call, n=n, dim=dim)
    wide = 2 * n * dim
    x = _bytes_ok(x_dev, wide, dev, "x", call, "bf16")
    weight = _bytes_ok(weight_dev, 2 * dim, dev, "weight", call, "bf16")
    residual = _bytes_ok(residual_dev, wide, dev, "residual", call, "bf16") if residual_dev is not None else 0
    total = _bytes_ok(sum_dev, wide, dev, "sum", call, "bf16") if sum_dev is not None else 0
    y = _bytes_ok(y_dev, wide, dev, "y", call, "bf16") if y_dev is not None else 0
    codes = _bytes_ok(codes_dev, n * dim, dev, "codes", call, _CODE_KIND) if codes_dev is not None else 0
    scales = (_bytes_ok(scales_dev, 4 * n * -(-dim // FP8_BLOCK), dev, "scales", call, "f32")
              if scales_dev is not None else 0)
    rstd = _bytes_ok(rstd_dev, 4 * n, dev, "rstd", call, "f32") if rstd_dev is not None else 0
    _check(_lib.wc_rms_norm_async(x, residual, weight, n, dim, eps, total, y, codes, scales, rstd,
                                  _stream_handle(stream)), call)


def rms_norm_grad_work_bytes(n: int, dim: int) -> int:
    """wc_rms_norm_grad_work_bytes: device scratch of rms_norm_grad_async for n tokens."""
    _sizes("wc_rms_norm_grad_work_bytes", n=n, dim=dim)
    b = ctypes.c_uint64(0)
    _check(_lib.wc_rms_norm_grad_work_bytes(n, dim, ctypes.byref(b)), "wc_rms_norm_grad_work_bytes")
    return b.value


def rms_norm_grad_async(dy_dev, h_dev, weight_dev, rstd_dev, n: int, dim: int, dh_dev, dweight_dev, work_dev,
                        work_bytes: int, dsum_dev=None, accumulate: bool = False, stream=None) -> None:
    """wc_rms_norm_grad_async: dh (bf16, of x and the residual alike) and dweight (float32) of rms_norm_async's y; either
    may be None.

    h_dev: what rms_norm_async wrote to sum_dev (x without a residual); dsum_dev: the gradient that h has from where
    else it goes, or None.  accumulate: add to dweight instead of writing it."""
    call = "wc_rms_norm_grad_async"
    dev = _current_device()
    if (n | dim) >> 32:
        _sizes(call, n=n, dim=dim)
    wide = 2 * n * dim
    dy = _bytes_ok(dy_dev, wide, dev, "dy", call, "bf16")
    h = _bytes_ok(h_dev, wide, dev, "h", call, "bf16")
    weight = _bytes_ok(weight_dev, 2 * dim, dev, "weight", call, "bf16")
    rstd = _bytes_ok(rstd_dev, 4 * n, dev, "rstd", call, "f32")
    dsum = _bytes_ok(dsum_dev, wide, dev, "dsum", call, "bf16") if dsum_dev is not None else 0
    dh = _bytes_ok(dh_dev, wide, dev, "dh", call, "bf16") if dh_dev is not None else 0
    dweight = _bytes_ok(dweight_dev, 4 * dim, dev, "dweight", call, "f32") if dweight_dev is not None else 0
    work, work_bytes = _scratch(work_dev, work_bytes, dev, call)
    _check(_lib.wc_rms_norm_grad_async(dy, h, weight, rstd, dsum, n, dim, dh, dweight, bool(accumulate), work,
                                       work_bytes, _stream_handle(stream)), call)


def _scratch(work_dev, work_bytes: int, device, call: str):
    """_workspace of a call that may need none: (0, 0) where none is given."""
    if work_dev is None:
        if work_bytes:
            raise WCError(WC_ERR_INVALID_ARG, call, f"work is None, work_bytes {work_bytes}")
        return 0, 0
    return _workspace(work_dev, work_bytes, device, call)


class Fp8Matrix:
    """A wc_fp8_matrix over device tensors (kept alive by this handle): rows x cols e4m3 codes (float8_e4m3fn, or bytes as
    decode_u8_async leaves a plane of them) and a float32 scale per block of FP8_BLOCK x FP8_BLOCK."""

    def __init__(self, codes, scales, rows: int, cols: int):
        call = "wc_fp8_check"
        _sizes(call, rows=rows, cols=cols)
        self.rows, self.cols = int(rows), int(cols)
        self._tensors = (codes, scales)
        self.device = _current_device()
        c = _bytes_ok(codes, self.rows * self.cols, self.device, "codes", call, _CODE_KIND)
        s = _bytes_ok(scales, 4 * -(-self.rows // FP8_BLOCK) * -(-self.cols // FP8_BLOCK), self.device, "scales", call,
                      "f32")
        self._struct = _Fp8(c, s, self.rows, self.cols)
        self._ref = ctypes.addressof(self._struct)
        _check(_lib.wc_fp8_check(self._ref), call)


def gemm_fp8_work_bytes(W: Fp8Matrix, tokens: int) -> int:
    """wc_gemm_fp8_work_bytes: device scratch of gemm_fp8_async for this many tokens."""
    _sizes("wc_gemm_fp8_work_bytes", tokens=tokens)
    b = ctypes.c_uint64(0)
    _check(_lib.wc_gemm_fp8_work_bytes(W._ref, tokens, ctypes.byref(b)), "wc_gemm_fp8_work_bytes")
    return b.value


def gemm_fp8_async(W: Fp8Matrix, x_codes_dev, x_scales_dev, tokens: int, y_dev, work_dev, work_bytes: int,
                   out: str = "bf16", stream=None) -> None:
    """wc_gemm_fp8_async: y[t] = W x[t] for e4m3 activations with a float32 scale per token and FP8_BLOCK columns.

    x_codes_dev, x_scales_dev: as quant_fp8_async or rms_norm_async writes them; y_dev: tokens x W.rows of `out` ("f32"
    or "bf16"); work_dev may be None where gemm_fp8_work_bytes is 0."""
    call = "wc_gemm_fp8_async"
    dev = _on_device(W, call)
    if tokens >> 32:
        _sizes(call, tokens=tokens)
    if out not in OUT_KINDS:
        raise WCError(WC_ERR_INVALID_ARG, call, f"out is {out!r}, not one of {sorted(OUT_KINDS)}")
    x = _bytes_ok(x_codes_dev, tokens * W.cols, dev, "x_codes", call, _CODE_KIND)
    xs = _bytes_ok(x_scales_dev, 4 * tokens * -(-W.cols // FP8_BLOCK), dev, "x_scales", call, "f32")
    y = _bytes_ok(y_dev, (4 if out == "f32" else 2) * tokens * W.rows, dev, "y", call, out)
    work, work_bytes = _scratch(work_dev, work_bytes, dev, call)
    _check(_lib.wc_gemm_fp8_async(W._ref, x, xs, tokens, y, OUT_KINDS[out], work, work_bytes, _stream_handle(stream)),
           call)


class GradList:
    """A list of gradients for clip_grads_async (kept alive by this handle): float32 or bf16 device tensors, and where the
    clipped ones go (outs: tensors of the same sizes and types, any of them the gradient itself; None: all in place).
    No output may overlap another tensor of the list.

    Each tensor's type, device, size and place is looked at here and no more in the calls: about 2 us per tensor (291 of
    them 0.54 ms).  Keep the handle while the tensors stay where they are."""

    def __init__(self, grads, outs=None):
        call = "wc_clip_grads_async"
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if len(outs) != len(grads) or len(grads) > MAX_GRADS:
            raise WCError(WC_ERR_INVALID_ARG, call, f"{len(grads)} gradients and {len(outs)} outputs")
        self.device = _current_device()
        self._tensors = (grads, outs)
        self._array = (_Grad * max(len(grads), 1))()
        self._n = len(grads)
        spans = []   # what is read and written: (begin, end, writes, index)
        for i, (g, out) in enumerate(zip(grads, outs)):
            kind = _kind_of(g.dtype)
            if kind not in OUT_KINDS or _kind_of(out.dtype) != kind:
                raise WCError(WC_ERR_INVALID_ARG, call, f"gradient {i} is {g.dtype}, its output {out.dtype}")
            n = g.numel()
            if out.numel() != n:
                raise WCError(WC_ERR_INVALID_ARG, call, f"gradient {i} has {n} elements, its output {out.numel()}")
            size = (4 if kind == "f32" else 2) * n
            self._array[i] = _Grad(_bytes_ok(g, size, self.device, f"gradient {i}", call),
                                   _bytes_ok(out, size, self.device, f"output {i}", call), n, OUT_KINDS[kind])
            if n:
                read, write = self._array[i].g, self._array[i].out
                spans.append((write, write + size, True, i))
                if read != write:
                    spans.append((read, read + size, False, i))
        # an element that is written must be no other's: workgroups read and write in no order
        written = seen = 0
        for begin, end, writes, i in sorted(spans):
            if begin < (seen if writes else written):
                raise WCError(WC_ERR_INVALID_ARG, call, f"gradient {i} overlaps another one's output")
            seen = max(seen, end)
            written = max(written, end) if writes else written


def clip_grads_work_bytes(grads: GradList) -> int:
    """wc_clip_grads_work_bytes: device scratch of clip_grads_async for this list."""
    b = ctypes.c_uint64(0)
    _check(_lib.wc_clip_grads_work_bytes(ctypes.addressof(grads._array), grads._n, ctypes.byref(b)),
           "wc_clip_grads_work_bytes")
    return b.value


def clip_grads_async(grads: GradList, max_norm: float, norm_dev, work_dev, work_bytes: int, stream=None) -> None:
    """wc_clip_grads_async: norm = sqrt(sum of g^2 over all gradients); out = g * max_norm / norm where the norm is finite
    and larger than max_norm, else g.

    norm_dev: one float32; max_norm: at least 0 (infinity: the norm alone)."""
    call = "wc_clip_grads_async"
    dev = _current_device()
    if grads.device != dev:
        raise WCError(WC_ERR_INVALID_ARG, call, f"the gradients are on cuda:{grads.device}, not on cuda:{dev}")
    norm = _bytes_ok(norm_dev, 4, dev, "norm", call, "f32")
    work, work_bytes = _scratch(work_dev, work_bytes, dev, call)
    _check(_lib.wc_clip_grads_async(ctypes.addressof(grads._array), grads._n, max_norm, norm, work, work_bytes,
                                    _stream_handle(stream)), call)


def exported_symbols():
    """Names of the C ABI entry points resolvable in the loaded library."""
    return [name for name in EXPORTED if hasattr(_lib, name)]
