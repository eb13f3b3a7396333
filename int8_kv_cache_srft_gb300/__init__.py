"""int8_kv_cache_srft_gb300 -- Python binding of libsrftkv (GB300, sm_103a).

A thin ctypes layer over the C ABI in ``include/srftkv.h``: it turns torch
tensors into device pointers and the current torch stream into a
cudaStream_t, calls the entry point of the same name and raises on a
non-zero return.  All arithmetic happens in the library's CUDA kernels;
there is no CPU or PyTorch fallback, and importing this package fails
loudly when the library has not been built (``python -m
int8_kv_cache_srft_gb300.build``).
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsrftkv.so")

SRFTKV_OK = 0
SRFTKV_ERR_INVALID = -1
SRFTKV_ERR_CUDA = -2
SRFTKV_ERR_DEVICE = -3


class SrftKvError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} returned {code}: {msg}")
        self.code = code


class _Side(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("lambda_", ctypes.c_void_p),
        ("lambda_outer_stride", ctypes.c_int64),
        ("bits", ctypes.c_int),
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("transform", ctypes.c_int),
        ("scale_format", ctypes.c_int),
    ]


class _Pages(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("lambda_", ctypes.c_void_p),
                ("n_pages", ctypes.c_int), ("H", ctypes.c_int), ("page_size", ctypes.c_int), ("d", ctypes.c_int),
                ("group", ctypes.c_int), ("bits", ctypes.c_int), ("transform", ctypes.c_int),
                ("scale_format", ctypes.c_int)]


class _PagedBatch(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("B", ctypes.c_int), ("max_pages", ctypes.c_int), ("total_q", ctypes.c_int), ("max_q", ctypes.c_int),
                ("max_seq_len", ctypes.c_int)]


TRANSFORMS = {"srft": 0, "srht": 1}  # SRFTKV_TRANSFORM_SRFT / _SRHT in include/srftkv.h
SCALE_FORMATS = {"fp32": 0, "fp16": 1, "e8m0": 2}  # SRFTKV_SCALE_FP32 / _FP16 / _E8M0
DTYPES = {torch.float16: 0, torch.bfloat16: 1}  # SRFTKV_DTYPE_FP16 / _BF16 (rows of the paged calls)
SCALE_DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "e8m0": torch.uint8}


_lib = None


def library() -> ctypes.CDLL:
    """Load libsrftkv.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m int8_kv_cache_srft_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    i, u64, vp, sz = ctypes.c_int, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_size_t
    sp = ctypes.POINTER(_Side)
    lib.srft_kv_quantize.argtypes = [sp, sp, i, i, i, i, i, i, i, u64, vp]
    lib.srft_kv_dequantize.argtypes = [sp, sp, i, i, i, i, i, i, i, u64, vp]
    lib.q4kv_decode_attention.argtypes = [vp, vp, sp, sp, i, i, i, i, i, i, vp, ctypes.c_float, u64, i, vp, sz, vp]
    lib.q4kv_decode_attention_static.argtypes = [vp, vp, sp, sp, i, i, i, i, i, i, vp, ctypes.c_float, u64, i, vp]
    lib.q4kv_decode_attention_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.q4kv_decode_attention_workspace_size.restype = sz
    lib.srft_kv_vector_bytes.argtypes = [i, i, i, i, ctypes.POINTER(sz), ctypes.POINTER(sz)]
    lib.srft_transform.argtypes = [vp, vp, i, i, u64, i, vp]
    lib.srht_transform.argtypes = [vp, vp, i, i, u64, i, vp]
    pp, bp, i64, f32 = ctypes.POINTER(_Pages), ctypes.POINTER(_PagedBatch), ctypes.c_int64, ctypes.c_float
    lib.srft_kv_quantize_paged.argtypes = [pp, vp, i64, pp, vp, i64, vp, i, i, u64, vp]
    lib.srft_kv_dequantize_paged.argtypes = [pp, vp, i64, pp, vp, i64, vp, i, i, u64, vp]
    lib.q4kv_paged_attention.argtypes = [vp, i64, vp, i64, i, i, pp, pp, bp, f32, i, u64, vp, sz, vp]
    lib.q4kv_paged_attention_workspace_size.argtypes = [pp, i, bp, i]
    lib.q4kv_paged_attention_workspace_size.restype = sz
    lib.srftkv_last_error.restype = ctypes.c_char_p
    lib.srftkv_device_fault.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    lib.srftkv_set_attention_poll_limit_for_testing.argtypes = [i]
    lib.srftkv_set_codec_poll_limit_for_testing.argtypes = [i]
    for name in ("srft_kv_quantize", "srft_kv_dequantize", "q4kv_decode_attention", "q4kv_decode_attention_static",
                 "srft_kv_quantize_paged", "srft_kv_dequantize_paged", "q4kv_paged_attention",
                 "srft_kv_vector_bytes", "srft_transform", "srht_transform", "srftkv_device_fault",
                 "srftkv_set_attention_poll_limit_for_testing", "srftkv_set_codec_poll_limit_for_testing"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _check(fn: str, rc: int) -> None:
    if rc != SRFTKV_OK:
        raise SrftKvError(fn, rc, library().srftkv_last_error().decode())


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:  # torch's current stream on the current device
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


@dataclass
class Side:
    """One side (K or V) of a packed cache: the code plane, the scale plane,
    an optional per-channel lambda and, for the codec calls, the fp16 rows."""

    codes: torch.Tensor            # uint8 [n_outer][H][t_cap][d*bits/8] (or fp16 [B][Hkv][t_cap][d] for bits 16)
    scales: torch.Tensor | None    # [n_outer][H][t_cap][d/group]: fp32, fp16 or uint8 (e8m0) per scale_format
    bits: int
    x: torch.Tensor | None = None  # fp16 [n_outer][n_tokens][H][d]
    lam: torch.Tensor | None = None  # fp32 [n_lam][H][d]; n_lam == 1 broadcasts
    lam_outer_stride: int | None = None
    transform: str = "srft"        # "srft" or "srht"
    scale_format: str = "fp32"     # "fp32", "fp16" or "e8m0"

    # The marshalled struct is built once and reused until a field is assigned again (a tensor changed in
    # place keeps its address; one resized or replaced must be assigned anew).
    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_c":
            object.__setattr__(self, "_c", None)

    def c_pointer(self):
        c = getattr(self, "_c", None)
        if c is None:
            c = ctypes.pointer(self.to_c())
            object.__setattr__(self, "_c", c)
        return c

    def to_c(self) -> _Side:
        stride = self.lam_outer_stride
        if stride is None:
            stride = 0 if self.lam is None or self.lam.shape[0] == 1 else self.lam.shape[1] * self.lam.shape[2]
        return _Side(_ptr(self.x), _ptr(self.lam), stride, self.bits, _ptr(self.codes), _ptr(self.scales),
                     TRANSFORMS[self.transform], SCALE_FORMATS[self.scale_format])


def alloc_side(n_outer: int, t_cap: int, H: int, d: int, bits: int, group: int, device="cuda",
               transform: str = "srft", scale_format: str = "fp32") -> Side:
    """Allocate empty (head-major) code and scale planes for one side."""
    if bits == 16:
        return Side(torch.empty((n_outer, H, t_cap, d), dtype=torch.float16, device=device), None, 16)
    codes = torch.empty((n_outer, H, t_cap, d * bits // 8), dtype=torch.uint8, device=device)
    scales = torch.empty((n_outer, H, t_cap, d // group), dtype=SCALE_DTYPES[scale_format], device=device)
    return Side(codes, scales, bits, transform=transform, scale_format=scale_format)


def _sidep(s: Side | None):
    return None if s is None else s.c_pointer()


def srft_kv_quantize(k: Side | None, v: Side | None, n_outer: int, n_tokens: int, H: int, d: int, group: int,
                     t_cap: int, t_offset: int, sign_seed: int, stream=None) -> None:
    rc = library().srft_kv_quantize(_sidep(k), _sidep(v), n_outer, n_tokens, H, d, group, t_cap, t_offset,
                                    sign_seed, _stream(stream))
    _check("srft_kv_quantize", rc)


def srft_kv_dequantize(k: Side | None, v: Side | None, n_outer: int, n_tokens: int, H: int, d: int, group: int,
                       t_cap: int, t_offset: int, sign_seed: int, stream=None) -> None:
    rc = library().srft_kv_dequantize(_sidep(k), _sidep(v), n_outer, n_tokens, H, d, group, t_cap, t_offset,
                                      sign_seed, _stream(stream))
    _check("srft_kv_dequantize", rc)


def q4kv_decode_attention_workspace_size(B: int, Hq: int, Hkv: int, d: int, t_cap: int, n_splits: int = 0) -> int:
    return int(library().q4kv_decode_attention_workspace_size(B, Hq, Hkv, d, t_cap, n_splits))


def q4kv_decode_attention(q: torch.Tensor, out: torch.Tensor, k: Side, v: Side, B: int, Hq: int, Hkv: int, d: int,
                          group: int, t_cap: int, seq_lens: torch.Tensor | None, sm_scale: float, sign_seed: int,
                          n_splits: int, workspace: torch.Tensor, stream=None) -> None:
    rc = library().q4kv_decode_attention(_ptr(q), _ptr(out), _sidep(k), _sidep(v), B, Hq, Hkv, d, group, t_cap,
                                         _ptr(seq_lens), sm_scale, sign_seed, n_splits, _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream))
    _check("q4kv_decode_attention", rc)


STATIC_SCRATCH_BYTES = 16 << 20  # SRFTKV_STATIC_SCRATCH_BYTES in include/srftkv.h


def q4kv_decode_attention_static(q: torch.Tensor, out: torch.Tensor, k: Side, v: Side, B: int, Hq: int, Hkv: int,
                                 d: int, group: int, t_cap: int, seq_lens: torch.Tensor | None, sm_scale: float,
                                 sign_seed: int, n_splits: int, stream=None) -> None:
    """Decode attention without a caller workspace, for callers that cannot allocate device memory: the
    library's own fixed-size device array is the scratch (see include/srftkv.h for its size and the rules on
    overlapping calls)."""
    rc = library().q4kv_decode_attention_static(_ptr(q), _ptr(out), _sidep(k), _sidep(v), B, Hq, Hkv, d, group,
                                                t_cap, _ptr(seq_lens), sm_scale, sign_seed, n_splits,
                                                _stream(stream))
    _check("q4kv_decode_attention_static", rc)


# ---------------------------------------------------------------------------
# The paged cache
# ---------------------------------------------------------------------------
def _invalid(fn: str, msg: str):
    raise SrftKvError(fn, SRFTKV_ERR_INVALID, msg)


@dataclass
class Pages:
    """One side (K or V) of a layer's page pool; the sizes come from the tensors' shapes."""

    codes: torch.Tensor              # uint8 [n_pages][H][page_size][d*bits/8]
    scales: torch.Tensor             # [n_pages][H][page_size][d/group]: fp32, fp16 or uint8 (e8m0) per scale_format
    bits: int
    d: int
    group: int
    lam: torch.Tensor | None = None  # fp32 [H][d]
    transform: str = "srft"          # "srft" or "srht"
    scale_format: str = "fp32"       # "fp32", "fp16" or "e8m0"

    # The marshalled struct is built (and the tensors checked) once and reused until a field is assigned again (a
    # tensor changed in place keeps its address; one resized or replaced must be assigned anew).
    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_c":
            object.__setattr__(self, "_c", None)

    def c_pointer(self):
        c = getattr(self, "_c", None)
        if c is None:
            c = ctypes.pointer(self.to_c())
            object.__setattr__(self, "_c", c)
        return c

    def to_c(self) -> _Pages:
        c, s, lam = self.codes, self.scales, self.lam
        if c.dim() != 4 or c.dtype != torch.uint8 or not c.is_contiguous() or c.shape[3] * 8 != self.d * self.bits:
            _invalid("Pages", "codes must be a contiguous uint8 [n_pages][H][page_size][d*bits/8]")
        if (s.dtype != SCALE_DTYPES[self.scale_format] or not s.is_contiguous() or s.shape[:-1] != c.shape[:-1]
                or s.shape[-1] * self.group != self.d):
            _invalid("Pages", "scales must be contiguous [n_pages][H][page_size][d/group] of the scale format's type")
        if lam is not None and (lam.dtype != torch.float32 or not lam.is_contiguous()
                                or tuple(lam.shape) != (c.shape[1], self.d)):
            _invalid("Pages", "lam must be a contiguous fp32 [H][d]")
        if any(t is not None and t.device != c.device for t in (s, lam)):
            _invalid("Pages", "codes, scales and lam must be on one device")
        return _Pages(_ptr(c), _ptr(s), _ptr(lam), c.shape[0], c.shape[1], c.shape[2], self.d, self.group, self.bits,
                      TRANSFORMS[self.transform], SCALE_FORMATS[self.scale_format])


def alloc_pages(n_pages: int, page_size: int, H: int, d: int, bits: int, group: int, device="cuda",
                transform: str = "srft", scale_format: str = "fp32", lam: torch.Tensor | None = None) -> Pages:
    """Allocate the empty code and scale planes of one side of a page pool."""
    codes = torch.empty((n_pages, H, page_size, d * bits // 8), dtype=torch.uint8, device=device)
    scales = torch.empty((n_pages, H, page_size, d // group), dtype=SCALE_DTYPES[scale_format], device=device)
    return Pages(codes, scales, bits, d, group, lam, transform, scale_format)


@dataclass
class PagedBatch:
    """The sequences of an attention call (srftkv_paged_batch in include/srftkv.h).  The tensors stay where they
    are and may change in place between calls, within total_q, max_q and max_seq_len (one resized or replaced must
    be assigned anew)."""

    block_table: torch.Tensor       # int32 [B][max_pages]
    seq_lens: torch.Tensor          # int32 [B]
    cu_q: torch.Tensor | None = None  # int32 [B+1]; None: one query token a sequence
    total_q: int | None = None      # rows of q and out; None: B (with cu_q None)
    max_q: int = 1                  # upper bound of a sequence's query tokens
    max_seq_len: int = 0            # upper bound of seq_lens; 0: the block table's capacity

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_c":
            object.__setattr__(self, "_c", None)

    def c_pointer(self):
        c = getattr(self, "_c", None)
        if c is None:
            c = ctypes.pointer(self.to_c())
            object.__setattr__(self, "_c", c)
        return c

    def to_c(self) -> _PagedBatch:
        t, n, cu = self.block_table, self.seq_lens, self.cu_q
        if t.dim() != 2 or t.dtype != torch.int32 or not t.is_contiguous():
            _invalid("PagedBatch", "block_table must be a contiguous int32 [B][max_pages]")
        if n.dtype != torch.int32 or not n.is_contiguous() or tuple(n.shape) != (t.shape[0],):
            _invalid("PagedBatch", "seq_lens must be a contiguous int32 [B]")
        if cu is not None and (cu.dtype != torch.int32 or not cu.is_contiguous()
                               or tuple(cu.shape) != (t.shape[0] + 1,)):
            _invalid("PagedBatch", "cu_q must be a contiguous int32 [B+1]")
        if any(x is not None and x.device != t.device for x in (n, cu)):
            _invalid("PagedBatch", "block_table, seq_lens and cu_q must be on one device")
        if self.total_q is None and cu is not None:
            _invalid("PagedBatch", "total_q must be given with cu_q")
        total = t.shape[0] if self.total_q is None else self.total_q
        return _PagedBatch(_ptr(t), _ptr(n), _ptr(cu), t.shape[0], t.shape[1], total, self.max_q, self.max_seq_len)


def _rows_arg(fn: str, name: str, x: torch.Tensor, n: int, H: int, d: int, dtype, device) -> int:
    """The token stride of rows [n][H][d]; raises when they are not rows the library can take."""
    if x.shape != (n, H, d) or x.dtype != dtype:
        _invalid(fn, f"{name} must be [{n}][{H}][{d}] of one 16-bit type, got {tuple(x.shape)} {x.dtype}")
    s0, s1, s2 = x.stride()
    if n * H and (s2 != 1 or (s1 != d and H > 1)):
        _invalid(fn, f"{name} must have its last two dimensions dense (strides {tuple(x.stride())})")
    if n > 1 and H and s0 < H * d:  # (0, an expanded tensor's, would mean dense rows to the library)
        _invalid(fn, f"{name}'s rows must not overlap (strides {tuple(x.stride())})")
    if x.device != device:
        _invalid(fn, f"{name} must be on the pools' device")
    return s0 if n > 1 else 0


def _paged_device(fn: str, pages: Pages, stream):
    """The pools' device, which has to be the current one, and the stream of the call."""
    dev = pages.codes.device
    if dev.type != "cuda":
        if torch.cuda.is_available():
            _invalid(fn, f"the pools must be CUDA tensors, not on {dev}")
        return dev, None
    now = torch.cuda.current_device()
    if dev.index != now:
        _invalid(fn, f"the pools are on {dev}, the current device is cuda:{now}")
    return dev, _raw_stream(now) if stream is None and _raw_stream is not None else _stream(stream)


def _paged_codec(fn: str, k: Pages | None, xk, v: Pages | None, xv, slots: torch.Tensor, sign_seed: int, stream):
    side = k if k is not None else v
    if side is None:
        _invalid(fn, "at least one of k, v must be given")
    if (k is not None and xk is None) or (v is not None and xv is None):
        _invalid(fn, "each side that is given needs its rows")
    dev, stream = _paged_device(fn, side, stream)
    if slots.dtype != torch.int64 or slots.dim() != 1 or not slots.is_contiguous() or slots.device != dev:
        _invalid(fn, "slots must be a contiguous int64 [n_tokens] on the pools' device")
    n, H, dtype = slots.shape[0], side.codes.shape[1], (xk if k is not None else xv).dtype
    if dtype not in DTYPES:
        _invalid(fn, f"rows must be fp16 or bf16, got {dtype}")
    sk = _rows_arg(fn, "xk", xk, n, H, k.d, dtype, dev) if k is not None else 0
    sv = _rows_arg(fn, "xv", xv, n, v.codes.shape[1], v.d, dtype, dev) if v is not None else 0
    lib = library()
    rc = getattr(lib, fn)(k.c_pointer() if k is not None else None, xk.data_ptr() if k is not None else None, sk,
                          v.c_pointer() if v is not None else None, xv.data_ptr() if v is not None else None, sv,
                          slots.data_ptr(), n, DTYPES[dtype], sign_seed, stream)
    if rc:
        _check(fn, rc)


def srft_kv_quantize_paged(k: Pages | None, xk: torch.Tensor | None, v: Pages | None, xv: torch.Tensor | None,
                           slots: torch.Tensor, sign_seed: int, stream=None) -> None:
    """Encode rows [n_tokens][H][d] (fp16 or bf16, any token stride that is a multiple of 8) into their slots;
    a negative slot skips its token."""
    _paged_codec("srft_kv_quantize_paged", k, xk, v, xv, slots, sign_seed, stream)


def srft_kv_dequantize_paged(k: Pages | None, xk: torch.Tensor | None, v: Pages | None, xv: torch.Tensor | None,
                             slots: torch.Tensor, sign_seed: int, stream=None) -> None:
    """Decode the rows of `slots` into xk, xv; rows with a negative slot are left as they were."""
    _paged_codec("srft_kv_dequantize_paged", k, xk, v, xv, slots, sign_seed, stream)


def q4kv_paged_attention_workspace_size(k: Pages, Hq: int, batch: PagedBatch, window: int = 0) -> int:
    return int(library().q4kv_paged_attention_workspace_size(k.c_pointer(), Hq, batch.c_pointer(), window))


def q4kv_paged_attention(q: torch.Tensor, out: torch.Tensor, k: Pages, v: Pages, batch: PagedBatch, sm_scale: float,
                         window: int, sign_seed: int, workspace: torch.Tensor | None, stream=None) -> None:
    """Causal attention of the query rows q [total_q][Hq][d] over the pages; out like q (see include/srftkv.h).
    workspace: at least q4kv_paged_attention_workspace_size(...) bytes; None where that is 0."""
    fn = "q4kv_paged_attention"
    dev, stream = _paged_device(fn, k, stream)
    if q.dtype not in DTYPES or q.dim() != 3:
        _invalid(fn, f"q must be [total_q][Hq][d] of fp16 or bf16, got {tuple(q.shape)} {q.dtype}")
    b = batch.c_pointer()
    n, Hq = b.contents.total_q, q.shape[1]
    qs = _rows_arg(fn, "q", q, n, Hq, k.d, q.dtype, dev)
    os = _rows_arg(fn, "out", out, n, Hq, k.d, q.dtype, dev)
    if batch.block_table.device != dev or v.codes.device != dev or (
            workspace is not None and (workspace.device != dev or not workspace.is_contiguous())):
        _invalid(fn, "the pools, the batch's tables and the workspace must be on one device")
    rc = library().q4kv_paged_attention(q.data_ptr(), qs, out.data_ptr(), os, DTYPES[q.dtype], Hq, k.c_pointer(),
                                        v.c_pointer(), b, sm_scale, window, sign_seed, _ptr(workspace),
                                        workspace.nbytes if workspace is not None else 0, stream)
    if rc:
        _check(fn, rc)


def srft_kv_vector_bytes(d: int, bits: int, group: int, scale_format: str = "fp32") -> tuple[int, int]:
    """(code bytes, scale bytes) of one packed vector."""
    cb, sb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    fmt = SCALE_FORMATS[scale_format] if isinstance(scale_format, str) else int(scale_format)
    _check("srft_kv_vector_bytes", library().srft_kv_vector_bytes(d, bits, group, fmt, ctypes.byref(cb),
                                                                  ctypes.byref(sb)))
    return cb.value, sb.value


def srft_transform(x: torch.Tensor, y: torch.Tensor, n: int, d: int, sign_seed: int, inverse: bool,
                   stream=None) -> None:
    rc = library().srft_transform(_ptr(x), _ptr(y), n, d, sign_seed, int(bool(inverse)), _stream(stream))
    _check("srft_transform", rc)


def srht_transform(x: torch.Tensor, y: torch.Tensor, n: int, d: int, sign_seed: int, inverse: bool,
                   stream=None) -> None:
    rc = library().srht_transform(_ptr(x), _ptr(y), n, d, sign_seed, int(bool(inverse)), _stream(stream))
    _check("srht_transform", rc)


def srftkv_device_fault() -> int:
    f = ctypes.c_uint(0)
    _check("srftkv_device_fault", library().srftkv_device_fault(ctypes.byref(f)))
    return f.value


def srftkv_set_attention_poll_limit_for_testing(polls: int) -> None:
    """Test hook: polls of the attention kernel's chunk wait before a warp gives up (negative = the default,
    0 = give up at the first chunk)."""
    _check("srftkv_set_attention_poll_limit_for_testing",
           library().srftkv_set_attention_poll_limit_for_testing(int(polls)))


def srftkv_set_codec_poll_limit_for_testing(polls: int) -> None:
    """Test hook: polls of the register-path quantize kernels' tile wait before a warp gives up (negative = the
    default, 0 = give up at the first tile)."""
    _check("srftkv_set_codec_poll_limit_for_testing",
           library().srftkv_set_codec_poll_limit_for_testing(int(polls)))


def srftkv_last_error() -> str:
    return library().srftkv_last_error().decode()
