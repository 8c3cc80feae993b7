"""Python binding of the sm_103a token-sparse MLA decode library (libmla.so).

Argument marshalling only: every step of the decode runs in the library's
CUDA kernels, declared in ``include/mla.h``.  PyTorch supplies device memory
and the current stream.  There is no CPU path: if the library is missing or
a tensor is not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from . import build as _build

__all__ = [
    "MLAError", "Problem", "load", "get_metadata", "sparse_decode", "sparse_decode_rope_fp8", "combine",
    "dequantize", "kv_write",
    "SparseMLADecoder", "decode", "KV_NONE", "KV_FP8_528", "KV_FP4_288", "KV_BF16",
    "DEVERR_BAD_INDEX", "DEVERR_TIMEOUT", "DEVERR_BAD_METADATA", "DEVERR_NO_ROOM", "DEVERR_BAD_LENGTH", "SCHED_INTS",
    "page_plan", "RopeScaling", "RopeTable", "rope", "kv_append", "page_means", "rms_norm_fp8",
    "PagedProblem", "paged_decode_plan", "paged_decode_fp4", "PagedFP4Decoder",
    "PagedSparseProblem", "paged_sparse_plan", "paged_sparse_decode_fp4", "PagedSparseFP4Decoder",
    "PagedSharedProblem", "paged_shared_plan", "paged_shared_decode_fp4", "PagedSharedFP4Decoder",
]

KV_NONE, KV_FP8_528, KV_FP4_288, KV_BF16 = 0, 1, 2, 3
DEVERR_BAD_INDEX, DEVERR_TIMEOUT, DEVERR_BAD_METADATA = 1, 2, 4
DEVERR_NO_ROOM, DEVERR_BAD_LENGTH = 8, 16
ROPE_MAX_DIM = 256
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
SCHED_INTS = 8
HEAD_DIM = 512
PAGE_SIZE = 64
FP8_RECORD_BYTES = 528
FP4_RECORD_BYTES = 288
MEAN_BYTES = 528

STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_WORKSPACE",
          4: "MLA_ERR_CUDA", 5: "MLA_ERR_TIMEOUT"}


class MLAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class Problem(ctypes.Structure):
    """mla_problem_t (include/mla.h)."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("seq_len_q", ctypes.c_int32), ("h_q", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("topk", ctypes.c_int32),
        ("extra_topk", ctypes.c_int32), ("num_pages", ctypes.c_int64), ("extra_num_pages", ctypes.c_int64),
        ("page_size", ctypes.c_int32), ("kv_format", ctypes.c_int32), ("extra_kv_format", ctypes.c_int32),
        ("sm_scale", ctypes.c_float),
    ]

    @classmethod
    def make(cls, batch, seq_len_q, h_q, topk, num_pages, extra_topk=0, extra_num_pages=0,
             sm_scale=None, kv_format=KV_FP8_528, extra_kv_format=None, head_dim=HEAD_DIM,
             page_size=PAGE_SIZE, num_kv_heads=1) -> "Problem":
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(head_dim)
        if extra_kv_format is None:
            extra_kv_format = KV_FP4_288 if extra_topk else KV_NONE
        return cls(batch, seq_len_q, h_q, head_dim, num_kv_heads, topk, extra_topk, num_pages,
                   extra_num_pages, page_size, kv_format, extra_kv_format, sm_scale)


class _RopeTableC(ctypes.Structure):
    """mla_rope_table_t (include/mla.h)."""
    _fields_ = [("rope_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("factor", ctypes.c_float),
                ("step", ctypes.c_uint64 * (ROPE_MAX_DIM // 2))]


class PagedProblem(ctypes.Structure):
    """mla_paged_problem_t (include/mla.h)."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("seq_len_q", ctypes.c_int32), ("h_q", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("num_pages", ctypes.c_int64),
        ("kv_format", ctypes.c_int32), ("sm_scale", ctypes.c_float),
    ]

    @classmethod
    def make(cls, batch, seq_len_q, h_q, max_pages, num_pages, window=0, sinks=0, sm_scale=None,
             head_dim=HEAD_DIM, page_size=PAGE_SIZE, kv_format=KV_FP4_288) -> "PagedProblem":
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(head_dim)
        return cls(batch, seq_len_q, h_q, head_dim, page_size, max_pages, window, sinks, num_pages, kv_format,
                   sm_scale)


class PagedSparseProblem(ctypes.Structure):
    """mla_paged_sparse_problem_t (include/mla.h)."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("seq_len_q", ctypes.c_int32), ("h_q", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("top_pages", ctypes.c_int32), ("sink_pages", ctypes.c_int32), ("local_pages", ctypes.c_int32),
        ("num_pages", ctypes.c_int64), ("kv_format", ctypes.c_int32), ("sm_scale", ctypes.c_float),
    ]

    @classmethod
    def make(cls, batch, seq_len_q, h_q, max_pages, num_pages, top_pages, sink_pages=1, local_pages=1, sm_scale=None,
             head_dim=HEAD_DIM, page_size=PAGE_SIZE, kv_format=KV_FP4_288) -> "PagedSparseProblem":
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(head_dim)
        return cls(batch, seq_len_q, h_q, head_dim, page_size, max_pages, top_pages, sink_pages, local_pages, num_pages,
                   kv_format, sm_scale)


class PagedSharedProblem(ctypes.Structure):
    """mla_paged_shared_problem_t (include/mla.h)."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("seq_len_q", ctypes.c_int32), ("h_q", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("groups", ctypes.c_int32),
        ("max_prefix_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("num_pages", ctypes.c_int64),
        ("kv_format", ctypes.c_int32), ("sm_scale", ctypes.c_float),
    ]

    @classmethod
    def make(cls, batch, seq_len_q, h_q, max_pages, max_prefix_pages, num_pages, groups=1, sm_scale=None,
             head_dim=HEAD_DIM, page_size=PAGE_SIZE, kv_format=KV_FP4_288) -> "PagedSharedProblem":
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(head_dim)
        return cls(batch, seq_len_q, h_q, head_dim, page_size, groups, max_prefix_pages, max_pages, num_pages, kv_format,
                   sm_scale)


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libmla.so (built in-tree by ``build.build()``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"libmla.so not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    PP = ctypes.POINTER(Problem)
    lib.mla_get_metadata.argtypes = [PP, I32, P, P, ctypes.POINTER(I32), ctypes.POINTER(SZ), P]
    lib.mla_sparse_decode.argtypes = [PP, P, P, P, P, P, P, P, I32, P, SZ, P, P, P, P]
    lib.mla_sparse_decode_rope_fp8.argtypes = [PP, P, P, P, P, P, P, P, I32, P, SZ, P, ctypes.c_float, P, P, P, P]
    lib.mla_combine.argtypes = [PP, P, P, P, P, P, P]
    lib.mla_dequantize.argtypes = [I32, P, I64, P, P]
    lib.mla_kv_write.argtypes = [I32, P, P, I64, P, I64, P, P]
    F, D = ctypes.c_float, ctypes.c_double
    lib.mla_page_plan.argtypes = [P, P, I32, P, I32, P, I32, P, P, P, P, P, P, I32, P, P]
    lib.mla_rope_table.argtypes = [P, I32, I32, D, I32, D, D, D, D, D]
    lib.mla_rope_table_from_freqs.argtypes = [P, I32, I32, P, D]
    lib.mla_rope.argtypes = [I32, P, I64, I64, P, I64, I64, I64, I32, I32, I32, P, P, I32, P]
    lib.mla_kv_append.argtypes = [I32, I32, P, I64, I64, P, I32, P, P, P, I64, P, P]
    lib.mla_page_means.argtypes = [P, I64, P, I64, P, P, P]
    lib.mla_rms_norm_fp8.argtypes = [I32, P, I64, P, I64, P, F, P, I64, P, I64, P, I64, I64, I32, P, P]
    lib.mla_paged_decode_plan.argtypes = [P, I32, ctypes.POINTER(I32), ctypes.POINTER(SZ)]
    lib.mla_paged_decode_fp4.argtypes = [P, P, P, P, P, I32, P, SZ, P, P, P, P]
    lib.mla_paged_sparse_plan.argtypes = [P, I32, ctypes.POINTER(I32), ctypes.POINTER(SZ)]
    lib.mla_paged_sparse_decode_fp4.argtypes = [P, P, P, P, P, P, I32, P, SZ, P, P, P, P, P]
    lib.mla_paged_shared_plan.argtypes = [P, I32, ctypes.POINTER(I32), ctypes.POINTER(SZ)]
    lib.mla_paged_shared_decode_fp4.argtypes = [P, P, P, P, P, P, P, P, I32, P, SZ, P, P, P, P]
    lib.mla_status_string.argtypes = [ctypes.c_int]
    lib.mla_status_string.restype = ctypes.c_char_p
    for f in (lib.mla_get_metadata, lib.mla_sparse_decode, lib.mla_sparse_decode_rope_fp8, lib.mla_combine,
              lib.mla_dequantize, lib.mla_kv_write, lib.mla_page_plan, lib.mla_rope_table,
              lib.mla_rope_table_from_freqs, lib.mla_rope, lib.mla_kv_append, lib.mla_page_means, lib.mla_rms_norm_fp8, lib.mla_paged_decode_plan,
              lib.mla_paged_decode_fp4, lib.mla_paged_sparse_plan, lib.mla_paged_sparse_decode_fp4,
              lib.mla_paged_shared_plan, lib.mla_paged_shared_decode_fp4):
        f.restype = ctypes.c_int
    if path == _build.LIB:
        _lib = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        raise MLAError(status, what)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device (no CPU path)")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream=None):
    return stream.cuda_stream if stream is not None else _raw_stream(_current_device())


def get_metadata(problem: Problem, num_sms: int = 0, device=None, stream=None):
    """Return (sched int32[num_parts, 8], num_splits int32[b*s+1], num_parts, workspace_bytes)."""
    lib = load()
    parts = ctypes.c_int32(0)
    ws = ctypes.c_size_t(0)
    _check(lib.mla_get_metadata(ctypes.byref(problem), num_sms, None, None, ctypes.byref(parts),
                                ctypes.byref(ws), None), "mla_get_metadata (query)")
    device = device or torch.device("cuda", torch.cuda.current_device())
    sched = torch.empty((parts.value, SCHED_INTS), dtype=torch.int32, device=device)
    nsplit = torch.empty((problem.batch * problem.seq_len_q + 1,), dtype=torch.int32, device=device)
    _check(lib.mla_get_metadata(ctypes.byref(problem), num_sms, _ptr(sched), _ptr(nsplit),
                                ctypes.byref(parts), ctypes.byref(ws), _stream(stream)), "mla_get_metadata")
    return sched, nsplit, parts.value, ws.value


def sparse_decode(problem: Problem, q, kv, indices, sched, num_splits, num_parts, workspace,
                  out, lse, extra_kv=None, extra_indices=None, error=None, stream=None):
    lib = load()
    _check(lib.mla_sparse_decode(ctypes.byref(problem), _ptr(q), _ptr(kv), _ptr(indices), _ptr(extra_kv),
                                 _ptr(extra_indices), _ptr(sched), _ptr(num_splits), num_parts,
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _ptr(out), _ptr(lse), _ptr(error), _stream(stream)), "mla_sparse_decode")


def sparse_decode_rope_fp8(problem: Problem, q, kv, indices, sched, num_splits, num_parts, workspace,
                           positions, rope_theta, out_fp8, lse, extra_kv=None, extra_indices=None, error=None,
                           stream=None):
    """The decode step with the fused output epilogue: conjugate rotary
    embedding of dims 448..511 and the cast to 528-byte FP8 records
    (out_fp8 uint8 [b, s, h, 528]); positions int32 [b, s]."""
    lib = load()
    _check(lib.mla_sparse_decode_rope_fp8(ctypes.byref(problem), _ptr(q), _ptr(kv), _ptr(indices), _ptr(extra_kv),
                                          _ptr(extra_indices), _ptr(sched), _ptr(num_splits), num_parts,
                                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _ptr(positions), float(rope_theta), _ptr(out_fp8), _ptr(lse),
                                          _ptr(error), _stream(stream)), "mla_sparse_decode_rope_fp8")


def combine(problem: Problem, num_splits, o_partial, lse_partial, out, lse, stream=None):
    lib = load()
    _check(lib.mla_combine(ctypes.byref(problem), _ptr(num_splits), _ptr(o_partial), _ptr(lse_partial),
                           _ptr(out), _ptr(lse), _stream(stream)), "mla_combine")


def kv_write(latents: torch.Tensor, slots: torch.Tensor, pool: torch.Tensor, kv_format: int = KV_FP8_528,
             num_pages: int = None, error: torch.Tensor = None, stream=None) -> None:
    """Quantize bf16 latents [n, 512] into FP8 (528-byte) or FP4 (288-byte)
    records and store each at its slot (page*64 + offset, -1 = skip) of the
    uint8 pool [num_pages, 64, record] (or [tokens, record])."""
    lib = load()
    rec = FP8_RECORD_BYTES if kv_format == KV_FP8_528 else FP4_RECORD_BYTES
    if num_pages is None:
        num_pages = pool.numel() // (PAGE_SIZE * rec)
    n = latents.shape[0] if latents.dim() > 0 else 0
    _check(lib.mla_kv_write(kv_format, _ptr(latents), _ptr(slots), n, _ptr(pool), num_pages, _ptr(error),
                            _stream(stream)), "mla_kv_write")


def dequantize(records: torch.Tensor, kv_format: int = KV_FP8_528, stream=None) -> torch.Tensor:
    """uint8 [n, 528|288] records -> bf16 [n, 512], with the decode kernel's dequantization."""
    lib = load()
    n = records.shape[0]
    out = torch.empty((n, HEAD_DIM), dtype=torch.bfloat16, device=records.device)
    _check(lib.mla_dequantize(kv_format, _ptr(records), n, _ptr(out), _stream(stream)), "mla_dequantize")
    return out


class SparseMLADecoder:
    """Metadata and workspace planned once for a problem shape; one call per step."""

    def __init__(self, problem: Problem, device=None, num_sms: int = 0, stream=None):
        self.problem = problem
        self.device = device or torch.device("cuda", torch.cuda.current_device())
        self.sched, self.num_splits, self.num_parts, self.ws_bytes = get_metadata(
            problem, num_sms, self.device, stream)
        self.workspace = torch.empty((max(self.ws_bytes, 16),), dtype=torch.uint8, device=self.device)
        self.error = torch.zeros((1,), dtype=torch.int32, device=self.device)

    def __call__(self, q, kv, indices, extra_kv=None, extra_indices=None, out=None, lse=None, stream=None):
        p = self.problem
        if out is None:
            out = torch.empty((p.batch, p.seq_len_q, p.h_q, HEAD_DIM), dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty((p.batch, p.seq_len_q, p.h_q), dtype=torch.float32, device=q.device)
        sparse_decode(p, q, kv, indices, self.sched, self.num_splits, self.num_parts, self.workspace,
                      out, lse, extra_kv, extra_indices, self.error, stream)
        return out, lse

    def rope_fp8(self, q, kv, indices, positions, rope_theta=10000.0, extra_kv=None, extra_indices=None,
                 out=None, lse=None, stream=None):
        """Decode with the fused epilogue; returns (FP8 records uint8 [b, s, h, 528], lse)."""
        p = self.problem
        if out is None:
            out = torch.empty((p.batch, p.seq_len_q, p.h_q, FP8_RECORD_BYTES), dtype=torch.uint8, device=q.device)
        if lse is None:
            lse = torch.empty((p.batch, p.seq_len_q, p.h_q), dtype=torch.float32, device=q.device)
        sparse_decode_rope_fp8(p, q, kv, indices, self.sched, self.num_splits, self.num_parts, self.workspace,
                               positions, rope_theta, out, lse, extra_kv, extra_indices, self.error, stream)
        return out, lse


def decode(q, kv, indices, extra_kv=None, extra_indices=None, sm_scale=None):
    """One-shot decode.  q bf16 [b, s, h, 512]; kv uint8 [pages, 64, 528] (or
    [tokens, 528]); indices int32 [b, s, topk]; optional FP4 extra cache.
    Returns (out bf16 [b, s, h, 512], lse float32 [b, s, h])."""
    b, s, h, d = q.shape
    num_pages = kv.numel() // (PAGE_SIZE * FP8_RECORD_BYTES)
    xtopk = extra_indices.shape[-1] if extra_indices is not None else 0
    xpages = extra_kv.numel() // (PAGE_SIZE * FP4_RECORD_BYTES) if extra_kv is not None else 0
    prob = Problem.make(b, s, h, indices.shape[-1], num_pages, extra_topk=xtopk, extra_num_pages=xpages,
                        sm_scale=sm_scale, head_dim=d)
    return SparseMLADecoder(prob, q.device)(q, kv, indices, extra_kv, extra_indices)


# ---------------------------------------------------------------------------
# The operators around the paged FP4 cache.  Every tensor of a call lies on
# one CUDA device; the call runs there, on `stream` or that device's current
# stream, whichever device is current.
# ---------------------------------------------------------------------------


def _device_of(t, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what}: tensor must be on a CUDA device (no CPU path)")
    return dev


def _refuse(t, dev, dtype, what, shape):
    if _device_of(t, what) != dev:
        raise ValueError(f"{what}: all tensors of a call must be on one device")
    if t.dtype is not dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{what}: tensor must be contiguous")


def _arg(t, dev, dtype, what, shape=None):
    """Address of a dense tensor of this type (and shape) on device dev; None stays None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not dtype or (
            shape is not None and t.shape != shape) or not t.is_contiguous():
        _refuse(t, dev, dtype, what, shape)
    return t.data_ptr()


def _call(fn, what, dev, stream, *args):
    """fn(*args, stream) on device dev."""
    if stream is not None and getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"{what}: stream of device {stream.device_index}, tensors on device {dev}")
    raw = stream.cuda_stream if stream is not None else _raw_stream(dev)
    if dev == _current_device():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != 0:
        raise MLAError(status, what)


def page_plan(cached_lens, new_lens, block_table, free_pages, num_free, seq_lens, num_free_out, cu_new, slots,
              positions, error=None, stream=None) -> None:
    """Pages and slots for the new tokens of each request, on the device
    (mla_page_plan): new_lens[r] tokens are appended to cached_lens[r], -1
    ends a request and gives its pages back.  All int32: cached_lens,
    new_lens, seq_lens [b]; block_table [b, max_pages]; free_pages
    [num_pages], a stack of num_free [1] ids; cu_new [b + 1]; slots and
    positions [max_new].  seq_lens may be cached_lens and num_free_out
    num_free."""
    lib = load()
    dev = _device_of(cached_lens, "page_plan")
    i32 = torch.int32
    if block_table.dim() != 2 or cached_lens.dim() != 1 or slots.dim() != 1 or free_pages.dim() != 1:
        raise ValueError("page_plan: block_table is [b, max_pages]; lengths, slots and free_pages are one-dimensional")
    b, max_pages = block_table.shape
    _call(lib.mla_page_plan, "mla_page_plan", dev, stream,
          _arg(cached_lens, dev, i32, "cached_lens", (b,)), _arg(new_lens, dev, i32, "new_lens", (b,)), b,
          _arg(block_table, dev, i32, "block_table"), max_pages, _arg(free_pages, dev, i32, "free_pages"),
          free_pages.shape[0], _arg(num_free, dev, i32, "num_free", (1,)), _arg(seq_lens, dev, i32, "seq_lens", (b,)),
          _arg(num_free_out, dev, i32, "num_free_out", (1,)), _arg(cu_new, dev, i32, "cu_new", (b + 1,)),
          _arg(slots, dev, i32, "slots"), _arg(positions, dev, i32, "positions", slots.shape), slots.shape[0],
          _arg(error, dev, i32, "error"))


class RopeScaling:
    """How rotary frequencies are scaled for contexts past the trained length."""

    def __init__(self, kind: int, scale: float, original_len: float = 0.0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, attention_factor: float = 1.0):
        self.kind, self.scale, self.original_len = kind, float(scale), float(original_len)
        self.beta_fast, self.beta_slow, self.attention_factor = float(beta_fast), float(beta_slow), attention_factor

    @classmethod
    def linear(cls, scale: float) -> "RopeScaling":
        """Every frequency divided by scale."""
        return cls(1, scale)

    @classmethod
    def yarn(cls, scale: float, original_len: float, beta_fast: float = 32.0, beta_slow: float = 1.0) -> "RopeScaling":
        """Frequencies of fewer than beta_slow turns over original_len divided
        by scale, those of more than beta_fast kept, a ramp between; the
        rotated dims grow by 0.1 ln(scale) + 1."""
        factor = 0.1 * math.log(scale) + 1.0 if scale > 1.0 else 1.0
        return cls(2, scale, original_len, beta_fast, beta_slow, factor)


class RopeTable:
    """Rotary frequencies of rope_dim / 2 pairs (mla_rope_table_t), made once
    on the host.  interleaved: pairs (2j, 2j + 1); else (j, j + rope_dim / 2).
    attention_factor overrides the scaling's factor; freqs (radians per
    position, one per pair) replaces theta and scaling."""

    def __init__(self, rope_dim: int, theta: float = 10000.0, interleaved: bool = True, scaling: RopeScaling = None,
                 attention_factor: float = None, freqs=None):
        lib = load()
        self.c = _RopeTableC()
        self.ref = ctypes.addressof(self.c)
        layout = 0 if interleaved else 1
        factor = attention_factor
        if factor is None:
            factor = scaling.attention_factor if scaling is not None else 1.0
        if freqs is not None:
            freqs = [float(f) for f in freqs]
            if scaling is not None or len(freqs) != rope_dim // 2:
                raise ValueError("RopeTable: freqs gives one frequency per pair, with no scaling on top")
            status = lib.mla_rope_table_from_freqs(self.ref, rope_dim, layout, (ctypes.c_double * len(freqs))(*freqs),
                                                   factor)
        else:
            k = scaling or RopeScaling(0, 1.0)
            status = lib.mla_rope_table(self.ref, rope_dim, layout, theta, k.kind, k.scale, k.original_len, k.beta_fast,
                                        k.beta_slow, factor)
        _check(status, "mla_rope_table")
        self.rope_dim = rope_dim


def rope(x, positions, table: RopeTable, offset: int = 0, conjugate: bool = False, out=None, stream=None):
    """Turn dims offset .. offset + table.rope_dim - 1 of every head of x [n,
    heads, d] (or [n, d]) to its row's position (positions int32 [n]); any
    row and head strides, the last dim dense.  In place without `out`; with
    it the other dims are copied.  conjugate: the inverse turn, which is also
    how a gradient of the result becomes the gradient of x.  Returns out."""
    lib = load()
    dev = _device_of(x, "rope")
    y = x if out is None else out
    if _device_of(y, "rope") != dev:
        raise ValueError("out: all tensors of a call must be on one device")
    dtype = _DTYPES.get(x.dtype)
    if dtype is None or y.dtype is not x.dtype:
        raise ValueError(f"rope: bfloat16, float16 or float32, the same for x and out (got {x.dtype}, {y.dtype})")
    if x.dim() not in (2, 3) or y.shape != x.shape:
        raise ValueError("rope: x is [n, heads, d] or [n, d], out of the same shape")
    n, d = x.shape[0], x.shape[-1]
    heads = x.shape[1] if x.dim() == 3 else 1
    xs, ys = x.stride(), y.stride()
    if d > 1 and (xs[-1] != 1 or ys[-1] != 1):
        raise ValueError("rope: the last dim must be dense")
    if n == 0 or heads == 0:
        return y
    three = x.dim() == 3
    _call(lib.mla_rope, "mla_rope", dev, stream, dtype, x.data_ptr(), xs[0], xs[1] if three else 0, y.data_ptr(), ys[0],
          ys[1] if three else 0, n, heads, d, offset, _arg(positions, dev, torch.int32, "positions", (n,)), table.ref,
          1 if conjugate else 0)
    return y


def _rows(t, dev, dtype, what, shape):
    """Address and row stride of a [n, d] tensor whose rows are dense."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(t, dev, dtype, what, shape)
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError(f"{what}: rows must be dense")
    return t.data_ptr(), s0 if shape[0] > 1 else shape[1]


def _pool(pool, dev, rec, num_pages, what):
    """Address and page count of a uint8 pool of records: [num_pages, 64, rec] or [tokens, rec], or any of that size."""
    ptr = _arg(pool, dev, torch.uint8, "pool")
    held = pool.numel() // (PAGE_SIZE * rec)
    if num_pages is None:
        num_pages = held
    if num_pages < 0 or num_pages > held:
        raise ValueError(f"{what}: the pool holds {held} pages of {rec}-byte records, not {num_pages}")
    return ptr, num_pages


def kv_append(latents, slots, pool, kv_format: int = KV_FP8_528, rope: RopeTable = None, positions=None,
              offset: int = 448, num_pages: int = None, error=None, stream=None) -> None:
    """New tokens into the paged pool, their rotary positions applied on the
    way (mla_kv_append): dims offset .. offset + rope.rope_dim - 1 of each row
    of latents [n, 512] (bf16, fp16 or fp32, any row stride of whole 16 bytes)
    turn to positions int32 [n]; each row becomes an FP8 (528-byte) or FP4
    (288-byte) record at its slot (page*64 + offset, -1 = skip) of the uint8
    pool [num_pages, 64, record].  Without rope nothing turns."""
    lib = load()
    dev = _device_of(latents, "kv_append")
    dtype = _DTYPES.get(latents.dtype)
    if dtype is None or latents.dim() != 2 or latents.shape[1] != HEAD_DIM:
        raise ValueError("kv_append: latents are [n, 512] in bfloat16, float16 or float32 "
                         f"(got {latents.dtype}, {tuple(latents.shape)})")
    n = latents.shape[0]
    px, sx = _rows(latents, dev, latents.dtype, "latents", latents.shape)
    if rope is None and positions is not None:
        raise ValueError("kv_append: positions without a rope table")
    if rope is not None and positions is None:
        raise ValueError("kv_append: a rope table needs positions")
    if kv_format not in (KV_FP8_528, KV_FP4_288):
        raise MLAError(2 if kv_format == KV_BF16 else 1, "mla_kv_append")
    ptr, num_pages = _pool(pool, dev, FP8_RECORD_BYTES if kv_format == KV_FP8_528 else FP4_RECORD_BYTES, num_pages,
                           "kv_append")
    ps = _arg(slots, dev, torch.int32, "slots", (n,))
    pp = _arg(positions, dev, torch.int32, "positions", (n,))
    _call(lib.mla_kv_append, "mla_kv_append", dev, stream, kv_format, dtype, px, sx, n, rope.ref if rope is not None else None,
          offset, pp, ps, ptr, num_pages, _arg(error, dev, torch.int32, "error"))


def page_means(pool, slots, means, num_pages: int = None, error=None, stream=None) -> None:
    """The 8-bit means of the pages that slots (int32 [n]) complete, those with
    a slot % 64 == 63 in the list, from the FP4 pool [num_pages, 64, 288] into
    means uint8 [num_pages, 528] (mla_page_means): 512 int8 codes, the byte
    127 + e of their scale, zeros."""
    lib = load()
    dev = _device_of(pool, "page_means")
    ptr, num_pages = _pool(pool, dev, FP4_RECORD_BYTES, num_pages, "page_means")
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("page_means: slots are int32 [n]")
    pm = _arg(means, dev, torch.uint8, "means")
    if means.numel() < num_pages * MEAN_BYTES:
        raise ValueError(f"means: expected {num_pages} records of {MEAN_BYTES} bytes")
    _call(lib.mla_page_means, "mla_page_means", dev, stream, ptr, num_pages, _arg(slots, dev, torch.int32, "slots"),
          slots.shape[0], pm, _arg(error, dev, torch.int32, "error"))


def rms_norm_fp8(x, weight, eps: float, codes, scales, residual=None, residual_out=None, error=None,
                 stream=None) -> None:
    """codes, scales = FP8 blocks of (x + residual) / rms * weight, and the sum
    itself, rounded, into residual_out (mla_rms_norm_fp8).  x, residual,
    residual_out [n, d], weight [d] of one type (bf16, fp16, fp32); codes
    uint8 [n, d] (E4M3FN) and scales uint8 [n, d / 32] (e8m0); any row
    strides, so records[:, :512] and records[:, 512:] of 528-byte rows serve.
    error: optional int32 [1] error word."""
    lib = load()
    dev = _device_of(x, "rms_norm_fp8")
    dtype = _DTYPES.get(x.dtype)
    if dtype is None or x.dim() != 2:
        raise ValueError(f"rms_norm_fp8: x is [n, d] in bfloat16, float16 or float32 (got {x.dtype}, {tuple(x.shape)})")
    n, d = x.shape
    px, sx = _rows(x, dev, x.dtype, "x", (n, d))
    pr, sr = _rows(residual, dev, x.dtype, "residual", (n, d))
    po, so = _rows(residual_out, dev, x.dtype, "residual_out", (n, d))
    pc, sc = _rows(codes, dev, torch.uint8, "codes", (n, d))
    ps, ss = _rows(scales, dev, torch.uint8, "scales", (n, d // 32))
    pw = _arg(weight, dev, x.dtype, "weight", (d,))
    if n == 0 and d % 32 == 0 and d > 0:
        return
    _call(lib.mla_rms_norm_fp8, "mla_rms_norm_fp8", dev, stream, dtype, px, sx, pr, sr, pw, eps, po, so, pc, sc, ps, ss,
          n, d, _arg(error, dev, torch.int32, "error"))


def paged_decode_plan(problem: PagedProblem, num_sms: int = 0):
    """(num_parts, workspace_bytes) of a paged decode (host only; num_sms = 0 asks the current device)."""
    lib = load()
    parts, ws = ctypes.c_int32(0), ctypes.c_size_t(0)
    _check(lib.mla_paged_decode_plan(ctypes.addressof(problem), num_sms, ctypes.byref(parts), ctypes.byref(ws)),
           "mla_paged_decode_plan")
    return parts.value, ws.value


def paged_decode_fp4(problem: PagedProblem, q, kv, block_table, seq_lens, num_parts, workspace, out, lse, error=None,
                     stream=None) -> None:
    """Attention of each sequence's last seq_len_q tokens over its pages of
    288-byte FP4 records (mla_paged_decode_fp4).  q, out bf16 [b, s, h, 512];
    kv uint8 [num_pages, 64, 288]; block_table int32 [b, max_pages]; seq_lens
    int32 [b]; lse float32 [b, s, h]; workspace uint8 as paged_decode_plan says."""
    lib = load()
    dev = _device_of(q, "paged_decode_fp4")
    p = problem
    rows = (p.batch, p.seq_len_q, p.h_q)
    if kv.numel() != p.num_pages * PAGE_SIZE * FP4_RECORD_BYTES:
        raise ValueError("kv: expected num_pages * 64 records of 288 bytes")
    _call(lib.mla_paged_decode_fp4, "mla_paged_decode_fp4", dev, stream, ctypes.addressof(p),
          _arg(q, dev, torch.bfloat16, "q", rows + (HEAD_DIM,)), _arg(kv, dev, torch.uint8, "kv"),
          _arg(block_table, dev, torch.int32, "block_table", (p.batch, p.max_pages)),
          _arg(seq_lens, dev, torch.int32, "seq_lens", (p.batch,)), num_parts,
          _arg(workspace, dev, torch.uint8, "workspace"), workspace.numel(),
          _arg(out, dev, torch.bfloat16, "out", q.shape), _arg(lse, dev, torch.float32, "lse", rows),
          _arg(error, dev, torch.int32, "error"))


class PagedFP4Decoder:
    """Plan and workspace of a paged decode, made once for a problem shape.
    The workspace serves one call at a time: concurrent streams, and graphs
    that are replayed concurrently, take a decoder each."""

    def __init__(self, problem: PagedProblem, device=None, num_sms: int = 0):
        self.problem = problem
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.device(self.device):
            self.num_parts, self.ws_bytes = paged_decode_plan(problem, num_sms)
        self.workspace = torch.empty((self.ws_bytes,), dtype=torch.uint8, device=self.device)
        self.error = torch.zeros((1,), dtype=torch.int32, device=self.device)

    def __call__(self, q, kv, block_table, seq_lens, out=None, lse=None, stream=None):
        if out is None or lse is None:
            # Memory of the stream that writes it, so that freeing it early cannot hand it to another one's kernels.
            with torch.cuda.stream(stream):
                out = torch.empty_like(q) if out is None else out
                lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device) if lse is None else lse
        paged_decode_fp4(self.problem, q, kv, block_table, seq_lens, self.num_parts, self.workspace, out, lse,
                         self.error, stream)
        return out, lse


def paged_sparse_plan(problem: PagedSparseProblem, num_sms: int = 0):
    """(num_parts, workspace_bytes) of a decode over selected pages (host only; num_sms = 0 asks the current device)."""
    lib = load()
    parts, ws = ctypes.c_int32(0), ctypes.c_size_t(0)
    _check(lib.mla_paged_sparse_plan(ctypes.addressof(problem), num_sms, ctypes.byref(parts), ctypes.byref(ws)),
           "mla_paged_sparse_plan")
    return parts.value, ws.value


def paged_sparse_decode_fp4(problem: PagedSparseProblem, q, kv, means, block_table, seq_lens, num_parts, workspace, out,
                            lse, selected=None, error=None, stream=None) -> None:
    """Attention of each sequence's last seq_len_q tokens over the pages that
    the pages' means (uint8 [num_pages, 528], page_means) select for each of
    them (mla_paged_sparse_decode_fp4).  selected: optional int32 [b, s,
    top_pages], the pages taken, ascending, -1 after the last; the others as
    in paged_decode_fp4, the workspace as paged_sparse_plan says."""
    lib = load()
    dev = _device_of(q, "paged_sparse_decode_fp4")
    p = problem
    rows = (p.batch, p.seq_len_q, p.h_q)
    u8, i32 = torch.uint8, torch.int32
    if kv.numel() != p.num_pages * PAGE_SIZE * FP4_RECORD_BYTES:
        raise ValueError("kv: expected num_pages * 64 records of 288 bytes")
    _call(lib.mla_paged_sparse_decode_fp4, "mla_paged_sparse_decode_fp4", dev, stream, ctypes.addressof(p),
          _arg(q, dev, torch.bfloat16, "q", rows + (HEAD_DIM,)), _arg(kv, dev, u8, "kv"),
          _arg(means, dev, u8, "means", (p.num_pages, MEAN_BYTES)),
          _arg(block_table, dev, i32, "block_table", (p.batch, p.max_pages)),
          _arg(seq_lens, dev, i32, "seq_lens", (p.batch,)), num_parts, _arg(workspace, dev, u8, "workspace"),
          workspace.numel(), _arg(out, dev, torch.bfloat16, "out", q.shape), _arg(lse, dev, torch.float32, "lse", rows),
          _arg(selected, dev, i32, "selected", (p.batch, p.seq_len_q, p.top_pages)), _arg(error, dev, i32, "error"))


class PagedSparseFP4Decoder:
    """Plan and workspace of a decode over selected pages, made once for a
    problem shape.  The workspace serves one call at a time: concurrent
    streams, and graphs that are replayed concurrently, take a decoder each."""

    def __init__(self, problem: PagedSparseProblem, device=None, num_sms: int = 0):
        self.problem = problem
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.device(self.device):
            self.num_parts, self.ws_bytes = paged_sparse_plan(problem, num_sms)
        self.workspace = torch.empty((self.ws_bytes,), dtype=torch.uint8, device=self.device)
        self.error = torch.zeros((1,), dtype=torch.int32, device=self.device)

    def __call__(self, q, kv, means, block_table, seq_lens, out=None, lse=None, selected=None, stream=None):
        """(out, lse, selected); memory for those not given comes from the call's stream."""
        p = self.problem
        if out is None or lse is None or selected is None:
            with torch.cuda.stream(stream):
                out = torch.empty_like(q) if out is None else out
                lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device) if lse is None else lse
                if selected is None:
                    selected = torch.empty(q.shape[:2] + (p.top_pages,), dtype=torch.int32, device=q.device)
        paged_sparse_decode_fp4(p, q, kv, means, block_table, seq_lens, self.num_parts, self.workspace, out, lse, selected,
                                self.error, stream)
        return out, lse, selected


def paged_shared_plan(problem: PagedSharedProblem, num_sms: int = 0):
    """(num_parts, workspace_bytes) of a decode with shared prefixes (host only; num_sms = 0 asks the current device)."""
    lib = load()
    parts, ws = ctypes.c_int32(0), ctypes.c_size_t(0)
    _check(lib.mla_paged_shared_plan(ctypes.addressof(problem), num_sms, ctypes.byref(parts), ctypes.byref(ws)),
           "mla_paged_shared_plan")
    return parts.value, ws.value


def paged_shared_decode_fp4(problem: PagedSharedProblem, q, kv, group_start, prefix_table, prefix_lens, block_table,
                            seq_lens, num_parts, workspace, out, lse, error=None, stream=None) -> None:
    """Attention of each sequence's last seq_len_q tokens over its group's
    prefix and its own pages (mla_paged_shared_decode_fp4).  All int32:
    group_start [groups + 1], prefix_table [groups, max_prefix_pages],
    prefix_lens [groups], block_table [b, max_pages] and seq_lens [b] of the
    sequences' own tokens; the others as in paged_decode_fp4, the workspace as
    paged_shared_plan says."""
    lib = load()
    dev = _device_of(q, "paged_shared_decode_fp4")
    p = problem
    rows = (p.batch, p.seq_len_q, p.h_q)
    i32 = torch.int32
    if kv.numel() != p.num_pages * PAGE_SIZE * FP4_RECORD_BYTES:
        raise ValueError("kv: expected num_pages * 64 records of 288 bytes")
    _call(lib.mla_paged_shared_decode_fp4, "mla_paged_shared_decode_fp4", dev, stream, ctypes.addressof(p),
          _arg(q, dev, torch.bfloat16, "q", rows + (HEAD_DIM,)), _arg(kv, dev, torch.uint8, "kv"),
          _arg(group_start, dev, i32, "group_start", (p.groups + 1,)),
          _arg(prefix_table, dev, i32, "prefix_table", (p.groups, p.max_prefix_pages)),
          _arg(prefix_lens, dev, i32, "prefix_lens", (p.groups,)),
          _arg(block_table, dev, i32, "block_table", (p.batch, p.max_pages)),
          _arg(seq_lens, dev, i32, "seq_lens", (p.batch,)), num_parts, _arg(workspace, dev, torch.uint8, "workspace"),
          workspace.numel(), _arg(out, dev, torch.bfloat16, "out", q.shape), _arg(lse, dev, torch.float32, "lse", rows),
          _arg(error, dev, i32, "error"))


class PagedSharedFP4Decoder:
    """Plan and workspace of a decode with shared prefixes, made once for a
    problem shape.  The workspace serves one call at a time: concurrent
    streams, and graphs that are replayed concurrently, take a decoder each."""

    def __init__(self, problem: PagedSharedProblem, device=None, num_sms: int = 0):
        self.problem = problem
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.device(self.device):
            self.num_parts, self.ws_bytes = paged_shared_plan(problem, num_sms)
        self.workspace = torch.empty((self.ws_bytes,), dtype=torch.uint8, device=self.device)
        self.error = torch.zeros((1,), dtype=torch.int32, device=self.device)

    def __call__(self, q, kv, group_start, prefix_table, prefix_lens, block_table, seq_lens, out=None, lse=None,
                 stream=None):
        if out is None or lse is None:
            with torch.cuda.stream(stream):  # memory of the stream that writes it
                out = torch.empty_like(q) if out is None else out
                lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device) if lse is None else lse
        paged_shared_decode_fp4(self.problem, q, kv, group_start, prefix_table, prefix_lens, block_table, seq_lens,
                                self.num_parts, self.workspace, out, lse, self.error, stream)
        return out, lse
