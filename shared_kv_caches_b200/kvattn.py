"""Thin ctypes binding of libkvattn.so (include/kvattn.h).

The functions carry the C names and only marshal arguments: device pointers
are Python ints (``tensor.data_ptr()``), streams are ``cudaStream_t`` handles
as ints (``torch.cuda.current_stream().cuda_stream``).  Every step of the
computation runs in the library's CUDA kernels; there is no fallback.  If the
library is missing, loading raises.

``decode_tensors`` is a convenience that reads pointers and sizes from torch
tensors and calls ``kvattn_decode``.
"""

from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvattn.so")

KVATTN_GQA, KVATTN_MQA, KVATTN_MLA, KVATTN_GLA, KVATTN_MLRA, KVATTN_GTA = range(6)
VARIANTS = {"gqa": KVATTN_GQA, "mqa": KVATTN_MQA, "mla": KVATTN_MLA, "gla": KVATTN_GLA,
            "mlra": KVATTN_MLRA, "gta": KVATTN_GTA}
KVATTN_OUT_BF16, KVATTN_OUT_FP32 = 0, 1
KVATTN_OK = 0
KVATTN_ERR_INVALID_ARG = -1
KVATTN_ERR_UNSUPPORTED = -2
KVATTN_ERR_WORKSPACE_TOO_SMALL = -3
KVATTN_ERR_MISALIGNED = -4
KVATTN_ERR_CUDA = -5
KVATTN_DEVERR_PAGE_OUT_OF_RANGE = 1
KVATTN_DEVERR_SEQ_TOO_LONG = 2
KVATTN_DEVERR_WAIT_TIMEOUT = 4
KVATTN_DEVERR_POS_OUT_OF_RANGE = 8
KVATTN_DEVERR_POOL_EXHAUSTED = 16
KVATTN_DEVERR_TOO_MANY_TOKENS = 32
KVATTN_DEVERR_BAD_LENGTH = 64
KERNEL_NAMES = {0: "generic", 1: "gqa", 2: "latent_tc", 3: "mqa_tc", 4: "latent_pair", 5: "gqa_fp8"}
KVATTN_CACHE_BF16, KVATTN_CACHE_FP8_E4M3 = 0, 1
KVATTN_SELFTEST_MISSED_PHASE = 256

EXPORTS = ("kvattn_get_plan", "kvattn_workspace_size", "kvattn_workspace_init", "kvattn_decode",
           "kvattn_decode_timed", "kvattn_decode_noalloc", "kvattn_get_device_error",
           "kvattn_status_string", "kvattn_version", "kvattn_selftest_bounded_wait", "kvattn_rope",
           "kvattn_append_kv", "kvattn_head_proj", "kvattn_build_tables", "kvattn_append_slots",
           "kvattn_expand_workspace_size", "kvattn_expand_kv", "kvattn_prefill_workspace_size",
           "kvattn_prefill")
KVATTN_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


class kvattn_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_q_heads", "num_kv", "d_nope", "d_rope", "page_size", "max_pages_per_seq",
        "num_pages", "max_seq_len", "num_splits", "out_dtype", "q_len", "branch_out", "cache_dtype")] + [
        ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class kvattn_plan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("num_splits", ctypes.c_int32),
                ("pages_per_split", ctypes.c_int32), ("ctas", ctypes.c_int32),
                ("launches", ctypes.c_int32), ("header_bytes", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_uint64)]


class kvattn_prefill_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_q_heads", "num_kv_heads", "d_nope", "d_rope", "d_v", "max_q_tokens", "max_kv_tokens",
        "causal", "out_dtype", "num_q_nope_heads")] + [(n, ctypes.c_int64 * 2) for n in (
            "q_nope_stride", "q_rope_stride", "k_stride", "v_stride", "out_stride")] + [
        ("k_rope_stride", ctypes.c_int64)]


class KvattnError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {kvattn_status_string(status)} ({status})")
        self.status = status


_lib = None


def load():
    """Load libkvattn.so (must have been built; see ``build.py``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with shared_kv_caches_b200.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(kvattn_params)
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    lib.kvattn_get_plan.argtypes = [i32, P, ctypes.POINTER(kvattn_plan)]
    lib.kvattn_workspace_size.argtypes = [i32, P, ctypes.POINTER(ctypes.c_size_t)]
    lib.kvattn_workspace_init.argtypes = [vp, ctypes.c_size_t, vp]
    lib.kvattn_decode.argtypes = [i32, P, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp,
                                  ctypes.c_size_t, vp]
    lib.kvattn_decode_timed.argtypes = [i32, P, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp,
                                        ctypes.c_size_t, vp, ctypes.POINTER(ctypes.c_void_p)]
    lib.kvattn_decode_noalloc.argtypes = [i32, P, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp]
    lib.kvattn_get_device_error.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int32)]
    lib.kvattn_status_string.argtypes = [ctypes.c_int]
    lib.kvattn_status_string.restype = ctypes.c_char_p
    lib.kvattn_version.argtypes = []
    lib.kvattn_selftest_bounded_wait.argtypes = [vp, i32, vp]
    lib.kvattn_rope.argtypes = [vp, i32, i32, i32, i32, i32, vp, ctypes.c_float, vp]
    lib.kvattn_append_kv.argtypes = [i32, P, vp, vp, vp, vp, ctypes.c_float, vp, vp]
    lib.kvattn_head_proj.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
    lib.kvattn_build_tables.argtypes = [i32] * 4 + [vp] * 13
    lib.kvattn_append_slots.argtypes = [i32, P, vp, i32, vp, vp, vp, ctypes.c_float, vp, vp]
    lib.kvattn_expand_workspace_size.argtypes = [i32, P, i32, ctypes.POINTER(ctypes.c_size_t)]
    lib.kvattn_expand_kv.argtypes = [i32, P, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp, vp]
    PP = ctypes.POINTER(kvattn_prefill_params)
    lib.kvattn_prefill_workspace_size.argtypes = [PP, ctypes.POINTER(ctypes.c_size_t)]
    lib.kvattn_prefill.argtypes = [PP] + [vp] * 7 + [ctypes.c_float, vp, vp, vp, ctypes.c_size_t, vp, vp]
    for name in ("kvattn_build_tables", "kvattn_append_slots", "kvattn_expand_workspace_size", "kvattn_expand_kv",
                 "kvattn_prefill_workspace_size", "kvattn_prefill"):
        getattr(lib, name).restype = ctypes.c_int
    for name in ("kvattn_get_plan", "kvattn_workspace_size", "kvattn_workspace_init", "kvattn_decode",
                 "kvattn_decode_timed", "kvattn_decode_noalloc", "kvattn_get_device_error",
                 "kvattn_version", "kvattn_selftest_bounded_wait", "kvattn_rope", "kvattn_append_kv",
                 "kvattn_head_proj"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def make_params(batch, num_q_heads, num_kv, d_nope, d_rope, max_pages_per_seq, num_pages,
                max_seq_len, num_splits=0, out_dtype=KVATTN_OUT_BF16, page_size=64, q_len=1,
                branch_out=0, cache_dtype=0, k_scale=1.0, v_scale=1.0) -> kvattn_params:
    return kvattn_params(int(batch), int(num_q_heads), int(num_kv), int(d_nope), int(d_rope),
                         int(page_size), int(max_pages_per_seq), int(num_pages), int(max_seq_len),
                         int(num_splits), int(out_dtype), int(q_len), int(branch_out), int(cache_dtype),
                         float(k_scale), float(v_scale))


def kvattn_version() -> int:
    return load().kvattn_version()


def kvattn_status_string(status: int) -> str:
    return load().kvattn_status_string(int(status)).decode()


def kvattn_get_plan(variant: int, params: kvattn_params) -> kvattn_plan:
    plan = kvattn_plan()
    st = load().kvattn_get_plan(int(variant), ctypes.byref(params), ctypes.byref(plan))
    if st:
        raise KvattnError(st, "kvattn_get_plan")
    return plan


def kvattn_workspace_size(variant: int, params: kvattn_params) -> int:
    n = ctypes.c_size_t(0)
    st = load().kvattn_workspace_size(int(variant), ctypes.byref(params), ctypes.byref(n))
    if st:
        raise KvattnError(st, "kvattn_workspace_size")
    return n.value


def kvattn_workspace_init(workspace: int, workspace_bytes: int, stream: int = 0) -> int:
    return load().kvattn_workspace_init(workspace, workspace_bytes, stream)


def kvattn_decode(variant, params, q_nope, q_rope, kv_cache, block_table, seq_lens, sm_scale, out,
                  lse, workspace, workspace_bytes, stream=0) -> int:
    """Call the C entry point; returns its status (0 = enqueued)."""
    return load().kvattn_decode(int(variant), ctypes.byref(params), q_nope, q_rope, kv_cache,
                                block_table, seq_lens, float(sm_scale), out, lse, workspace,
                                int(workspace_bytes), stream)


def kvattn_decode_timed(variant, params, q_nope, q_rope, kv_cache, block_table, seq_lens, sm_scale,
                        out, lse, workspace, workspace_bytes, stream, events) -> int:
    """``kvattn_decode`` recording three cudaEvent_t handles (ints or None)."""
    ev = (ctypes.c_void_p * 3)(*[e for e in events])
    return load().kvattn_decode_timed(int(variant), ctypes.byref(params), q_nope, q_rope, kv_cache,
                                      block_table, seq_lens, float(sm_scale), out, lse, workspace,
                                      int(workspace_bytes), stream, ev)


def kvattn_decode_noalloc(variant, params, q_nope, q_rope, kv_cache, block_table, seq_lens, sm_scale,
                          out, lse, device_error, stream=0) -> int:
    """Decode without a caller workspace (for callers that cannot allocate
    device memory); scratch is the library's own fixed device array."""
    return load().kvattn_decode_noalloc(int(variant), ctypes.byref(params), q_nope, q_rope, kv_cache,
                                        block_table, seq_lens, float(sm_scale), out, lse, device_error,
                                        stream)


def kvattn_selftest_bounded_wait(result: int, tries: int, stream: int = 0) -> int:
    """Enqueue the bounded-wait self-test; returns its status."""
    return load().kvattn_selftest_bounded_wait(result, int(tries), stream)


def kvattn_get_device_error(workspace: int, stream: int = 0) -> int:
    code = ctypes.c_int32(0)
    st = load().kvattn_get_device_error(workspace, stream, ctypes.byref(code))
    if st:
        raise KvattnError(st, "kvattn_get_device_error")
    return code.value


# ----------------------------------------------------------------- torch glue

def _ptr(t):
    return None if t is None else t.data_ptr()


def params_for(shape, max_pages_per_seq, num_pages, max_seq_len, num_splits=0) -> kvattn_params:
    """Params of a ``workloads.Shape`` problem."""
    return make_params(shape.batch, shape.num_q_heads, shape.num_kv, shape.d_nope, shape.d_rope,
                       max_pages_per_seq, num_pages, max_seq_len, num_splits,
                       KVATTN_OUT_FP32 if shape.out_dtype == "fp32" else KVATTN_OUT_BF16,
                       shape.page_size, shape.q_len, 1 if getattr(shape, "branch_out", False) else 0,
                       KVATTN_CACHE_FP8_E4M3 if getattr(shape, "cache_dtype", "bf16") == "fp8" else KVATTN_CACHE_BF16,
                       getattr(shape, "k_scale", 1.0), getattr(shape, "v_scale", 1.0))


def decode_tensors(variant, params, q_nope, q_rope, kv, block_table, seq_lens, sm_scale, out, lse,
                   workspace, stream=None, events=None) -> None:
    """``kvattn_decode`` on torch tensors; raises on a non-zero status.

    ``events``: three ``torch.cuda.Event`` (or None) recorded around the split
    pass and the combine pass on the launching stream.
    """
    if stream is None:
        import torch
        stream = torch.cuda.current_stream(q_nope.device).cuda_stream
    args = (variant, params, _ptr(q_nope), _ptr(q_rope), _ptr(kv), _ptr(block_table), _ptr(seq_lens),
            sm_scale, _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
            stream)
    if events is None:
        st = kvattn_decode(*args)
    else:
        st = kvattn_decode_timed(*args, [None if e is None else e.cuda_event for e in events])
    if st:
        raise KvattnError(st, "kvattn_decode")


# ------------------------------------------------- the steps either side

def kvattn_rope(x, rows, row_elems, rot_offset, rot_dim, rows_per_pos, pos, rope_base, stream=0) -> int:
    return load().kvattn_rope(x, int(rows), int(row_elems), int(rot_offset), int(rot_dim), int(rows_per_pos),
                              pos, float(rope_base), stream)


def kvattn_append_kv(variant, params, new_kv, pos, block_table, kv_cache, rope_base, device_error=None,
                     stream=0) -> int:
    return load().kvattn_append_kv(int(variant), ctypes.byref(params), new_kv, pos, block_table, kv_cache,
                                   float(rope_base), device_error, stream)


def kvattn_head_proj(x, w, y, out_dtype, rows, heads, k, n, device_error=None, stream=0) -> int:
    return load().kvattn_head_proj(x, w, y, int(out_dtype), int(rows), int(heads), int(k), int(n),
                                   device_error, stream)


def rope_tensor(x, pos, rot_offset, rot_dim, rope_base, rows_per_pos):
    """In-place RoPE on a contiguous bf16 tensor whose last axis is the row
    (argument marshalling only; the rotation runs in kvattn_rope)."""
    import torch
    assert x.dtype == torch.bfloat16 and x.is_contiguous() and pos.dtype == torch.int32
    row_elems = x.shape[-1]
    rows = x.numel() // row_elems
    st = kvattn_rope(_ptr(x), rows, row_elems, rot_offset, rot_dim, rows_per_pos, _ptr(pos), rope_base,
                     torch.cuda.current_stream(x.device).cuda_stream)
    if st:
        raise KvattnError(st, "kvattn_rope")


def head_proj_tensor(x, w, out_fp32=False):
    """y[r, h] = x[r, h] @ w[h] for bf16 x [rows][H][k] and w [H][k][n] on the
    device (kvattn_head_proj); returns y [rows][H][n]."""
    import torch
    assert x.dtype == torch.bfloat16 and w.dtype == torch.bfloat16 and x.is_contiguous() and w.is_contiguous()
    rows, heads, k = x.shape
    n = w.shape[2]
    assert w.shape[:2] == (heads, k)
    y = torch.empty((rows, heads, n), dtype=torch.float32 if out_fp32 else torch.bfloat16, device=x.device)
    st = kvattn_head_proj(_ptr(x), _ptr(w), _ptr(y), KVATTN_OUT_FP32 if out_fp32 else KVATTN_OUT_BF16, rows,
                          heads, k, n, None, torch.cuda.current_stream(x.device).cuda_stream)
    if st:
        raise KvattnError(st, "kvattn_head_proj")
    return y


# ------------------------------------------------------- the prompt side

def kvattn_build_tables(batch, max_pages_per_seq, num_pages, max_tokens, cached_lens, new_lens, free_pages, free_count,
                        block_table, seq_lens, free_left, q_start, kv_start, pos, slots, device_error=None,
                        stream=0) -> int:
    return load().kvattn_build_tables(int(batch), int(max_pages_per_seq), int(num_pages), int(max_tokens), cached_lens,
                                      new_lens, free_pages, free_count, block_table, seq_lens, free_left, q_start,
                                      kv_start, pos, slots, device_error, stream)


def kvattn_append_slots(variant, params, new_kv, num_tokens, pos, slots, kv_cache, rope_base, device_error=None,
                        stream=0) -> int:
    return load().kvattn_append_slots(int(variant), ctypes.byref(params), new_kv, int(num_tokens), pos, slots, kv_cache,
                                      float(rope_base), device_error, stream)


def kvattn_expand_workspace_size(variant, params, max_kv_tokens) -> int:
    n = ctypes.c_size_t(0)
    st = load().kvattn_expand_workspace_size(int(variant), ctypes.byref(params), int(max_kv_tokens), ctypes.byref(n))
    if st:
        raise KvattnError(st, "kvattn_expand_workspace_size")
    return n.value


def kvattn_expand_kv(variant, params, kv_cache, block_table, kv_start, max_kv_tokens, d_k, d_v, w_uk, w_uv, k_nope, v,
                     k_rope, workspace, workspace_bytes, device_error=None, stream=0) -> int:
    return load().kvattn_expand_kv(int(variant), ctypes.byref(params), kv_cache, block_table, kv_start,
                                   int(max_kv_tokens), int(d_k), int(d_v), w_uk, w_uv, k_nope, v, k_rope, workspace,
                                   int(workspace_bytes), device_error, stream)


def kvattn_prefill_workspace_size(params) -> int:
    n = ctypes.c_size_t(0)
    st = load().kvattn_prefill_workspace_size(ctypes.byref(params), ctypes.byref(n))
    if st:
        raise KvattnError(st, "kvattn_prefill_workspace_size")
    return n.value


def kvattn_prefill(params, q_nope, q_rope, k_nope, k_rope, v, q_start, kv_start, sm_scale, out, lse, workspace,
                   workspace_bytes, device_error=None, stream=0) -> int:
    return load().kvattn_prefill(ctypes.byref(params), q_nope, q_rope, k_nope, k_rope, v, q_start, kv_start,
                                 float(sm_scale), out, lse, workspace, int(workspace_bytes), device_error, stream)


def _check(t, dtype, dims, index, what):
    """The tensor a helper was given: its type, its axes and its CUDA device's
    number; returns it."""
    if t.dtype is not dtype or t.dim() != dims or t.get_device() != index or index < 0:
        raise ValueError(f"{what}: {dims}-d {dtype} on CUDA device {index} wanted, got {t.dim()}-d {t.dtype} on {t.device}")
    return t


def _dense(t, dtype, dims, index, what):
    if not _check(t, dtype, dims, index, what).is_contiguous():
        raise ValueError(f"{what} is not contiguous")
    return t


def _last_axis(t, dtype, dims, index, what):
    """The strides of a tensor whose last axis is contiguous."""
    s = _check(t, dtype, dims, index, what).stride()
    if s[-1] != 1 or (0 in s and any(x == 0 and n > 1 for x, n in zip(s, t.shape))):
        raise ValueError(f"{what}: the last axis is not contiguous, or an axis is broadcast")
    return s


def _enqueue(what, index, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream, with that device
    current (a kernel runs on the device that is current at its launch).

    The stream and the device are read by torch's own private lookups (in torch
    2.11; a torch without them raises AttributeError here): the public ones
    build objects, 2.3 us of a 9 us call."""
    import torch
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            st = fn(*args, stream)
    if st:
        raise KvattnError(st, what)


def _error_word(t, index):
    import torch
    return None if t is None else _dense(t, torch.int32, 1, index, "device_error").data_ptr()


def build_tables_tensors(cached_lens, new_lens, free_pages, free_count, block_table, max_tokens, device_error=None,
                         inplace=False) -> dict:
    """``kvattn_build_tables`` on int32 tensors: cached_lens and new_lens [B],
    free_pages [num_pages], free_count [1], block_table [B][max pages] (updated
    in place).  Returns block_table, seq_lens, free_left, q_start, kv_start,
    pos and slots.  inplace: seq_lens and free_left are cached_lens and
    free_count, updated (no new lengths are allocated)."""
    import torch
    dev, i32 = cached_lens.get_device(), torch.int32
    _dense(cached_lens, i32, 1, dev, "cached_lens")
    _dense(new_lens, i32, 1, dev, "new_lens")
    _dense(free_pages, i32, 1, dev, "free_pages")
    _dense(free_count, i32, 1, dev, "free_count")
    _dense(block_table, i32, 2, dev, "block_table")
    B, mpps = block_table.shape
    n = int(max_tokens)
    if cached_lens.shape[0] != B or new_lens.shape[0] != B or free_count.shape[0] != 1 or n < 0:
        raise ValueError("cached_lens, new_lens and block_table have one row a request, free_count one value")
    # the outputs share one allocation, pos and slots in front (on 16 bytes)
    sizes = [n, n, B + 1, B + 1] if inplace else [n, n, B + 1, B + 1, B, 1]
    r = cached_lens.new_empty(sum(sizes))
    pos = r.data_ptr()
    slots, q_start, kv_start, end = pos + 4 * n, pos + 8 * n, pos + 8 * n + 4 * B + 4, pos + 8 * n + 8 * B + 8
    if inplace:
        lens, left = cached_lens.data_ptr(), free_count.data_ptr()
    else:
        lens, left = end, end + 4 * B
    _enqueue("kvattn_build_tables", dev, load().kvattn_build_tables, B, mpps, free_pages.shape[0], n,
             cached_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(),
             block_table.data_ptr(), lens, left, q_start, kv_start, pos, slots, _error_word(device_error, dev))
    v = torch.split_with_sizes(r, sizes)
    return dict(block_table=block_table, pos=v[0], slots=v[1], q_start=v[2], kv_start=v[3],
                seq_lens=cached_lens if inplace else v[4], free_left=free_count if inplace else v[5])


def append_slots_tensor(variant, params, new_kv, pos, slots, kv_cache, rope_base, device_error=None) -> None:
    """``kvattn_append_slots`` on tensors: new_kv bf16 [tokens][...], pos and
    slots int32 [tokens], kv_cache the pool (bf16, or e4m3 bytes)."""
    import torch
    dev, variant = kv_cache.get_device(), int(variant)
    fp8 = params.cache_dtype == KVATTN_CACHE_FP8_E4M3
    n = _dense(slots, torch.int32, 1, dev, "slots").shape[0]
    _dense(new_kv, torch.bfloat16, new_kv.dim(), dev, "new_kv")
    if pos is not None and _dense(pos, torch.int32, 1, dev, "pos").shape[0] != n:
        raise ValueError("pos has one position for each slot")
    row = params.num_kv * params.d_nope + params.d_rope
    if variant in (KVATTN_GQA, KVATTN_MQA):
        row *= 2
    if new_kv.numel() != n * row:
        raise ValueError("new_kv has one row for each slot")
    if kv_cache.numel() != params.num_pages * 64 * row or not kv_cache.is_contiguous() or (
            kv_cache.element_size() != 1 if fp8 else kv_cache.dtype is not torch.bfloat16):
        raise ValueError("kv_cache is not the pool that params describe")
    if n:
        _enqueue("kvattn_append_slots", dev, load().kvattn_append_slots, variant, ctypes.byref(params),
                 new_kv.data_ptr(), n, None if pos is None else pos.data_ptr(), slots.data_ptr(), kv_cache.data_ptr(),
                 rope_base, _error_word(device_error, dev))


def expand_kv_tensors(variant, params, kv_cache, block_table, kv_start, w_uk, w_uv, max_kv_tokens,
                      device_error=None) -> dict:
    """``kvattn_expand_kv`` on tensors: w_uk [H][d_k][d_nope], w_uv
    [H][d_nope][d_v] (MLRA: R * d_nope).  Returns k [H][max_kv_tokens][d_k], v
    [H][max_kv_tokens][d_v] (MLRA: H * R blocks) and k_rope
    [max_kv_tokens][d_rope] (None without a rope part)."""
    import torch
    dev, bf16 = kv_cache.get_device(), torch.bfloat16
    H, dn, dr, B, n = params.num_q_heads, params.d_nope, params.d_rope, params.batch, int(max_kv_tokens)
    if _dense(kv_cache, bf16, kv_cache.dim(), dev, "kv_cache").numel() != params.num_pages * 64 * (
            params.num_kv * dn + dr):
        raise ValueError("kv_cache is not the pool that params describe")
    h1, d_k, c1 = _dense(w_uk, bf16, 3, dev, "w_uk").shape
    h2, c2, d_v = _dense(w_uv, bf16, 3, dev, "w_uv").shape
    R = params.num_kv if int(variant) == KVATTN_MLRA else 1
    if h1 != H or h2 != H or c1 != R * dn or c2 != R * dn or _dense(kv_start, torch.int32, 1, dev, "kv_start").numel() != B + 1:
        raise ValueError("w_uk is [H][d_k][d_nope], w_uv [H][d_nope][d_v] (MLRA: R * d_nope), kv_start [batch + 1]")
    if block_table is not None and _dense(block_table, torch.int32, 2, dev, "block_table").shape != (
            B, params.max_pages_per_seq):
        raise ValueError("block_table is [batch][max_pages_per_seq]")
    k, v = kv_cache.new_empty((H * R, n, d_k)), kv_cache.new_empty((H * R, n, d_v))
    k_rope = kv_cache.new_empty((n, dr)) if dr else None
    if n:
        ws_bytes = kvattn_expand_workspace_size(variant, params, n)
        ws = kv_cache.new_empty(ws_bytes // 2) if ws_bytes else None
        _enqueue("kvattn_expand_kv", dev, load().kvattn_expand_kv, int(variant), ctypes.byref(params),
                 kv_cache.data_ptr(), _ptr(block_table), kv_start.data_ptr(), n, d_k, d_v, w_uk.data_ptr(),
                 w_uv.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(k_rope), _ptr(ws), ws_bytes,
                 _error_word(device_error, dev))
    return dict(k=k, v=v, k_rope=k_rope)


def prefill_tensors(q_nope, q_rope, k, k_rope, v, q_start, kv_start, sm_scale, causal=True, out=None, lse=None,
                    out_fp32=False, device_error=None) -> dict:
    """``kvattn_prefill`` on bf16 tensors: q_nope [T][H][d_nope] (or fewer
    heads, that divide H), q_rope [T][H][d_rope] or None, k [KH][Tk][d_nope], v [KH][Tk][d_v], k_rope
    [Tk][d_rope] or None, in any strides with a contiguous last axis (keys laid
    out token by token: ``k.transpose(0, 1)``); q_start and kv_start int32
    [B + 1].  Returns out [T][H][d_v] and lse [T][H]; rows past the last
    sequence are left as they were."""
    import torch
    dev, bf16 = q_nope.get_device(), torch.bfloat16
    rope = q_rope is not None
    if rope != (k_rope is not None):
        raise ValueError("q_rope and k_rope go together")
    qs = _last_axis(q_nope, bf16, 3, dev, "q_nope")
    ks = _last_axis(k, bf16, 3, dev, "k")
    vs = _last_axis(v, bf16, 3, dev, "v")
    (T, H, dn), (KH, Tk, d_v) = q_nope.shape, v.shape
    QH = H
    B = _dense(q_start, torch.int32, 1, dev, "q_start").numel() - 1
    if k.shape != (KH, Tk, dn) or _dense(kv_start, torch.int32, 1, dev, "kv_start").numel() != B + 1:
        raise ValueError("the shapes of queries, keys, values and starts do not fit together")
    dr, rs, krs = 0, (0, 0), 0
    if rope:
        rs, krs = _last_axis(q_rope, bf16, 3, dev, "q_rope"), _last_axis(k_rope, bf16, 2, dev, "k_rope")[0]
        t2, H, dr = q_rope.shape
        if t2 != T or k_rope.shape != (Tk, dr):
            raise ValueError("the shapes of queries, keys, values and starts do not fit together")
    dtype = torch.float32 if out_fp32 else bf16
    if out is None:
        out, os = q_nope.new_empty((T, H, d_v), dtype=dtype), (0, 0)
    else:
        os = _last_axis(out, dtype, 3, dev, "out")
        if out.shape != (T, H, d_v):
            raise ValueError("out is [T][H][d_v]")
    if lse is None:
        lse = q_nope.new_empty((T, H), dtype=torch.float32)
    elif _dense(lse, torch.float32, 2, dev, "lse").shape != (T, H):
        raise ValueError("lse is [T][H]")
    if T:
        # an axis of one element has no stride of its own
        t1, h1, qh1, k1, kh1 = T > 1, H > 1, QH > 1, Tk > 1, KH > 1
        p = kvattn_prefill_params(B, H, KH, dn, dr, d_v, T, Tk, 1 if causal else 0,
                                  KVATTN_OUT_FP32 if out_fp32 else KVATTN_OUT_BF16, QH, (qs[0] * t1, qs[1] * qh1),
                                  (rs[0] * t1, rs[1] * h1), (ks[1] * k1, ks[0] * kh1), (vs[1] * k1, vs[0] * kh1),
                                  (os[0] * t1, os[1] * h1), krs * k1)
        ws_bytes = kvattn_prefill_workspace_size(p)
        ws = q_nope.new_empty(ws_bytes // 2) if ws_bytes else None
        _enqueue("kvattn_prefill", dev, load().kvattn_prefill, ctypes.byref(p), q_nope.data_ptr(), _ptr(q_rope),
                 k.data_ptr(), _ptr(k_rope), v.data_ptr(), q_start.data_ptr(), kv_start.data_ptr(), sm_scale,
                 out.data_ptr(), lse.data_ptr(), _ptr(ws), ws_bytes, _error_word(device_error, dev))
    return dict(out=out, lse=lse)
