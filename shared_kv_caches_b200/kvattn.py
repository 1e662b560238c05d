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
        "causal", "out_dtype")] + [(n, ctypes.c_int64 * 2) for n in (
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


def _check(t, dtypes, dims, device, what):
    """The tensor a helper was given: its type, its axes and its device."""
    if t.dtype not in dtypes or t.dim() != dims or t.device != device:
        raise ValueError(f"{what}: {dims}-d {' or '.join(str(d) for d in dtypes)} on {device} wanted, "
                         f"got {t.dim()}-d {t.dtype} on {t.device}")
    return t


def _launch(device):
    """The device's guard and its current stream (a kernel runs on the device
    that is current when it is launched)."""
    import torch
    return torch.cuda.device(device), torch.cuda.current_stream(device).cuda_stream


def build_tables_tensors(cached_lens, new_lens, free_pages, free_count, block_table, max_tokens, device_error=None,
                         inplace=False) -> dict:
    """``kvattn_build_tables`` on int32 tensors: cached_lens and new_lens [B],
    free_pages [num_pages], free_count [1], block_table [B][max pages] (updated
    in place).  Returns block_table, seq_lens, free_left, q_start, kv_start,
    pos and slots.  inplace: seq_lens and free_left are cached_lens and
    free_count, updated (no new lengths are allocated)."""
    import torch
    dev, i32 = cached_lens.device, (torch.int32,)
    for t, dims, what in ((cached_lens, 1, "cached_lens"), (new_lens, 1, "new_lens"), (free_pages, 1, "free_pages"),
                          (free_count, 1, "free_count"), (block_table, 2, "block_table")):
        if not _check(t, i32, dims, dev, what).is_contiguous():
            raise ValueError(f"{what} is not contiguous")
    B = cached_lens.shape[0]
    if new_lens.shape[0] != B or block_table.shape[0] != B or free_count.numel() != 1:
        raise ValueError("cached_lens, new_lens and block_table have one row a request, free_count one value")
    guard, stream = _launch(dev)

    def new(n):
        return torch.empty(n, dtype=torch.int32, device=dev)
    r = dict(block_table=block_table, seq_lens=cached_lens if inplace else new(B),
             free_left=free_count if inplace else new(1), q_start=new(B + 1), kv_start=new(B + 1),
             pos=new(max_tokens), slots=new(max_tokens))
    with guard:
        st = kvattn_build_tables(B, block_table.shape[1], free_pages.shape[0], max_tokens, _ptr(cached_lens),
                                 _ptr(new_lens), _ptr(free_pages), _ptr(free_count), _ptr(block_table),
                                 _ptr(r["seq_lens"]), _ptr(r["free_left"]), _ptr(r["q_start"]), _ptr(r["kv_start"]),
                                 _ptr(r["pos"]), _ptr(r["slots"]), _ptr(device_error), stream)
    if st:
        raise KvattnError(st, "kvattn_build_tables")
    return r


def append_slots_tensor(variant, params, new_kv, pos, slots, kv_cache, rope_base, device_error=None) -> None:
    """``kvattn_append_slots`` on tensors: new_kv bf16 [tokens][...], pos and
    slots int32 [tokens], kv_cache the pool (bf16, or e4m3 bytes)."""
    import torch
    dev = kv_cache.device
    _check(slots, (torch.int32,), 1, dev, "slots")
    _check(new_kv, (torch.bfloat16,), new_kv.dim(), dev, "new_kv")
    if pos is not None:
        _check(pos, (torch.int32,), 1, dev, "pos")
    n = slots.shape[0]
    variant = int(variant)
    row = params.num_kv * params.d_nope + params.d_rope
    row *= 2 if variant in (KVATTN_GQA, KVATTN_MQA) else 1
    if new_kv.numel() != n * row or (pos is not None and pos.shape[0] != n):
        raise ValueError("new_kv has one row, and pos one position, for each slot")
    if kv_cache.numel() != params.num_pages * 64 * row or kv_cache.element_size() != (
            1 if params.cache_dtype == KVATTN_CACHE_FP8_E4M3 else 2):
        raise ValueError("kv_cache is not the pool that params describe")
    for t, what in ((new_kv, "new_kv"), (slots, "slots"), (kv_cache, "kv_cache")) + (
            () if pos is None else ((pos, "pos"),)):
        if not t.is_contiguous():
            raise ValueError(f"{what} is not contiguous")
    if n == 0:
        return
    guard, stream = _launch(dev)
    with guard:
        st = kvattn_append_slots(variant, params, _ptr(new_kv), n, _ptr(pos), _ptr(slots), _ptr(kv_cache), rope_base,
                                 _ptr(device_error), stream)
    if st:
        raise KvattnError(st, "kvattn_append_slots")


def expand_kv_tensors(variant, params, kv_cache, block_table, kv_start, w_uk, w_uv, max_kv_tokens,
                      device_error=None) -> dict:
    """``kvattn_expand_kv`` on tensors: w_uk [H][d_k][d_nope], w_uv
    [H][d_nope][d_v].  Returns k [H][max_kv_tokens][d_k], v
    [H][max_kv_tokens][d_v] and k_rope [max_kv_tokens][d_rope] (None without a
    rope part)."""
    import torch
    dev, bf16 = kv_cache.device, (torch.bfloat16,)
    H, dn, dr, n = params.num_q_heads, params.d_nope, params.d_rope, int(max_kv_tokens)
    _check(kv_cache, bf16, kv_cache.dim(), dev, "kv_cache")
    _check(w_uk, bf16, 3, dev, "w_uk")
    _check(w_uv, bf16, 3, dev, "w_uv")
    _check(kv_start, (torch.int32,), 1, dev, "kv_start")
    d_k, d_v = w_uk.shape[1], w_uv.shape[2]
    if w_uk.shape != (H, d_k, dn) or w_uv.shape != (H, dn, d_v) or kv_start.shape[0] != params.batch + 1:
        raise ValueError("w_uk is [H][d_k][d_nope], w_uv [H][d_nope][d_v], kv_start [batch + 1]")
    if kv_cache.numel() != params.num_pages * 64 * (params.num_kv * dn + dr):
        raise ValueError("kv_cache is not the pool that params describe")
    if block_table is not None and _check(block_table, (torch.int32,), 2, dev, "block_table").shape != (
            params.batch, params.max_pages_per_seq):
        raise ValueError("block_table is [batch][max_pages_per_seq]")
    for t, what in ((kv_cache, "kv_cache"), (w_uk, "w_uk"), (w_uv, "w_uv"), (kv_start, "kv_start")) + (
            () if block_table is None else ((block_table, "block_table"),)):
        if not t.is_contiguous():
            raise ValueError(f"{what} is not contiguous")

    def new(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=dev)
    r = dict(k=new(H, n, d_k), v=new(H, n, d_v), k_rope=new(n, dr) if dr else None)
    ws = torch.empty(kvattn_expand_workspace_size(variant, params, n), dtype=torch.uint8, device=dev)
    if n == 0:
        return r
    guard, stream = _launch(dev)
    with guard:
        st = kvattn_expand_kv(variant, params, _ptr(kv_cache), _ptr(block_table), _ptr(kv_start), n, d_k, d_v,
                              _ptr(w_uk), _ptr(w_uv), _ptr(r["k"]), _ptr(r["v"]), _ptr(r["k_rope"]), _ptr(ws),
                              ws.numel(), _ptr(device_error), stream)
    if st:
        raise KvattnError(st, "kvattn_expand_kv")
    return r


def prefill_tensors(q_nope, q_rope, k, k_rope, v, q_start, kv_start, sm_scale, causal=True, out=None, lse=None,
                    out_fp32=False, device_error=None) -> dict:
    """``kvattn_prefill`` on bf16 tensors: q_nope [T][H][d_nope], q_rope
    [T][H][d_rope] or None, k [KH][Tk][d_nope], v [KH][Tk][d_v], k_rope
    [Tk][d_rope] or None, in any strides with a contiguous last axis (keys laid
    out token by token: ``k.transpose(0, 1)``); q_start and kv_start int32
    [B + 1].  Returns out [T][H][d_v] and lse [T][H]; rows past the last
    sequence are left as they were."""
    import torch
    dev, bf16 = q_nope.device, (torch.bfloat16,)
    for t, dims, what in ((q_nope, 3, "q_nope"), (k, 3, "k"), (v, 3, "v")) + (
            () if q_rope is None else ((q_rope, 3, "q_rope"), (k_rope, 2, "k_rope"))):
        if _check(t, bf16, dims, dev, what).shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{what}: the last axis is not contiguous")
    for t, what in ((q_start, "q_start"), (kv_start, "kv_start")):
        if not _check(t, (torch.int32,), 1, dev, what).is_contiguous():
            raise ValueError(f"{what} is not contiguous")
    (T, H, dn), (KH, Tk, d_v), B = q_nope.shape, v.shape, q_start.shape[0] - 1
    dr = 0 if q_rope is None else q_rope.shape[2]
    if k.shape != (KH, Tk, dn) or kv_start.shape[0] != B + 1 or (
            dr and (q_rope.shape != (T, H, dr) or k_rope.shape != (Tk, dr))) or (q_rope is None) != (k_rope is None):
        raise ValueError("the shapes of queries, keys, values and starts do not fit together")
    if out is None:
        out = torch.empty((T, H, d_v), dtype=torch.float32 if out_fp32 else torch.bfloat16, device=dev)
    elif _check(out, (torch.bfloat16, torch.float32), 3, dev, "out").shape != (T, H, d_v) or out.stride(-1) != 1:
        raise ValueError("out is [T][H][d_v] with a contiguous last axis")
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    elif _check(lse, (torch.float32,), 2, dev, "lse").shape != (T, H) or not lse.is_contiguous():
        raise ValueError("lse is [T][H]")
    r = dict(out=out, lse=lse)
    if T == 0:
        return r

    def steps(t, token, head):
        return (ctypes.c_int64 * 2)(t.stride(token), t.stride(head))
    p = kvattn_prefill_params(B, H, KH, dn, dr, d_v, T, Tk, 1 if causal else 0,
                              KVATTN_OUT_FP32 if out.dtype == torch.float32 else KVATTN_OUT_BF16, steps(q_nope, 0, 1),
                              steps(q_rope, 0, 1) if dr else steps(q_nope, 0, 1), steps(k, 1, 0), steps(v, 1, 0),
                              steps(out, 0, 1), k_rope.stride(0) if dr else 0)
    ws = torch.empty(kvattn_prefill_workspace_size(p), dtype=torch.uint8, device=dev)
    guard, stream = _launch(dev)
    with guard:
        st = kvattn_prefill(p, _ptr(q_nope), _ptr(q_rope), _ptr(k), _ptr(k_rope), _ptr(v), _ptr(q_start),
                            _ptr(kv_start), sm_scale, _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _ptr(device_error),
                            stream)
    if st:
        raise KvattnError(st, "kvattn_prefill")
    return r
