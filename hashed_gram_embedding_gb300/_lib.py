"""ctypes binding of libple (the C ABI declared in include/ple.h).

Argument marshalling only: every step of the path runs in libple's CUDA
kernels. Functions take torch tensors for device buffers (their data
pointers are passed through) and raise PleError on a non-OK status. There is
no fallback: if libple.so is missing the first call raises.
"""

import ctypes
import os

import numpy as np
import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libple.so")

PLE_OK = 0
PLE_ERR_INVALID_ARG = 1
PLE_ERR_UNSUPPORTED = 2
PLE_ERR_CUDA = 3
PLE_ERR_TIMEOUT = 4
PLE_ERR_BOUNDS = 5
STATUS_NAMES = {0: "PLE_OK", 1: "PLE_ERR_INVALID_ARG", 2: "PLE_ERR_UNSUPPORTED",
                3: "PLE_ERR_CUDA", 4: "PLE_ERR_TIMEOUT", 5: "PLE_ERR_BOUNDS"}

PLE_DEVERR_BOUNDS = 1
PLE_DEVERR_QSL = 2
PLE_DEVERR_TIMEOUT = 4

PLE_BF16 = 0
PLE_FP8_E4M3 = 1
PLE_FP8_E4M3_TENSOR = 2
PLE_HBM = 0
PLE_HOST_UVA = 1
PLE_SHARD_HEADS = 0
PLE_SHARD_ROWS = 1
PLE_HOST_TABLE_REGISTER = 1
PLE_SILU = 0
PLE_GELU = 1

# Every entry point of include/ple.h with its ctypes signature.
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F32 = ctypes.c_float
_I64P = ctypes.POINTER(ctypes.c_int64)
_I32P = ctypes.POINTER(ctypes.c_int32)
SIGNATURES = {
    "ple_ngram_ids": [_P, _I64, _P, _I32, _P, _I32, _I64P, _I64P, _I64P, _I32, _I32, _P, _P, _P, _P],
    "ple_lookup": [_P, _I64, _I32, _P, _I64, _I32, ctypes.c_int, _P, ctypes.c_int, _P, _I32, _P, _P],
    "ple_ngram_lookup": [_P, _I64, _P, _I32, _P, _I32, _I64P, _I64P, _I64P, _I32, _I32, _P, _I64,
                         _I32, ctypes.c_int, _P, ctypes.c_int, _P, _P, _P, _I32, _P, _P],
    "ple_lookup_prefetch": [_P, _I64, _I32, _P, _I64, _I32, ctypes.c_int, _P, ctypes.c_int, _P, _I32,
                            _P, _P, _P],
    "ple_lookup_ordered_workspace": [_I64, _I32, _I64, _I32, ctypes.c_int],
    "ple_lookup_ordered": [_P, _I64, _I32, _P, _I64, _I32, ctypes.c_int, _P, ctypes.c_int, _P, _I32,
                           _P, ctypes.c_size_t, _P, _P],
    "ple_lookup_ordered_static": [_P, _I64, _I32, _P, _I64, _I32, ctypes.c_int, _P, ctypes.c_int, _P,
                                  _I32, _P, _P],
    "ple_lookup_shard": [_P, _I64, _I32, _I32, _I32, _P, _I64, _I64, _I32, ctypes.c_int, _P,
                         ctypes.c_int, ctypes.c_int, _P, _P, _I32, _P, _P],
    "ple_select_rows": [_P, _I32, _I64, _I32, _P, _I64, _I64, _I32, _I32P, _I32P, _I32,
                        ctypes.c_int, _P, _P],
    "ple_wait": [_P, _P, _I32],
    "ple_kv_proj": [_P, _P, _I64, _I32, _I32, _P, _P, _P],
    "ple_kv_proj_gate_workspace": [_I64, _I32],
    "ple_kv_proj_gate": [_P, _P, _I64, _I32, _I32, _P, _P, _P, _F32, _P, _P, _P, ctypes.c_size_t,
                         _P, _P],
    "ple_gate": [_P, _P, _P, _P, _F32, _I64, _I32, _P, _P, _P],
    "ple_conv": [_P, _P, _I32, _I64, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P],
    "ple_gate_conv": [_P, _P, _P, _P, _F32, _P, _I32, _I64, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P, _P],
    "ple_gated_conv": [_P, _P, _P, _I32, _I64, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P],
    "ple_host_table_alloc": [ctypes.c_size_t, ctypes.POINTER(ctypes.c_void_p)],
    "ple_host_table_free": [ctypes.c_void_p, ctypes.c_size_t],
    "ple_host_table_create_shared": [ctypes.c_char_p, ctypes.c_size_t, _I32,
                                     ctypes.POINTER(ctypes.c_void_p)],
    "ple_host_table_attach_shared": [ctypes.c_char_p, ctypes.c_size_t, _I32,
                                     ctypes.POINTER(ctypes.c_void_p)],
    "ple_host_table_unlink_shared": [ctypes.c_char_p],
    "ple_host_table_map_file": [ctypes.c_char_p, ctypes.c_size_t, _I32,
                                ctypes.POINTER(ctypes.c_void_p)],
    "ple_host_table_unmap": [ctypes.c_void_p, ctypes.c_size_t, _I32],
    "ple_graph_begin": [_P],
    "ple_graph_end": [_P, ctypes.POINTER(ctypes.c_void_p)],
    "ple_graph_launch": [_P, _P],
    "ple_graph_destroy": [_P],
    "ple_event_create": [ctypes.POINTER(ctypes.c_void_p)],
    "ple_event_destroy": [_P],
    "ple_event_synchronize": [_P],
    "ple_step_begin": [_P, _P, _P, _I32, _P, _P, _P],
    "ple_step_end": [_P, _P, _P, _I32, _P, _P],
    "ple_step": [_P, _P, _P, _P, _I32, _P, _P, _I32, _P, _P, _P],
    "ple_kv_block_bytes": [_I32],
    "ple_kv_append": [_P, _I64, _P, _I64, _P, _I64, _I64, _I32, _I32, _I32, _P, _I64, _I32, _I32,
                      _P, _P, _I64, _I32, _P, _I32, _P, _I32, _P, _P, _I64, _P, _P],
    "ple_kv_read": [_P, _I64, _I32, _P, _I32, _P, _I32, _P, _I64, _I32, _I32, _P, _P, _P, _P],
    "ple_kv_attention_workspace": [_I32, _I32, _I32],
    "ple_kv_attention": [_P, _I64, _I64, _I32, _I32, _I32, _P, _I64, _I32, _P, _I32, _P, _I32, _P,
                         _I32, _F32, _I32, _I32, _P, _I64, _P, ctypes.c_size_t, _P, _P],
    "ple_proj_w4": [_P, _I64, _I64, _I32, _I32, _P, _P, _P, _I32, _P, _P, _P],
    "ple_mx8_scale_bytes": [_I64, _I32],
    "ple_mx8_read": [_P, _P, _I64, _I32, _P, _P],
    "ple_norm_mx8": [_P, _I64, _P, _I64, _P, _F32, _I64, _I32, _P, _I64, _P, _P, _P],
    "ple_gated_mx8": [_P, _P, _I64, _I32, _P, _P, _I32, _I32, _P, _P, _P, _P],
    "ple_proj_mx8": [_P, _P, _I64, _I32, _P, _P, _I32, _P, _I64, _P, _P, _P],
    "ple_last_error": [],
    "ple_version": [],
}
_VOID = ("ple_graph_destroy", "ple_event_destroy")


class PleCopy(ctypes.Structure):
    """ple_copy: one host<->device copy of the step runtime."""
    _fields_ = [("dst", ctypes.c_void_p), ("src", ctypes.c_void_p), ("bytes", ctypes.c_size_t)]


class PleError(RuntimeError):
    def __init__(self, func, status, detail):
        self.status = status
        super().__init__(f"{func} -> {STATUS_NAMES.get(status, status)}: {detail}")


_lib = None


def lib():
    """The loaded libple (built in-tree); raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m hashed_gram_embedding_gb300.build` (there is no non-CUDA path)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, args in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = (ctypes.c_char_p if name in ("ple_last_error", "ple_version") else
                          ctypes.c_size_t if name.endswith(("_workspace", "_bytes")) else
                          None if name in _VOID else ctypes.c_int)
        _lib = handle
    return _lib


def _check(name, status):
    if status != PLE_OK:
        detail = lib().ple_last_error().decode(errors="replace")
        raise PleError(name, status, detail)
    return status


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _i64_array(values):
    a = np.ascontiguousarray(np.asarray(values, dtype=np.int64))
    return a, a.ctypes.data_as(_I64P)


def ple_ngram_ids(input_ids, query_start_loc, ngram_context, layer_multipliers,
                  vocab_sizes, offsets, eos_token_id, heads_per_ngram, out,
                  ngram_context_out=None, dev_err=None, stream=None):
    """Device tensors: input_ids int32 [T], query_start_loc int32 [R+1],
    ngram_context int32 [R, L] or None, out int64 [T, H], ngram_context_out
    int32 [R, L] or None, dev_err int32 [1] or None. Host arrays:
    layer_multipliers [L+1], vocab_sizes [H], offsets [H] (int64)."""
    mult, mult_p = _i64_array(layer_multipliers)
    V, V_p = _i64_array(vocab_sizes)
    O, O_p = _i64_array(offsets)
    return _check("ple_ngram_ids", lib().ple_ngram_ids(
        _ptr(input_ids), input_ids.numel(), _ptr(query_start_loc), query_start_loc.numel() - 1,
        _ptr(ngram_context), len(mult) - 1, mult_p, V_p, O_p, int(eos_token_id),
        int(heads_per_ngram), _ptr(out), _ptr(ngram_context_out), _ptr(dev_err), _stream(stream)))


def _fp8_dtype(row_scale):
    """bf16 without a scale; one scale value -> the whole-table-scale fp8
    type (a one-row table means the same either way); else per-row fp8."""
    if row_scale is None:
        return PLE_BF16
    return PLE_FP8_E4M3_TENSOR if row_scale.numel() == 1 else PLE_FP8_E4M3


def _lookup_args(ids, table, row_scale, out, max_ctas, dev_err, loc):
    dtype = _fp8_dtype(row_scale)
    if loc is None:
        loc = PLE_HBM if table.is_cuda else PLE_HOST_UVA
    T, H = ids.shape
    return (_ptr(ids), T, H, _ptr(table), table.shape[0], table.shape[1], dtype, _ptr(row_scale),
            loc, _ptr(out), int(max_ctas), _ptr(dev_err))


def ple_lookup(ids, table, out, row_scale=None, max_ctas=0, dev_err=None, loc=None, stream=None):
    """ids int64 [T, H]; table [rows, D] bf16 (or uint8 e4m3 codes with
    row_scale float32 [rows], or [1] for one scale for the whole table), on
    the device or pinned on the host; out bf16 [T, H*D]."""
    return _check("ple_lookup", lib().ple_lookup(
        *_lookup_args(ids, table, row_scale, out, max_ctas, dev_err, loc), _stream(stream)))


def ple_ngram_lookup(input_ids, query_start_loc, ngram_context, layer_multipliers, vocab_sizes,
                     offsets, eos_token_id, heads_per_ngram, table, out, row_scale=None,
                     ids_out=None, ngram_context_out=None, max_ctas=0, dev_err=None, loc=None,
                     stream=None):
    """ple_ngram_ids + ple_lookup in one kernel: out bf16 [T, H*D] gets the
    rows of the hashed ids (ids_out int64 [T, H] also gets the ids when
    given). Other arguments as in ple_ngram_ids and ple_lookup."""
    mult, mult_p = _i64_array(layer_multipliers)
    V, V_p = _i64_array(vocab_sizes)
    O, O_p = _i64_array(offsets)
    if loc is None:
        loc = PLE_HBM if table.is_cuda else PLE_HOST_UVA
    return _check("ple_ngram_lookup", lib().ple_ngram_lookup(
        _ptr(input_ids), input_ids.numel(), _ptr(query_start_loc), query_start_loc.numel() - 1,
        _ptr(ngram_context), len(mult) - 1, mult_p, V_p, O_p, int(eos_token_id),
        int(heads_per_ngram), _ptr(table), table.shape[0], table.shape[1], _fp8_dtype(row_scale),
        _ptr(row_scale), loc, _ptr(out), _ptr(ids_out), _ptr(ngram_context_out), int(max_ctas),
        _ptr(dev_err), _stream(stream)))


def ple_lookup_ordered_workspace(num_tokens, num_heads, table, row_scale=None):
    """Bytes of device workspace ple_lookup_ordered needs."""
    dtype = _fp8_dtype(row_scale)
    return int(lib().ple_lookup_ordered_workspace(int(num_tokens), int(num_heads),
                                                  table.shape[0], table.shape[1], dtype))


def ple_lookup_ordered(ids, table, out, workspace, row_scale=None, max_ctas=0, dev_err=None,
                       loc=None, stream=None):
    """ple_lookup with the rows read in table order; workspace: a device
    uint8 tensor of at least ple_lookup_ordered_workspace(...) bytes."""
    a = _lookup_args(ids, table, row_scale, out, max_ctas, dev_err, loc)
    return _check("ple_lookup_ordered", lib().ple_lookup_ordered(
        *a[:-1], _ptr(workspace), workspace.numel() * workspace.element_size(), a[-1],
        _stream(stream)))


def ple_lookup_ordered_static(ids, table, out, row_scale=None, max_ctas=0, dev_err=None,
                              loc=None, stream=None):
    """ple_lookup_ordered with the library's fixed per-device scratch (no
    workspace, no allocation); calls in flight at once must not overlap."""
    return _check("ple_lookup_ordered_static", lib().ple_lookup_ordered_static(
        *_lookup_args(ids, table, row_scale, out, max_ctas, dev_err, loc), _stream(stream)))


def ple_lookup_shard(ids, table, out, kind, head_begin=0, num_heads=None, row_base=0,
                     row_scale=None, scale_out=None, max_ctas=0, dev_err=None, loc=None,
                     stream=None):
    """One rank's lookup in a table split over an exchange group.

    ids int64 [T, ids_heads] (global rows); the heads [head_begin,
    head_begin + num_heads) are looked up in ``table`` [rows, D], whose row 0
    is global row ``row_base``. kind PLE_SHARD_HEADS: out bf16 [T, heads*D]
    (fp8 dequantised). kind PLE_SHARD_ROWS: out holds the raw rows (bf16, or
    uint8 e4m3 codes with scale_out float32 [T, heads]); rows owned by other
    ranks are zero."""
    T, ids_heads = ids.shape
    if num_heads is None:
        num_heads = ids_heads - head_begin
    if loc is None:
        loc = PLE_HBM if table.is_cuda else PLE_HOST_UVA
    return _check("ple_lookup_shard", lib().ple_lookup_shard(
        _ptr(ids), T, ids_heads, int(head_begin), int(num_heads), _ptr(table), table.shape[0],
        int(row_base), table.shape[1], _fp8_dtype(row_scale), _ptr(row_scale), loc, int(kind),
        _ptr(out), _ptr(scale_out), int(max_ctas), _ptr(dev_err), _stream(stream)))


def ple_select_rows(src, row_begin, num_tokens, part_of_head, col_of_head, out, src_scale=None,
                    fp8_dtype=PLE_FP8_E4M3, stream=None):
    """out bf16 [num_tokens, H*D] <- rows [row_begin, row_begin + num_tokens)
    of src [parts, rows, part_heads*D] (bf16, or uint8 e4m3 codes with
    src_scale float32 [parts, rows, part_heads]), head h taken from part
    part_of_head[h], column col_of_head[h]."""
    parts, rows, width = src.shape
    H = len(part_of_head)
    D = out.shape[1] // H
    fp8 = src_scale is not None
    P = np.ascontiguousarray(np.asarray(part_of_head, dtype=np.int32))
    K = np.ascontiguousarray(np.asarray(col_of_head, dtype=np.int32))
    return _check("ple_select_rows", lib().ple_select_rows(
        _ptr(src), parts, rows, width // D, _ptr(src_scale), int(row_begin), int(num_tokens), H,
        P.ctypes.data_as(_I32P), K.ctypes.data_as(_I32P), D, fp8_dtype if fp8 else PLE_BF16,
        _ptr(out), _stream(stream)))


def _event_handle(event, stream):
    """Raw cudaEvent_t of a torch.cuda.Event (torch creates it lazily, on the
    first record: record it once on ``stream`` if it does not exist yet)."""
    if event.cuda_event == 0:
        event.record(stream)
    return ctypes.c_void_p(event.cuda_event)


def ple_lookup_prefetch(ids, table, out, side_stream, done_event, row_scale=None, max_ctas=0,
                        dev_err=None, loc=None):
    """ple_lookup on ``side_stream``, then ``done_event`` (torch.cuda.Event) recorded there."""
    done = _event_handle(done_event, side_stream)
    return _check("ple_lookup_prefetch", lib().ple_lookup_prefetch(
        *_lookup_args(ids, table, row_scale, out, max_ctas, dev_err, loc),
        ctypes.c_void_p(side_stream.cuda_stream), done))


def ple_wait(done_event, consumer_stream=None, timeout_ms=0):
    if done_event.cuda_event == 0:
        return PLE_OK  # never recorded: nothing to wait for
    return _check("ple_wait", lib().ple_wait(ctypes.c_void_p(done_event.cuda_event),
                                             _stream(consumer_stream), int(timeout_ms)))


def ple_kv_proj(emb, w, kv, dev_err=None, stream=None):
    """emb bf16 [T, E], w bf16 [2C, E], kv bf16 [T, 2C]."""
    T, E = emb.shape
    return _check("ple_kv_proj", lib().ple_kv_proj(
        _ptr(emb), _ptr(w), T, E, w.shape[0] // 2, _ptr(kv), _ptr(dev_err), _stream(stream)))


def ple_kv_proj_gate_workspace(num_tokens, hidden):
    """Bytes of device workspace ple_kv_proj_gate needs (0: sizes it rejects)."""
    return int(lib().ple_kv_proj_gate_workspace(int(num_tokens), int(hidden)))


def ple_kv_proj_gate(emb, w, hidden, gamma_h, gamma_k, kv, gate_out, workspace, eps=1e-6,
                     dev_err=None, stream=None):
    """Projection with the gate reductions fused: writes kv[:, C:] (v) and
    gate_out [T] float32; kv[:, :C] is left untouched. workspace: a device
    uint8 tensor of at least ple_kv_proj_gate_workspace(T, C) bytes,
    zero-filled before its first use (the call leaves it zeroed)."""
    T, E = emb.shape
    return _check("ple_kv_proj_gate", lib().ple_kv_proj_gate(
        _ptr(emb), _ptr(w), T, E, w.shape[0] // 2, _ptr(hidden), _ptr(gamma_h), _ptr(gamma_k),
        float(eps), _ptr(kv), _ptr(gate_out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_err), _stream(stream)))


def ple_gate(hidden, kv, gamma_h, gamma_k, out, eps=1e-6, gate_out=None, stream=None):
    T, C = hidden.shape
    return _check("ple_gate", lib().ple_gate(
        _ptr(hidden), _ptr(kv), _ptr(gamma_h), _ptr(gamma_k), float(eps), T, C, _ptr(out),
        _ptr(gate_out), _stream(stream)))


def ple_conv(x, query_start_loc, w, dilation, out, conv_state=None, conv_state_out=None,
             dev_err=None, stream=None):
    T, C = x.shape
    return _check("ple_conv", lib().ple_conv(
        _ptr(x), _ptr(query_start_loc), query_start_loc.numel() - 1, T, C, _ptr(w), w.shape[1],
        int(dilation), _ptr(conv_state), _ptr(conv_state_out), _ptr(out), _ptr(dev_err),
        _stream(stream)))


def ple_gate_conv(hidden, kv, gamma_h, gamma_k, query_start_loc, w, dilation, out, eps=1e-6,
                  conv_state=None, conv_state_out=None, gate_out=None, dev_err=None, stream=None):
    """gate_out [T] float32 receives the gate scalars (a fresh buffer is made
    when it is not given: pass one in to avoid the allocation)."""
    T, C = hidden.shape
    if gate_out is None:
        import torch
        gate_out = torch.empty((T,), dtype=torch.float32, device=hidden.device)
    return _check("ple_gate_conv", lib().ple_gate_conv(
        _ptr(hidden), _ptr(kv), _ptr(gamma_h), _ptr(gamma_k), float(eps), _ptr(query_start_loc),
        query_start_loc.numel() - 1, T, C, _ptr(w), w.shape[1], int(dilation), _ptr(conv_state),
        _ptr(conv_state_out), _ptr(out), _ptr(gate_out), _ptr(dev_err), _stream(stream)))


def ple_gated_conv(kv, gate, query_start_loc, w, dilation, out, conv_state=None,
                   conv_state_out=None, dev_err=None, stream=None):
    """Conv of u = bf16(gate * v), v = kv[:, C:]; kv [T, 2C] bf16, gate [T] float32."""
    T, C2 = kv.shape
    return _check("ple_gated_conv", lib().ple_gated_conv(
        _ptr(kv), _ptr(gate), _ptr(query_start_loc), query_start_loc.numel() - 1, T, C2 // 2,
        _ptr(w), w.shape[1], int(dilation), _ptr(conv_state), _ptr(conv_state_out), _ptr(out),
        _ptr(dev_err), _stream(stream)))


# ---- the 4-bit step of the attention block: paged cache, attention, projection ----
#
# These calls are made several times a layer for steps of a few microseconds,
# so their checks read each attribute once and pointers go to ctypes as plain
# integers.

_U8, _I32, _F32, _BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


_one_gpu = None  # whether the process sees no more than one; None: not asked yet


def _same_gpu(*tensors):
    """ValueError unless the tensors (or None) are on the current GPU, where a
    call's kernels go. Called unless there is one GPU, which is_cuda tells as well."""
    global _one_gpu
    if _one_gpu is None:
        _one_gpu = torch.cuda.device_count() <= 1
        if _one_gpu:
            return
    current = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != current:
            raise ValueError(f"all tensors must be on the current device, cuda:{current}; one is on {t.device}")


def _err_word(t):
    if t.dtype is not _I32 or not t.is_cuda or t.numel() < 1:
        raise ValueError("dev_err: a CUDA int32 word is needed")
    return t.data_ptr()


def _raw_stream(stream, t):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _heads(name, t, head_dim=None):
    """Row stride and shape of [T, heads, head_dim] bf16 rows: the heads of a
    row lie together, the rows any distance apart."""
    shape = t.shape
    if t.dtype is not _BF16 or not t.is_cuda or len(shape) != 3:
        raise ValueError(f"{name}: a CUDA bf16 tensor [T, heads, head_dim] is needed")
    T, H, D = shape
    stride, per_head, one = t.stride()
    if (T > 0 and ((one != 1 and D > 1) or (per_head != D and H > 1))) or (head_dim is not None and D != head_dim):
        raise ValueError(f"{name}: heads of {head_dim or D} elements must lie together in a row")
    return (stride if T > 1 else H * D), T, H, D


def _whole(name, t, dtype, dims):
    if t.dtype is not dtype or not t.is_contiguous() or not t.is_cuda or t.dim() != dims:
        raise ValueError(f"{name}: a contiguous CUDA {dtype} tensor of {dims} dimensions is needed")
    return t.data_ptr()


def _cache_args(cache, block_table, query_start_loc, kv_lens, head_dim):
    """Kv heads, and the arguments shared by the cache's calls."""
    if (cache.dtype is not _U8 or block_table.dtype is not _I32 or query_start_loc.dtype is not _I32
            or kv_lens.dtype is not _I32
            or not (cache.is_contiguous() and block_table.is_contiguous() and query_start_loc.is_contiguous()
                    and kv_lens.is_contiguous())
            or not (cache.is_cuda and block_table.is_cuda and query_start_loc.is_cuda and kv_lens.is_cuda)):
        raise ValueError("contiguous CUDA tensors are needed: cache uint8, block_table, query_start_loc and "
                         "kv_lens int32")
    pages, hk, sub, nbytes = cache.shape  # a ValueError, too, where there are more dimensions or fewer
    (rows, max_pages), (bounds,), (R,) = block_table.shape, query_start_loc.shape, kv_lens.shape
    if nbytes != 16 * (head_dim + 8):
        raise ValueError(f"cache: blocks of {nbytes} bytes, not {16 * (head_dim + 8)} (head_dim {head_dim})")
    if rows != R or bounds != R + 1:
        raise ValueError(f"block_table must have a row, and query_start_loc an entry and one more, for "
                         f"each of the {R} requests of kv_lens")
    return hk, (cache.data_ptr(), pages, sub * 16, block_table.data_ptr(), max_pages, query_start_loc.data_ptr(), R,
                kv_lens.data_ptr())


def ple_kv_block_bytes(head_dim):
    """Bytes of a cache block (16 tokens of one head); the cache is a uint8
    tensor [num_pages, num_kv_heads, page_size / 16, block bytes]."""
    return int(lib().ple_kv_block_bytes(int(head_dim)))


def ple_kv_append(q, k, v, cos_sin, cache, block_table, query_start_loc, kv_lens, q_out,
                  positions=None, interleaved=False, dev_err=None, stream=None):
    """Rotate q and k and store k and v in the 4-bit cache. q [T, H, D] (or
    None, with q_out None), k, v [T, Hk, D] bf16 (columns of one fused
    projection will do); cos_sin float32 [num_positions, rotary_dim] or None;
    cache uint8 [pages, Hk, page_size / 16, 16 * (D + 8)]; block_table int32
    [R, max_pages], query_start_loc int32 [R + 1], kv_lens int32 [R] (these
    tokens included); q_out like q, or q itself; positions int32 [T] or None."""
    k_stride, T, Hk, D = _heads("k", k)
    v_stride, Tv, Hv, _ = _heads("v", v, D)
    hk, c = _cache_args(cache, block_table, query_start_loc, kv_lens, D)
    H, q_at, q_stride, o_at, o_stride, Tq = 0, None, 0, None, 0, T
    if q is not None:
        q_stride, Tq, H, _ = _heads("q", q, D)
        o_stride, To, Ho, _ = _heads("q_out", q_out, D)
        if To != Tq or Ho != H:
            raise ValueError("q_out must have q's shape")
        q_at, o_at = q.data_ptr(), q_out.data_ptr()
    if Hk != hk or Hv != hk or Tv != T or Tq != T:
        raise ValueError("q, k, v and the cache differ in tokens or kv heads")
    if not _one_gpu:
        _same_gpu(q, k, v, cos_sin, cache, block_table, query_start_loc, kv_lens, q_out, positions, dev_err)
    cs, entries, rot = None, 0, 0
    if cos_sin is not None:
        cs = _whole("cos_sin", cos_sin, _F32, 2)
        entries, rot = cos_sin.shape
    at = None
    if positions is not None:
        at = _whole("positions", positions, _I32, 1)
        if positions.shape[0] != T:
            raise ValueError("positions must have one entry for each token")
    status = lib().ple_kv_append(
        q_at, q_stride, k.data_ptr(), k_stride, v.data_ptr(), v_stride, T, H, hk, D, cs, entries, rot,
        1 if interleaved else 0, at, *c, o_at, o_stride, None if dev_err is None else _err_word(dev_err),
        _raw_stream(stream, k))
    return status if status == PLE_OK else _check("ple_kv_append", status)


def ple_kv_read(cache, block_table, query_start_loc, kv_lens, k_out, v_out, dev_err=None,
                stream=None):
    """Values of the tokens in query_start_loc's spans out of the 4-bit cache:
    k_out, v_out bf16 [T, Hk, D], contiguous (either may be None)."""
    some = k_out if k_out is not None else v_out
    if some is None:
        raise ValueError("k_out or v_out is needed")
    k_at = None if k_out is None else _whole("k_out", k_out, _BF16, 3)
    v_at = None if v_out is None else _whole("v_out", v_out, _BF16, 3)
    if k_at is not None and v_at is not None and k_out.shape != v_out.shape:
        raise ValueError("k_out and v_out differ in shape")
    T, Hk, D = some.shape
    hk, c = _cache_args(cache, block_table, query_start_loc, kv_lens, D)
    if Hk != hk:
        raise ValueError(f"{Hk} kv heads, and {hk} in the cache")
    if not _one_gpu:
        _same_gpu(cache, block_table, query_start_loc, kv_lens, k_out, v_out, dev_err)
    status = lib().ple_kv_read(*c, T, hk, D, k_at, v_at, None if dev_err is None else _err_word(dev_err),
                               _raw_stream(stream, some))
    return status if status == PLE_OK else _check("ple_kv_read", status)


def ple_kv_attention_workspace(num_heads, num_kv_heads, head_dim):
    """Bytes of device workspace ple_kv_attention needs (0: heads it rejects)."""
    return int(lib().ple_kv_attention_workspace(int(num_heads), int(num_kv_heads), int(head_dim)))


def ple_kv_attention(q, cache, block_table, query_start_loc, kv_lens, out, workspace, scale=None,
                     causal=True, window=0, max_query_len=0, dev_err=None, stream=None):
    """Grouped-query attention of q [T, H, D] bf16 over the 4-bit cache into
    out [T, H, D] bf16. workspace: a device uint8 tensor of at least
    ple_kv_attention_workspace(H, Hk, D) bytes, zero-filled before its first
    use. scale: 1 / sqrt(D) by default; max_query_len: the most query tokens
    of a request, if known (0: not known, which costs batches of single tokens
    several times as long); out may be q. Other arguments as in ple_kv_append."""
    q_stride, T, H, D = _heads("q", q)
    o_stride, To, Ho, _ = _heads("out", out, D)
    if To != T or Ho != H:
        raise ValueError("out must have q's shape")
    hk, c = _cache_args(cache, block_table, query_start_loc, kv_lens, D)
    room = _whole("workspace", workspace, _U8, 1)
    if not _one_gpu:
        _same_gpu(q, cache, block_table, query_start_loc, kv_lens, out, workspace, dev_err)
    status = lib().ple_kv_attention(
        q.data_ptr(), q_stride, T, H, hk, D, *c, max_query_len, D ** -0.5 if scale is None else scale,
        1 if causal else 0, window, out.data_ptr(), o_stride, room, workspace.shape[0],
        None if dev_err is None else _err_word(dev_err), _raw_stream(stream, q))
    return status if status == PLE_OK else _check("ple_kv_attention", status)


def ple_proj_w4(x, codes, scales, out, zeros=None, dev_err=None, stream=None):
    """out [T, N] bf16 = x [T, E] bf16 times the transpose of a 4-bit weight:
    codes uint8 [N, E / 2], scales bf16 [N, E / group], zeros uint8 like
    scales, or None for 8 everywhere."""
    if (x.dtype is not _BF16 or codes.dtype is not _U8 or scales.dtype is not _BF16 or out.dtype is not _BF16
            or not (codes.is_contiguous() and scales.is_contiguous() and out.is_contiguous())
            or not (x.is_cuda and codes.is_cuda and scales.is_cuda and out.is_cuda)):
        raise ValueError("CUDA tensors are needed: x bf16; contiguous codes uint8, scales and out bf16")
    # a ValueError, too, where one has more dimensions or fewer
    (T, E), (Nc, half), (N, groups), (To, No) = x.shape, codes.shape, scales.shape, out.shape
    stride, one = x.stride()
    if one != 1 and E > 1 and T > 0:
        raise ValueError("x: the columns of a row must lie together")
    if Nc != N or half * 2 != E or To != T or No != N or groups < 1 or E % groups != 0:
        raise ValueError(f"x {tuple(x.shape)}, codes {tuple(codes.shape)}, scales "
                         f"{tuple(scales.shape)} and out {tuple(out.shape)} do not fit")
    if not _one_gpu:
        _same_gpu(x, codes, scales, out, zeros, dev_err)
    zero_at = None
    if zeros is not None:
        zero_at = _whole("zeros", zeros, _U8, 2)
        if zeros.shape != scales.shape:
            raise ValueError("zeros must have the shape of scales")
    status = lib().ple_proj_w4(
        x.data_ptr(), stride if T > 1 else E, T, E, N, codes.data_ptr(), scales.data_ptr(), zero_at,
        E // groups, out.data_ptr(),
        None if dev_err is None else _err_word(dev_err), _raw_stream(stream, x))
    return status if status == PLE_OK else _check("ple_proj_w4", status)


# ---- the 8-bit step of the feed-forward block: norm, gated products, projection ----

_ACTIVATIONS = {"silu": PLE_SILU, "gelu": PLE_GELU}
_INT32_MAX = 2 ** 31 - 1


def ple_mx8_scale_bytes(rows, columns):
    """Bytes of the scales of an 8-bit tensor [rows, columns] (0: sizes that
    have none)."""
    rows, columns = int(rows), int(columns)
    if max(abs(rows), abs(columns)) > _INT32_MAX:  # (they would reach the library as what is left in its integers)
        return 0
    return int(lib().ple_mx8_scale_bytes(rows, columns))


def _mx8_error(name, codes, scales):
    """Why codes and scales are no 8-bit tensor."""
    if (codes.dtype is not _U8 or scales.dtype is not _U8 or not (codes.is_contiguous() and scales.is_contiguous())
            or not (codes.is_cuda and scales.is_cuda)):
        return ValueError(f"{name}: contiguous CUDA uint8 tensors are needed, codes [R, C] and scales of one dimension")
    return ValueError(f"{name}: codes {tuple(codes.shape)} (columns: a multiple of 128, below 2^31) and "
                      f"{scales.numel()} bytes of scales do not fit (ple_mx8_scale_bytes)")


def _mx8(name, codes, scales):
    """Shape of an 8-bit tensor: codes uint8 [R, C], scales uint8, their bytes
    in one dimension, as many as ple_mx8_scale_bytes says or more."""
    if (codes.dtype is not _U8 or scales.dtype is not _U8 or not (codes.is_contiguous() and scales.is_contiguous())
            or not (codes.is_cuda and scales.is_cuda)):
        raise _mx8_error(name, codes, scales)
    (R, C), (n,) = codes.shape, scales.shape  # a ValueError, too, where there are more dimensions or fewer
    if C % 128 != 0 or C > _INT32_MAX or n < (R + 127) // 128 * (C * 4):
        raise _mx8_error(name, codes, scales)
    return R, C


def _row_stride(name, t, shape):
    """Distance of bf16 rows that need not lie together."""
    if t.dtype is not _BF16 or not t.is_cuda or t.shape != shape:
        raise ValueError(f"{name}: a CUDA bf16 tensor {tuple(shape)} is needed")
    if t.is_contiguous():
        return shape[1]
    stride, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the columns of a row must lie together")
    return stride if shape[0] > 1 else shape[1]


def ple_mx8_read(codes, scales, out, stream=None):
    """out [R, C] bf16: the values of an 8-bit tensor, codes uint8 [R, C] and
    scales uint8 [ple_mx8_scale_bytes(R, C)]."""
    R, C = _mx8("codes, scales", codes, scales)
    if out.dtype is not _BF16 or not out.is_contiguous() or not out.is_cuda or out.shape != codes.shape:
        raise ValueError("out: a contiguous CUDA bf16 tensor of the shape of codes is needed")
    if not _one_gpu:
        _same_gpu(codes, scales, out)
    status = lib().ple_mx8_read(codes.data_ptr(), scales.data_ptr(), R, C, out.data_ptr(), _raw_stream(stream, codes))
    return status if status == PLE_OK else _check("ple_mx8_read", status)


def ple_norm_mx8(x, gamma, codes, scales, residual=None, sum_out=None, eps=1e-6, stream=None):
    """codes uint8 [T, C] and scales uint8 [ple_mx8_scale_bytes(T, C)]: the
    root-mean-square norm of x + residual, in 8 bits; sum_out: the sum. x,
    residual and sum_out bf16 [T, C], columns of a wider tensor will do;
    sum_out may be x or residual itself. gamma bf16 [C], or None for 1."""
    T, C = _mx8("codes, scales", codes, scales)
    shape = codes.shape
    x_stride = _row_stride("x", x, shape)
    r_at, r_stride, s_at, s_stride, g_at = None, C, None, C, None
    if residual is not None:
        r_at, r_stride = residual.data_ptr(), _row_stride("residual", residual, shape)
    if sum_out is not None:
        s_at, s_stride = sum_out.data_ptr(), _row_stride("sum_out", sum_out, shape)
    if gamma is not None:
        if gamma.dtype is not _BF16 or not gamma.is_contiguous() or not gamma.is_cuda or gamma.shape != shape[1:]:
            raise ValueError(f"gamma: a contiguous CUDA bf16 tensor of {C} entries is needed")
        g_at = gamma.data_ptr()
    if not _one_gpu:
        _same_gpu(x, gamma, codes, scales, residual, sum_out)
    status = lib().ple_norm_mx8(x.data_ptr(), x_stride, r_at, r_stride, g_at, eps, T, C, s_at, s_stride, codes.data_ptr(),
                                scales.data_ptr(), _raw_stream(stream, x))
    return status if status == PLE_OK else _check("ple_norm_mx8", status)


def ple_gated_mx8(x, x_scales, w, w_scales, codes, scales, activation="silu", dev_err=None, stream=None):
    """codes, scales: act(x Wg^T) * (x Wu^T) in 8 bits [T, I], for x in 8 bits
    [T, C] and w in 8 bits [2 I, C], Wg's rows before Wu's. activation: "silu"
    or "gelu" (its tanh form)."""
    T, C = _mx8("x", x, x_scales)
    rows, Cw = _mx8("w", w, w_scales)
    To, I = _mx8("codes, scales", codes, scales)
    if Cw != C or rows != 2 * I or To != T:
        raise ValueError(f"x {tuple(x.shape)}, w {tuple(w.shape)} and codes {tuple(codes.shape)} do not fit")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation {activation!r}: one of {', '.join(_ACTIVATIONS)} is needed")
    if not _one_gpu:
        _same_gpu(x, x_scales, w, w_scales, codes, scales, dev_err)
    status = lib().ple_gated_mx8(
        x.data_ptr(), x_scales.data_ptr(), T, C, w.data_ptr(), w_scales.data_ptr(), I, act, codes.data_ptr(),
        scales.data_ptr(), None if dev_err is None else _err_word(dev_err), _raw_stream(stream, x))
    return status if status == PLE_OK else _check("ple_gated_mx8", status)


def ple_proj_mx8(x, x_scales, w, w_scales, out, residual=None, dev_err=None, stream=None):
    """out [T, N] bf16 = residual + x W^T, for x in 8 bits [T, E] and w in 8
    bits [N, E]. residual bf16 [T, N], columns of a wider tensor will do; it
    may be out itself."""
    T, E = _mx8("x", x, x_scales)
    N, Ew = _mx8("w", w, w_scales)
    if out.dtype is not _BF16 or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out: a contiguous CUDA bf16 tensor is needed")
    shape = out.shape
    if Ew != E or shape != (T, N):
        raise ValueError(f"x {tuple(x.shape)}, w {tuple(w.shape)} and out {tuple(shape)} do not fit")
    r_at, r_stride = None, N
    if residual is not None:
        r_at, r_stride = residual.data_ptr(), _row_stride("residual", residual, shape)
    if not _one_gpu:
        _same_gpu(x, x_scales, w, w_scales, out, residual, dev_err)
    status = lib().ple_proj_mx8(
        x.data_ptr(), x_scales.data_ptr(), T, E, w.data_ptr(), w_scales.data_ptr(), N, r_at, r_stride, out.data_ptr(),
        None if dev_err is None else _err_word(dev_err), _raw_stream(stream, x))
    return status if status == PLE_OK else _check("ple_proj_mx8", status)


def ple_version():
    return lib().ple_version().decode()


class HostTable:
    """A table buffer from ple_host_table_alloc, viewed as a torch tensor.

    Keep this object alive as long as the tensor is used; the memory is
    unregistered and unmapped when it is garbage-collected (or on close()).
    """

    def __init__(self, rows, row_dim, dtype):
        import torch
        elem = torch.empty((), dtype=dtype).element_size()
        self.nbytes = int(rows) * int(row_dim) * elem
        ptr = ctypes.c_void_p()
        _check("ple_host_table_alloc", lib().ple_host_table_alloc(self.nbytes, ctypes.byref(ptr)))
        self.ptr = ptr.value
        buf = (ctypes.c_uint8 * self.nbytes).from_address(self.ptr)
        self.tensor = torch.frombuffer(buf, dtype=torch.uint8).view(dtype).view(int(rows), int(row_dim))

    def close(self):
        if getattr(self, "ptr", None):
            self.tensor = None
            lib().ple_host_table_free(ctypes.c_void_p(self.ptr), self.nbytes)
            self.ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MappedHostTable:
    """A table in a named shared-memory object or a file, mapped by
    ple_host_table_create_shared / _attach_shared / _map_file and viewed as a
    torch tensor [rows, row_dim]; ``register`` makes it readable by the GPU
    over UVA. Unmapped on close() (the shared object itself stays until
    unlink)."""

    def __init__(self, kind, target, rows, row_dim, dtype, register=True):
        import torch
        elem = torch.empty((), dtype=dtype).element_size()
        self.nbytes = int(rows) * int(row_dim) * elem
        self.flags = PLE_HOST_TABLE_REGISTER if register else 0
        fn = {"create": "ple_host_table_create_shared", "attach": "ple_host_table_attach_shared",
              "file": "ple_host_table_map_file"}[kind]
        ptr = ctypes.c_void_p()
        _check(fn, getattr(lib(), fn)(str(target).encode(), self.nbytes, self.flags,
                                      ctypes.byref(ptr)))
        self.ptr = ptr.value
        buf = (ctypes.c_uint8 * self.nbytes).from_address(self.ptr)
        view = torch.frombuffer(buf, dtype=torch.uint8)
        self.tensor = view.view(dtype).view(int(rows), int(row_dim))

    def close(self):
        if getattr(self, "ptr", None):
            self.tensor = None
            lib().ple_host_table_unmap(ctypes.c_void_p(self.ptr), self.nbytes, self.flags)
            self.ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def ple_host_table_unlink_shared(name):
    return _check("ple_host_table_unlink_shared", lib().ple_host_table_unlink_shared(name.encode()))


# ---- step runtime (graph capture, events, one step over three streams) ----

def copies(items):
    """PleCopy array of (dst, src, bytes) triples (pointers as ints)."""
    arr = (PleCopy * max(len(items), 1))()
    for i, (dst, src, nbytes) in enumerate(items):
        arr[i].dst, arr[i].src, arr[i].bytes = dst, src, nbytes
    return arr


def ple_graph_begin(stream):
    _check("ple_graph_begin", lib().ple_graph_begin(_stream(stream)))


def ple_graph_end(stream):
    """End the capture begun on ``stream``; returns the graph handle (int)."""
    g = ctypes.c_void_p()
    _check("ple_graph_end", lib().ple_graph_end(_stream(stream), ctypes.byref(g)))
    return g.value


def ple_graph_launch(graph, stream):
    _check("ple_graph_launch", lib().ple_graph_launch(graph, _stream(stream)))


def ple_graph_destroy(graph):
    lib().ple_graph_destroy(graph)


def ple_event_create():
    ev = ctypes.c_void_p()
    _check("ple_event_create", lib().ple_event_create(ctypes.byref(ev)))
    return ev.value


def ple_event_destroy(event):
    lib().ple_event_destroy(event)


def ple_event_synchronize(event):
    _check("ple_event_synchronize", lib().ple_event_synchronize(event))


def ple_step_begin(copy_in, compute, uploads, num_uploads, loaded, computed, returned):
    _check("ple_step_begin", lib().ple_step_begin(_stream(copy_in), _stream(compute), uploads,
                                                  num_uploads, loaded, computed, returned))


def ple_step_end(compute, copy_out, downloads, num_downloads, computed, returned):
    _check("ple_step_end", lib().ple_step_end(_stream(compute), _stream(copy_out), downloads,
                                              num_downloads, computed, returned))


def ple_step(copy_in, compute, copy_out, uploads, num_uploads, graph, downloads, num_downloads,
             loaded, computed, returned):
    _check("ple_step", lib().ple_step(_stream(copy_in), _stream(compute), _stream(copy_out),
                                      uploads, num_uploads, graph, downloads, num_downloads,
                                      loaded, computed, returned))
