"""ctypes binding of libpa.so: the C ABI's entry points under the same names.

Argument marshalling only -- torch tensors become device pointers, sizes and
the current CUDA stream; every step of the path runs in the library's CUDA
kernels.  There is no fallback: if the library is missing the first call
raises, and every non-OK status raises PAError with the library's reason.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libpa.so")

PA_F32, PA_BF16, PA_F16, PA_FP8_E4M3 = 0, 1, 2, 3
PA_OPT_CHECK_MODE, PA_OPT_DECODE_KERNEL, PA_OPT_DECODE_CTAS, PA_OPT_VARLEN_KERNEL, PA_OPT_FP8_PAIR_STEP = 0, 1, 2, 3, 4
DTYPE_CODE = {torch.float32: PA_F32, torch.bfloat16: PA_BF16, torch.float16: PA_F16}
# pools that only move bytes (copy, swap) may also hold E4M3 codes
POOL_DTYPE_CODE = {**DTYPE_CODE, torch.uint8: PA_FP8_E4M3, torch.float8_e4m3fn: PA_FP8_E4M3}

EXPORTS = ("pa_status_string", "pa_last_error", "pa_set_option", "pa_get_option", "pa_set_check_mode",
           "pa_device_status", "pa_slot_mapping", "pa_write_kv", "pa_copy_blocks", "pa_decode_workspace_size",
           "pa_decode", "pa_decode_append", "pa_varlen_workspace_size", "pa_varlen", "pa_decode_noalloc",
           "pa_swap_blocks", "pa_write_kv_fp8", "pa_decode_fp8_workspace_size", "pa_decode_fp8",
           "pa_decode_append_fp8", "pa_selftest_wait_timeout", "pa_varlen_fp8_workspace_size", "pa_varlen_fp8",
           "pa_rope_write_kv", "pa_rope_write_kv_fp8", "pa_decode_weights_workspace_size", "pa_decode_weights",
           "pa_decode_weights_fp8_workspace_size", "pa_decode_weights_fp8", "pa_prompt_weights_workspace_size",
           "pa_prompt_weights", "pa_prompt_weights_fp8_workspace_size", "pa_prompt_weights_fp8",
           "pa_evict_workspace_size", "pa_evict")


class PAError(RuntimeError):
    def __init__(self, status, name, reason):
        super().__init__("%s failed: %s (%s)" % (name, name_of(status), reason))
        self.status = status


_lib = None


def lib():
    """The loaded library (loads it on first use; raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libpa.so is not built (%s); run __graft_entry__.build() first" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    ci, cf = ctypes.c_int, ctypes.c_float
    sig = {
        "pa_status_string": ([ci], ctypes.c_char_p),
        "pa_last_error": ([], ctypes.c_char_p),
        "pa_set_option": ([ci, i64], ci),
        "pa_get_option": ([ci], i64),
        "pa_set_check_mode": ([ci], ci),
        "pa_device_status": ([ci], ci),
        "pa_selftest_wait_timeout": ([i32, vp], ci),
        "pa_slot_mapping": ([vp, i32, i32, vp, vp, i64, i32, vp, vp], ci),
        "pa_write_kv": ([vp, vp, vp, i64, vp, vp, i32, i32, i32, i32, ci, vp], ci),
        "pa_write_kv_fp8": ([vp, vp, vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, ci, vp], ci),
        "pa_decode_fp8_workspace_size": ([i32, i32, i32, i32, i32, i32, ci], sz),
        "pa_decode_append_fp8": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i32, cf,
                                  ci, vp, sz, vp], ci),
        "pa_decode_fp8": ([vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i32, cf, ci, vp, sz,
                           vp], ci),
        "pa_copy_blocks": ([vp, vp, i32, vp, i32, i32, i32, i32, i32, ci, vp], ci),
        "pa_swap_blocks": ([vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, ci, vp], ci),
        "pa_decode_workspace_size": ([i32, i32, i32, i32, i32, i32, ci], sz),
        "pa_decode": ([vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i32, cf, ci, vp, sz, vp], ci),
        "pa_decode_append": ([vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i32, cf, ci, vp, sz,
                              vp], ci),
        "pa_varlen_workspace_size": ([i32, i32, i32, i32, i32, i32, i32, i32, ci], sz),
        "pa_decode_noalloc": ([vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i32, cf, ci, vp], ci),
        "pa_varlen": ([vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, i32, cf, ci, ci, vp,
                       sz, vp], ci),
        "pa_varlen_fp8_workspace_size": ([i32, i32, i32, i32, i32, i32, i32, i32, ci], sz),
        "pa_varlen_fp8": ([vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, i32, cf,
                           ci, ci, vp, sz, vp], ci),
        "pa_rope_write_kv": ([vp, vp, vp, vp, i64, i64, i64, vp, i32, vp, vp, i32, ci, vp, i64, vp, vp, i32, i32, i32,
                              i32, i32, ci, vp], ci),
        "pa_rope_write_kv_fp8": ([vp, vp, vp, vp, i64, i64, i64, vp, i32, vp, vp, i32, ci, vp, i64, vp, vp, vp, vp,
                                  i32, i32, i32, i32, i32, ci, vp], ci),
        "pa_decode_weights_workspace_size": ([i32, i32, i32, i32, i32, i32, ci], sz),
        "pa_decode_weights": ([vp, vp, i64, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i32, cf, ci, vp,
                               sz, vp], ci),
        "pa_decode_weights_fp8_workspace_size": ([i32, i32, i32, i32, i32, i32, ci], sz),
        "pa_decode_weights_fp8": ([vp, vp, i64, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i32,
                                   cf, ci, vp, sz, vp], ci),
        "pa_prompt_weights_workspace_size": ([i32, i32, i32, i32, i32, i32, i32, i32, i32, ci], sz),
        "pa_prompt_weights": ([vp, i64, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, i32, i32, cf,
                               ci, ci, vp, sz, vp], ci),
        "pa_prompt_weights_fp8_workspace_size": ([i32, i32, i32, i32, i32, i32, i32, i32, i32, ci], sz),
        "pa_prompt_weights_fp8": ([vp, i64, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, i32,
                                   i32, cf, ci, ci, vp, sz, vp], ci),
        "pa_evict_workspace_size": ([i32, i32, i32, i32], sz),
        "pa_evict": ([vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32,
                      i32, i32, i32, i32, ci, vp, sz, vp], ci),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def name_of(status):
    return lib().pa_status_string(status).decode()


def _check(status, name):
    if status != 0:
        raise PAError(status, name, lib().pa_last_error().decode())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype(t):
    try:
        return DTYPE_CODE[t.dtype]
    except KeyError:
        raise TypeError("unsupported dtype %s" % t.dtype)


def _pool_dtype(t):
    try:
        return POOL_DTYPE_CODE[t.dtype]
    except KeyError:
        raise TypeError("unsupported pool dtype %s" % t.dtype)


def _dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def pa_set_option(option, value):
    _check(lib().pa_set_option(option, value), "pa_set_option")


def pa_get_option(option):
    return lib().pa_get_option(option)


def pa_set_check_mode(on):
    _check(lib().pa_set_check_mode(1 if on else 0), "pa_set_check_mode")


def pa_selftest_wait_timeout(polls=1000, stream=None):
    """Run the bounded-wait self-test (a wait nothing completes gives up and sets the
    timeout bit that pa_device_status reports)."""
    _check(lib().pa_selftest_wait_timeout(polls, _stream(stream)), "pa_selftest_wait_timeout")


def pa_device_status(clear=True):
    _check(lib().pa_device_status(1 if clear else 0), "pa_device_status")


def pa_slot_mapping(block_tables, seq_idx, positions, block_size, slot_out=None, stream=None):
    """slot_out[i] = block_tables[seq_idx[i], positions[i] // bs] * bs + positions[i] % bs (-1 for pos < 0)."""
    if slot_out is None:
        slot_out = torch.empty(positions.shape[0], dtype=torch.int64, device=positions.device)
    _dev(block_tables, seq_idx, positions, slot_out)
    st = lib().pa_slot_mapping(_ptr(block_tables), block_tables.shape[0], block_tables.shape[1], _ptr(seq_idx),
                               _ptr(positions), positions.shape[0], block_size, _ptr(slot_out), _stream(stream))
    _check(st, "pa_slot_mapping")
    return slot_out


def pa_write_kv(k, v, slot_mapping, k_cache, v_cache, stream=None):
    """Row scatter of k, v [N, Hkv, hd] into caches [NB, bs, Hkv, hd] at slot_mapping [N]."""
    _dev(k, v, slot_mapping, k_cache, v_cache)
    nb, bs, hkv, hd = k_cache.shape
    st = lib().pa_write_kv(_ptr(k), _ptr(v), _ptr(slot_mapping), slot_mapping.shape[0], _ptr(k_cache),
                           _ptr(v_cache), nb, bs, hkv, hd, _dtype(k_cache), _stream(stream))
    _check(st, "pa_write_kv")


def pa_write_kv_fp8(k, v, slot_mapping, k_codes, v_codes, k_scales, v_scales, stream=None):
    """Quantizing write: rows of k, v [N, Hkv, hd] -> E4M3 codes [NB, bs, Hkv, hd] (uint8) at
    slot_mapping [N] and one fp32 scale per row in scales [NB, Hkv, bs]."""
    _dev(k, v, slot_mapping, k_codes, v_codes, k_scales, v_scales)
    nb, bs, hkv, hd = k_codes.shape
    if tuple(k_scales.shape) != (nb, hkv, bs) or tuple(v_scales.shape) != (nb, hkv, bs):
        raise ValueError("scales must be [num_blocks, num_kv_heads, block_size]")
    if k_scales.dtype != torch.float32 or v_scales.dtype != torch.float32:
        raise TypeError("scales must be float32")
    st = lib().pa_write_kv_fp8(_ptr(k), _ptr(v), _ptr(slot_mapping), slot_mapping.shape[0], _ptr(k_codes),
                               _ptr(v_codes), _ptr(k_scales), _ptr(v_scales), nb, bs, hkv, hd, _dtype(k),
                               _stream(stream))
    _check(st, "pa_write_kv_fp8")


def pa_copy_blocks(k_caches, v_caches, block_pairs, stream=None):
    """Copy block pairs [P, 2] (src, dst) in every layer's K and V cache.  Pools are
    [NB, bs, Hkv, hd] (uint8: E4M3 codes) or a quantized cache's scales [NB, Hkv, bs]."""
    if isinstance(k_caches, torch.Tensor):
        k_caches, v_caches = [k_caches], [v_caches]
    _dev(block_pairs, *k_caches, *v_caches)
    n = len(k_caches)
    kp = (ctypes.c_void_p * n)(*[c.data_ptr() for c in k_caches])
    vp = (ctypes.c_void_p * n)(*[c.data_ptr() for c in v_caches])
    if k_caches[0].dim() == 3:  # scale pools of a quantized cache: [NB, Hkv, bs]
        nb, hkv, bs = k_caches[0].shape
        hd = 1
    else:
        nb, bs, hkv, hd = k_caches[0].shape
    st = lib().pa_copy_blocks(kp, vp, n, _ptr(block_pairs), block_pairs.shape[0], nb, bs, hkv, hd,
                              _pool_dtype(k_caches[0]), _stream(stream))
    _check(st, "pa_copy_blocks")


def pa_swap_blocks(src_k, src_v, dst_k, dst_v, block_pairs, stream=None):
    """Copy blocks between two pools (device or pinned host tensors), every layer:
    dst[pairs[p, 1]] = src[pairs[p, 0]]."""
    if isinstance(src_k, torch.Tensor):
        src_k, src_v, dst_k, dst_v = [src_k], [src_v], [dst_k], [dst_v]
    for t in list(src_k) + list(src_v) + list(dst_k) + list(dst_v) + [block_pairs]:
        if not t.is_contiguous() or not (t.is_cuda or t.is_pinned()):
            raise ValueError("pools and pairs must be contiguous CUDA or pinned host tensors")
    n = len(src_k)
    arr = lambda ts: (ctypes.c_void_p * n)(*[t.data_ptr() for t in ts])  # noqa: E731
    nbs, bs, hkv, hd = src_k[0].shape
    st = lib().pa_swap_blocks(arr(src_k), arr(src_v), arr(dst_k), arr(dst_v), n, _ptr(block_pairs),
                              block_pairs.shape[0], nbs, dst_k[0].shape[0], bs, hkv, hd, _pool_dtype(src_k[0]),
                              _stream(stream))
    _check(st, "pa_swap_blocks")


def pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype):
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else dtype
    return lib().pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, code)


def pa_decode(out, q, k_cache, v_cache, block_tables, context_lens, max_context, scale, workspace=None,
              stream=None):
    """One query per sequence: out, q [S, Hq, hd]; context_lens [S]; tables [S, max_blocks]."""
    _dev(out, q, k_cache, v_cache, block_tables, context_lens, workspace)
    nb, bs, hkv, hd = k_cache.shape
    S, hq, _ = q.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().pa_decode(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                         block_tables.shape[1], _ptr(context_lens), S, hq, hkv, hd, nb, bs, max_context,
                         float(scale), _dtype(q), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "pa_decode")
    return out


def pa_decode_fp8_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype):
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else dtype
    return lib().pa_decode_fp8_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context,
                                              code)


def pa_decode_fp8(out, q, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, max_context, scale,
                  workspace=None, stream=None):
    """Decode over a quantized cache: codes [NB, bs, Hkv, hd] uint8, scales [NB, Hkv, bs] fp32;
    out, q [S, Hq, hd] of the query type."""
    _dev(out, q, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, workspace)
    nb, bs, hkv, hd = k_codes.shape
    S, hq, _ = q.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().pa_decode_fp8(_ptr(out), _ptr(q), _ptr(k_codes), _ptr(v_codes), _ptr(k_scales), _ptr(v_scales),
                             _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), S, hq, hkv, hd, nb, bs,
                             max_context, float(scale), _dtype(q), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "pa_decode_fp8")
    return out


def pa_decode_append_fp8(out, q, k_new, v_new, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens,
                         max_context, scale, workspace=None, stream=None):
    """The generation step over a quantized cache: each sequence's new rows k_new, v_new
    [S, Hkv, hd] (query type) are quantized into the slot of position L-1, then decoded."""
    _dev(out, q, k_new, v_new, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, workspace)
    nb, bs, hkv, hd = k_codes.shape
    S, hq, _ = q.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().pa_decode_append_fp8(_ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_codes), _ptr(v_codes),
                                    _ptr(k_scales), _ptr(v_scales), _ptr(block_tables), block_tables.shape[1],
                                    _ptr(context_lens), S, hq, hkv, hd, nb, bs, max_context, float(scale), _dtype(q),
                                    _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "pa_decode_append_fp8")
    return out


def pa_decode_append(out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, max_context, scale,
                     workspace=None, stream=None):
    """Write each sequence's new token (position L-1) into the pool and
    decode: out, q [S, Hq, hd]; k_new, v_new [S, Hkv, hd]."""
    _dev(out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, workspace)
    nb, bs, hkv, hd = k_cache.shape
    S, hq, _ = q.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().pa_decode_append(_ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), S, hq, hkv, hd, nb,
                                bs, max_context, float(scale), _dtype(q), _ptr(workspace), ws_bytes,
                                _stream(stream))
    _check(st, "pa_decode_append")
    return out


def pa_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, max_context, scale, stream=None):
    """pa_decode without a workspace: the scratch is the library's fixed
    per-device array (for callers that cannot allocate device memory)."""
    _dev(out, q, k_cache, v_cache, block_tables, context_lens)
    nb, bs, hkv, hd = k_cache.shape
    S, hq, _ = q.shape
    st = lib().pa_decode_noalloc(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                 block_tables.shape[1], _ptr(context_lens), S, hq, hkv, hd, nb, bs, max_context,
                                 float(scale), _dtype(q), _stream(stream))
    _check(st, "pa_decode_noalloc")
    return out


def pa_varlen_workspace_size(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, block_size, max_context,
                             dtype):
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else dtype
    return lib().pa_varlen_workspace_size(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, block_size,
                                          max_context, code)


def pa_varlen(out, q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, max_q, max_context, scale,
              causal=True, workspace=None, stream=None):
    """Mixed prefill/decode: q, out [T, Hq, hd]; cu_seqlens_q [S+1]; seq_lens [S]."""
    _dev(out, q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, workspace)
    nb, bs, hkv, hd = k_cache.shape
    T, hq, _ = q.shape
    S = seq_lens.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().pa_varlen(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                         block_tables.shape[1], _ptr(seq_lens), _ptr(cu_seqlens_q), S, T, max_q, hq, hkv, hd, nb,
                         bs, max_context, float(scale), 1 if causal else 0, _dtype(q), _ptr(workspace), ws_bytes,
                         _stream(stream))
    _check(st, "pa_varlen")
    return out


def pa_varlen_fp8_workspace_size(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, block_size,
                                 max_context, dtype):
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else dtype
    return lib().pa_varlen_fp8_workspace_size(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim,
                                              block_size, max_context, code)


def pa_varlen_fp8(out, q, k_codes, v_codes, k_scales, v_scales, block_tables, seq_lens, cu_seqlens_q, max_q,
                  max_context, scale, causal=True, workspace=None, stream=None):
    """Mixed prefill/decode over a quantized cache: codes [NB, bs, Hkv, hd] uint8, scales [NB, Hkv, bs] fp32;
    q, out [T, Hq, hd] of the query type; cu_seqlens_q [S+1]; seq_lens [S]."""
    _dev(out, q, k_codes, v_codes, k_scales, v_scales, block_tables, seq_lens, cu_seqlens_q, workspace)
    nb, bs, hkv, hd = k_codes.shape
    T, hq, _ = q.shape
    S = seq_lens.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().pa_varlen_fp8(_ptr(out), _ptr(q), _ptr(k_codes), _ptr(v_codes), _ptr(k_scales), _ptr(v_scales),
                             _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), _ptr(cu_seqlens_q), S, T, max_q,
                             hq, hkv, hd, nb, bs, max_context, float(scale), 1 if causal else 0, _dtype(q),
                             _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "pa_varlen_fp8")
    return out


def _raw(t):
    return None if t is None else t.data_ptr()


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else None
_device_count = None


def _devices():
    """How many devices there are (asked once)."""
    global _device_count
    if _device_count is None:
        _device_count = torch.cuda.device_count()
    return _device_count


def _raw_stream(stream, *ts):
    """The stream's handle (of the current stream without making a Stream object of it), for a call on these tensors:
    all on the current device, where the library launches (looked at where there is another one: 1 us of 10 per
    call)."""
    dev = _current_device()
    if (_device_count or _devices()) > 1:
        for t in ts:
            if t is not None and t.get_device() != dev:
                raise ValueError("the tensors must be on the current device (%d)" % dev)
        if stream is not None and stream.device_index != dev:
            raise ValueError("the stream must be of the current device (%d)" % dev)
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


_CODES = (torch.uint8, torch.float8_e4m3fn)


def _pools(k, v, dtype, codes=False):
    """K and V pools of one shape and type: the rows' dtype, or E4M3 codes.  (The library takes both pools' size from
    the first, and the width of a row from the call.)"""
    if (k.dtype not in _CODES) if codes else (k.dtype != dtype):
        raise ValueError("the pools must hold E4M3 codes (uint8)" if codes else
                         "the pools must be of the dtype of q, k and v (codes: use the _fp8 call)")
    if v is not None and (v.shape != k.shape or v.dtype != k.dtype):
        raise ValueError("the pools must be of one shape and dtype")


def _rope_rows(name, t, n, heads, hd):
    """Token stride (elements) of q, k or v [n, heads, hd]: heads contiguous, tokens at any stride."""
    m, h, d = t.shape
    st, sh, sd = t.stride()
    if not t.is_cuda or m != n or h != heads or d != hd or sd != 1 or (h > 1 and sh != hd):
        raise ValueError("%s must be a CUDA tensor [%d, %d, %d] whose heads are contiguous" % (name, n, heads, hd))
    return st if n > 1 else max(st, heads * hd)


def _rope_args(q_out, q, k, v, positions, inv_freq, slot_mapping, pair_axis, k_pool, v_pool, codes):
    _dev(q_out, positions, inv_freq, slot_mapping, pair_axis, k_pool, v_pool)
    shape = positions.shape
    if len(shape) not in (1, 2) or (q is not None and q_out is None):
        raise ValueError("positions must be [num_axes, n] or [n], and a q needs its q_out")
    n, axes = shape[-1], shape[0] if len(shape) == 2 else 1
    _, _, hkv, hd = k_pool.shape
    if positions.dtype != torch.int64 or inv_freq.dtype != torch.float64 or slot_mapping.dtype != torch.int64:
        raise TypeError("positions and slot_mapping must be int64 and inv_freq float64")
    if pair_axis is not None and (pair_axis.dtype != torch.int32 or pair_axis.numel() != inv_freq.numel()):
        raise ValueError("pair_axis must be int32 with one entry per frequency")
    dt = k.dtype
    if slot_mapping.shape != (n,) or v.dtype != dt:
        raise ValueError("positions and slot_mapping must hold one entry per token, k and v one dtype")
    _pools(k_pool, v_pool, dt, codes)
    hq, qs = 0, 0
    if q is not None:
        hq = q.shape[1]
        if q_out.shape != (n, hq, hd) or q.dtype != dt or q_out.dtype != dt:
            raise ValueError("q_out must be [n, heads, head_dim], and q, q_out, k and v of one dtype")
        qs = _rope_rows("q", q, n, hq, hd)
    ks, vs = _rope_rows("k", k, n, hkv, hd), _rope_rows("v", v, n, hkv, hd)
    return (_raw(q_out), _raw(q), _raw(k), _raw(v), qs, ks, vs, _raw(positions), axes, _raw(inv_freq),
            _raw(pair_axis), 2 * inv_freq.numel()), n, hq


def pa_rope_write_kv(q_out, q, k, v, positions, inv_freq, slot_mapping, k_cache, v_cache, pair_axis=None,
                     interleaved=False, stream=None):
    """Rotate q [n, Hq, hd] into q_out and k [n, Hkv, hd] into the cache, v with it, at slot_mapping [n].

    positions [num_axes, n] (or [n]) int64, inv_freq [rot_dim / 2] float64, pair_axis [rot_dim / 2] int32 (None: one
    axis), all on the device.  Tokens of q, k and v may lie at any stride; q None: keys and values only."""
    args, n, hq = _rope_args(q_out, q, k, v, positions, inv_freq, slot_mapping, pair_axis, k_cache, v_cache, False)
    nb, bs, hkv, hd = k_cache.shape
    st = lib().pa_rope_write_kv(*args, 1 if interleaved else 0, _raw(slot_mapping), n, _raw(k_cache), _raw(v_cache),
                                nb, bs, hq, hkv, hd, _dtype(k),
                                _raw_stream(stream, q_out, q, k, v, positions, inv_freq, slot_mapping, k_cache,
                                            v_cache, pair_axis))
    _check(st, "pa_rope_write_kv")
    return q_out


def pa_rope_write_kv_fp8(q_out, q, k, v, positions, inv_freq, slot_mapping, k_codes, v_codes, k_scales, v_scales,
                         pair_axis=None, interleaved=False, stream=None):
    """pa_rope_write_kv into a quantized cache: codes [NB, bs, Hkv, hd] uint8, scales [NB, Hkv, bs] fp32."""
    _dev(k_scales, v_scales)
    args, n, hq = _rope_args(q_out, q, k, v, positions, inv_freq, slot_mapping, pair_axis, k_codes, v_codes, True)
    nb, bs, hkv, hd = k_codes.shape
    _scale_pools(nb, hkv, bs, k_scales, v_scales)
    st = lib().pa_rope_write_kv_fp8(*args, 1 if interleaved else 0, _raw(slot_mapping), n, _raw(k_codes),
                                    _raw(v_codes), _raw(k_scales), _raw(v_scales), nb, bs, hq, hkv, hd, _dtype(k),
                                    _raw_stream(stream, q_out, q, k, v, positions, inv_freq, slot_mapping, k_codes,
                                                v_codes, k_scales, v_scales, pair_axis))
    _check(st, "pa_rope_write_kv_fp8")
    return q_out


def _scale_pools(nb, hkv, bs, *scales):
    for s in scales:
        if s is None or s.shape != (nb, hkv, bs) or s.dtype != torch.float32:
            raise ValueError("scales must be float32 [num_blocks, num_kv_heads, block_size]")


def _weight_rows(name, t, S, hkv, dtype=torch.float32):
    shape = t.shape
    if len(shape) != 3 or shape[0] != S or shape[1] != hkv or t.dtype != dtype:
        raise ValueError("%s must be %s [num_seqs, num_kv_heads, weights_stride]" % (name, dtype))
    return shape[2]


def _i32(*ts):
    for t in ts:
        if t is not None and t.dtype != torch.int32:
            raise TypeError("block tables, lengths and cu_seqlens_q must be int32")


def _same_batch(q, pool, lens, *tables):
    """A batch's parts fit each other: q's head_dim and the pools', a table row and a length per sequence."""
    if q is not None and q.shape[2] != pool.shape[3]:
        raise ValueError("q and the cache must be of one head_dim")
    for t in tables:
        if t.shape[0] != lens.shape[0]:
            raise ValueError("block tables must have one row per sequence")


def _ws(workspace):
    return _raw(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size()


def pa_decode_weights_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype):
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else dtype
    return lib().pa_decode_weights_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context,
                                                  code)


def pa_decode_weights(out, weights, q, k_cache, v_cache, block_tables, context_lens, max_context, scale, workspace,
                      stream=None):
    """pa_decode that adds each cached token's attention weight (summed over the query heads of a KV head) to
    weights [S, Hkv, stride] fp32; the newest token's entry is set."""
    _dev(out, weights, q, k_cache, v_cache, block_tables, context_lens, workspace)
    _i32(block_tables, context_lens)
    _same_batch(q, k_cache, context_lens, block_tables)
    nb, bs, hkv, hd = k_cache.shape
    S, hq, _ = q.shape
    _pools(k_cache, v_cache, q.dtype)
    if out.shape != q.shape or out.dtype != q.dtype or context_lens.shape[0] != S:
        raise ValueError("out must have q's shape and dtype, context_lens one entry per query")
    stride = _weight_rows("weights", weights, S, hkv)
    st = lib().pa_decode_weights(_raw(out), _raw(weights), stride, _raw(q), _raw(k_cache), _raw(v_cache),
                                 _raw(block_tables), block_tables.shape[1], _raw(context_lens), S, hq, hkv, hd, nb,
                                 bs, max_context, float(scale), _dtype(q), *_ws(workspace),
                                 _raw_stream(stream, out, weights, q, k_cache, v_cache, block_tables, context_lens,
                                             workspace))
    _check(st, "pa_decode_weights")
    return out


def pa_decode_weights_fp8_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype):
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else dtype
    return lib().pa_decode_weights_fp8_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                      max_context, code)


def pa_decode_weights_fp8(out, weights, q, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens,
                          max_context, scale, workspace, stream=None):
    """pa_decode_weights over a quantized cache: codes [NB, bs, Hkv, hd] uint8, scales [NB, Hkv, bs] fp32."""
    _dev(out, weights, q, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, workspace)
    _i32(block_tables, context_lens)
    _same_batch(q, k_codes, context_lens, block_tables)
    nb, bs, hkv, hd = k_codes.shape
    S, hq, _ = q.shape
    _pools(k_codes, v_codes, q.dtype, True)
    if out.shape != q.shape or out.dtype != q.dtype or context_lens.shape[0] != S:
        raise ValueError("out must have q's shape and dtype, context_lens one entry per query")
    _scale_pools(nb, hkv, bs, k_scales, v_scales)
    stride = _weight_rows("weights", weights, S, hkv)
    st = lib().pa_decode_weights_fp8(_raw(out), _raw(weights), stride, _raw(q), _raw(k_codes), _raw(v_codes),
                                     _raw(k_scales), _raw(v_scales), _raw(block_tables), block_tables.shape[1],
                                     _raw(context_lens), S, hq, hkv, hd, nb, bs, max_context, float(scale), _dtype(q),
                                     *_ws(workspace),
                                     _raw_stream(stream, out, weights, q, k_codes, v_codes, k_scales, v_scales,
                                                 block_tables, context_lens, workspace))
    _check(st, "pa_decode_weights_fp8")
    return out


def pa_prompt_weights_workspace_size(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, block_size,
                                     max_context, window, dtype):
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else dtype
    return lib().pa_prompt_weights_workspace_size(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim,
                                                  block_size, max_context, window, code)


def pa_prompt_weights(weights, q, k_cache, block_tables, seq_lens, cu_seqlens_q, max_q, max_context, window, scale,
                      causal=True, workspace=None, stream=None):
    """Attention weights that the last `window` (0: all) new tokens of each request give its cached tokens: added to
    weights [S, Hkv, stride] fp32 for tokens cached before the step, set for new ones.  q [T, Hq, hd]."""
    _dev(weights, q, k_cache, block_tables, seq_lens, cu_seqlens_q, workspace)
    _i32(block_tables, seq_lens, cu_seqlens_q)
    _same_batch(q, k_cache, seq_lens, block_tables)
    _pools(k_cache, None, q.dtype)
    nb, bs, hkv, hd = k_cache.shape
    T, hq, _ = q.shape
    S = seq_lens.shape[0]
    if cu_seqlens_q.shape[0] != S + 1:
        raise ValueError("cu_seqlens_q must hold one entry more than there are sequences")
    stride = _weight_rows("weights", weights, S, hkv)
    st = lib().pa_prompt_weights(_raw(weights), stride, _raw(q), _raw(k_cache), _raw(block_tables),
                                 block_tables.shape[1], _raw(seq_lens), _raw(cu_seqlens_q), S, T, max_q, hq, hkv, hd,
                                 nb, bs, max_context, window, float(scale), 1 if causal else 0, _dtype(q),
                                 *_ws(workspace),
                                 _raw_stream(stream, weights, q, k_cache, block_tables, seq_lens, cu_seqlens_q,
                                             workspace))
    _check(st, "pa_prompt_weights")
    return weights


def pa_prompt_weights_fp8_workspace_size(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, block_size,
                                         max_context, window, dtype):
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else dtype
    return lib().pa_prompt_weights_fp8_workspace_size(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim,
                                                      block_size, max_context, window, code)


def pa_prompt_weights_fp8(weights, q, k_codes, k_scales, block_tables, seq_lens, cu_seqlens_q, max_q, max_context,
                          window, scale, causal=True, workspace=None, stream=None):
    """pa_prompt_weights over a quantized cache's keys: codes [NB, bs, Hkv, hd] uint8, scales [NB, Hkv, bs] fp32."""
    _dev(weights, q, k_codes, k_scales, block_tables, seq_lens, cu_seqlens_q, workspace)
    _i32(block_tables, seq_lens, cu_seqlens_q)
    _same_batch(q, k_codes, seq_lens, block_tables)
    _pools(k_codes, None, q.dtype, True)
    nb, bs, hkv, hd = k_codes.shape
    T, hq, _ = q.shape
    S = seq_lens.shape[0]
    if cu_seqlens_q.shape[0] != S + 1:
        raise ValueError("cu_seqlens_q must hold one entry more than there are sequences")
    _scale_pools(nb, hkv, bs, k_scales)
    stride = _weight_rows("weights", weights, S, hkv)
    st = lib().pa_prompt_weights_fp8(_raw(weights), stride, _raw(q), _raw(k_codes), _raw(k_scales),
                                     _raw(block_tables), block_tables.shape[1], _raw(seq_lens), _raw(cu_seqlens_q), S,
                                     T, max_q, hq, hkv, hd, nb, bs, max_context, window, float(scale),
                                     1 if causal else 0, _dtype(q), *_ws(workspace),
                                     _raw_stream(stream, weights, q, k_codes, k_scales, block_tables, seq_lens,
                                                 cu_seqlens_q, workspace))
    _check(st, "pa_prompt_weights_fp8")
    return weights


def pa_evict_workspace_size(num_seqs, num_kv_heads, max_context, keep):
    return lib().pa_evict_workspace_size(num_seqs, num_kv_heads, max_context, keep)


def pa_evict(new_lens, weights_out, positions_out, weights, k_cache, v_cache, block_tables, new_block_tables,
             context_lens, max_context, keep, num_sink, num_recent, positions=None, recorded_lens=None,
             seen_lens=None, k_scales=None, v_scales=None, workspace=None, stream=None):
    """Drop the cached tokens with the least weight, per sequence and KV head, down to `keep` (besides the first
    num_sink and the newest num_recent positions); kept rows move to the front, through new_block_tables.

    weights, weights_out [S, Hkv, stride] fp32; positions, positions_out the same in int32 (positions_out may be
    None); new_lens, recorded_lens, seen_lens [S] int32.  Quantized pools (uint8) come with their scale pools."""
    _dev(new_lens, weights_out, positions_out, weights, k_cache, v_cache, block_tables, new_block_tables, context_lens,
         positions, recorded_lens, seen_lens, k_scales, v_scales, workspace)
    _i32(new_lens, block_tables, new_block_tables, context_lens, recorded_lens, seen_lens)
    _same_batch(None, k_cache, context_lens, block_tables, new_block_tables)
    nb, bs, hkv, hd = k_cache.shape
    S = context_lens.shape[0]
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("the pools must be of one shape and dtype")
    for t in (context_lens, new_lens, recorded_lens, seen_lens):
        if t is not None and t.numel() != S:
            raise ValueError("context_lens, new_lens, recorded_lens and seen_lens hold one entry per sequence")
    stride = _weight_rows("weights", weights, S, hkv)
    rows = [("weights_out", weights_out, torch.float32), ("positions_out", positions_out, torch.int32),
            ("positions", positions, torch.int32)]
    for name, t, dt in rows:
        if t is not None and _weight_rows(name, t, S, hkv, dt) != stride:
            raise ValueError("%s must have the row stride of weights" % name)
    if k_scales is not None or v_scales is not None:
        _scale_pools(nb, hkv, bs, k_scales, v_scales)
    st = lib().pa_evict(_raw(weights_out), _raw(positions_out), _raw(new_lens), _raw(weights), _raw(positions),
                        _raw(recorded_lens), _raw(seen_lens), stride, _raw(k_cache), _raw(v_cache), _raw(k_scales),
                        _raw(v_scales), _raw(block_tables), block_tables.shape[1], _raw(new_block_tables),
                        new_block_tables.shape[1], _raw(context_lens), S, hkv, hd, nb, bs, max_context, keep,
                        num_sink, num_recent, _pool_dtype(k_cache), *_ws(workspace),
                        _raw_stream(stream, new_lens, weights_out, positions_out, weights, k_cache, v_cache,
                                    block_tables, new_block_tables, context_lens, positions, recorded_lens, seen_lens,
                                    k_scales, v_scales, workspace))
    _check(st, "pa_evict")
    return new_lens
