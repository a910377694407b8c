"""Python binding of libsk: length-aware split-KV paged decode/verify attention
on GB300 (sm_103a).

Argument marshalling only: every step of the path (plan, attention, merge)
and the KV write and page conversion around it run in the CUDA kernels of
``libsk.so``; torch supplies device memory and streams.  The functions carry
the C names (``sk_build_plan``, ``sk_paged_decode_attn``,
``sk_merge_segments``, ``sk_plan_cache_reset``, ``sk_reshape_and_cache``,
``sk_std_to_shuffled``) and take torch tensors; ``paged_decode_attention``
chains the three attention calls the way a serving step does.  Around them:
``sk_rope_and_cache`` (rotary positions with the KV write),
``paged_prefill_attention`` (attention of a chunk of new tokens over the
pages), ``sk_accum_attn_weights`` (the attention weight each cached key
receives) and ``evict_rows`` (a cache cut down to its heaviest and latest
rows).  If ``libsk.so`` has not been built, every call raises: there is no
fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Optional, Tuple

__all__ = [
    "SkError", "lib", "sk_tile_tokens", "sk_fixed_nseg", "sk_build_plan", "sk_plan_cache_reset",
    "sk_plan_launch_count", "sk_paged_decode_attn", "sk_merge_segments", "sk_get_device_status",
    "paged_decode_attention", "plan_capacity", "sk_plan_capacity", "sk_paged_decode_attention_static",
    "sk_static_scratch_bytes", "sk_reshape_and_cache", "sk_std_to_shuffled", "sk_set_wait_limit",
    "SK_OK", "SK_CACHED", "SK_ERR_TIMEOUT", "SK_KV_BF16", "SK_KV_FP8_E4M3", "SK_DEV_BAD_BLOCK",
    "SK_DEV_BAD_SEQ", "SK_DEV_TIMEOUT", "sk_rope_frequencies", "sk_rope_and_cache", "sk_evict_capacity",
    "sk_evict_select", "sk_evict_move", "evict_rows", "sk_prefill_workspace_bytes",
    "sk_paged_prefill_attn", "paged_prefill_attention", "sk_accum_attn_weights", "sk_accum_workspace_bytes",
]

SK_OK = 0
SK_CACHED = 1
SK_ERR_TIMEOUT = -5
SK_KV_BF16 = 0
SK_KV_FP8_E4M3 = 1
SK_DEV_BAD_BLOCK = 0x1
SK_DEV_BAD_SEQ = 0x2
SK_DEV_TIMEOUT = 0x4

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsk.so")
_lock = threading.Lock()
_lib = None


class SkError(RuntimeError):
    pass


def lib():
    """Load libsk.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise SkError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, u64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_float
        L.sk_tile_tokens.restype = i32
        L.sk_tile_tokens.argtypes = []
        L.sk_fixed_nseg.restype = i32
        L.sk_fixed_nseg.argtypes = [i32, i32, i32, i32]
        L.sk_plan_capacity.restype = i32
        L.sk_plan_capacity.argtypes = [i32, i32, i32]
        L.sk_set_wait_limit.restype = ctypes.c_longlong
        L.sk_set_wait_limit.argtypes = [ctypes.c_longlong]
        L.sk_last_device_status.restype = i32
        L.sk_last_device_status.argtypes = []
        L.sk_build_plan.restype = i32
        L.sk_build_plan.argtypes = [P, u64, P, u64, i32, i32, i32, i32, i32, P, i32, P, P]
        L.sk_plan_cache_reset.restype = None
        L.sk_plan_cache_reset.argtypes = []
        L.sk_plan_launch_count.restype = ctypes.c_longlong
        L.sk_plan_launch_count.argtypes = []
        L.sk_paged_decode_attn.restype = i32
        L.sk_paged_decode_attn.argtypes = [P, P, i32, f32, f32, P, i32, i32, i32, P, P, P, i32,
                                           i32, i32, i32, i32, i32, i32, f32, i32, i32, i32,
                                           P, P, P, P]
        L.sk_merge_segments.restype = i32
        L.sk_merge_segments.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, P, P, P]
        L.sk_reshape_and_cache.restype = i32
        L.sk_reshape_and_cache.argtypes = [P, P, P, i32, i32, i32, P, i32, f32, f32, i32, i32, P]
        L.sk_std_to_shuffled.restype = i32
        L.sk_std_to_shuffled.argtypes = [P, i32, P, i32, i32, i32, i32, i32, P, P, P]
        i64, f64, PD = ctypes.c_int64, ctypes.c_double, ctypes.POINTER(ctypes.c_double)
        L.sk_rope_frequencies.restype = i32
        L.sk_rope_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, PD, PD]
        L.sk_rope_and_cache.restype = i32
        L.sk_rope_and_cache.argtypes = [P, P, P, i64, i64, i64, P, P, i32, i32, f32, P, i32, i32, i32, i32, P, P, i32,
                                        f32, f32, i32, i32, P, P, P]
        L.sk_prefill_workspace_bytes.restype = i64
        L.sk_prefill_workspace_bytes.argtypes = [i32, i32, i32]
        L.sk_paged_prefill_attn.restype = i32
        L.sk_paged_prefill_attn.argtypes = [P, P, i32, f32, f32, P, i32, i32, i32, P, P, i32, i32, i32, i32, i32, i32,
                                            f32, i32, i32, P, i64, P, P, P]
        L.sk_accum_workspace_bytes.restype = i64
        L.sk_accum_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.sk_accum_attn_weights.restype = i32
        L.sk_accum_attn_weights.argtypes = [P, P, i32, f32, P, i32, i32, i32, P, P, i32, i32, i32, i32, i32, i32, f32,
                                            i32, P, P, P, i64, P]
        L.sk_evict_capacity.restype = i32
        L.sk_evict_capacity.argtypes = [i32, i32]
        L.sk_evict_select.restype = i32
        L.sk_evict_select.argtypes = [P, P, P, i32, i32, i32, P, P, i32, i32, i32, i32, i32, i32, P, P, P, P, P]
        L.sk_evict_move.restype = i32
        L.sk_evict_move.argtypes = [P, P, P, i32, i32, i32, i32, P, i32, i32, i32, P, i32, P, P, P]
        L.sk_get_device_status.restype = i32
        L.sk_get_device_status.argtypes = [P, i32]
        L.sk_paged_decode_attention_static.restype = i32
        L.sk_paged_decode_attention_static.argtypes = [P, P, i32, f32, f32, P, i32, i32, i32, P, P,
                                                       i32, i32, i32, i32, i32, i32, i32, f32, i32,
                                                       i32, i32, P, P, P]
        L.sk_static_scratch_bytes.restype = ctypes.c_size_t
        L.sk_static_scratch_bytes.argtypes = []
        L.sk_last_error.restype = ctypes.c_char_p
        L.sk_last_error.argtypes = []
        _lib = L
        return L


def _check(rc: int, name: str) -> int:
    if rc < 0:
        msg = lib().sk_last_error()
        raise SkError(f"{name} returned {rc}: {msg.decode() if msg else ''}")
    return rc


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t, dtype, name, dims=None):
    """Type, layout and rank of one argument (where it lives is checked by _on_cuda)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, has {t.dim()}")


def _shape(t, shape, name):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _on_cuda(**tensors):
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")


def _check_batch(q, kv_pages, block_table, seq_lens, cu_seqlens_q):
    """The shapes an attention call reads through raw pointers: q [NT, H_q, D], kv_pages
    [NB, H_kv, page, 2D] with H_kv dividing H_q, seq_lens [bs], cu_seqlens_q [bs + 1] and at
    least bs block-table rows.  Returns (nt, hq, d, nb, hkv, page, bs)."""
    nt, hq, d = q.shape
    nb, hkv, page, d2 = kv_pages.shape
    if d2 != 2 * d:
        raise ValueError(f"kv_pages last dimension is {d2}, expected 2 * head_dim = {2 * d}")
    if hkv < 1 or hq % hkv != 0:
        raise ValueError(f"{hq} query heads are not a multiple of {hkv} KV heads")
    bs = seq_lens.numel()
    if cu_seqlens_q.numel() != bs + 1:
        raise ValueError(f"cu_seqlens_q has {cu_seqlens_q.numel()} entries, expected bs + 1 = {bs + 1}")
    if block_table.shape[0] < bs:
        raise ValueError(f"block_table has {block_table.shape[0]} rows for {bs} sequences")
    return nt, hq, d, nb, hkv, page, bs


def sk_tile_tokens() -> int:
    return lib().sk_tile_tokens()


def sk_fixed_nseg(bs: int, num_kv_heads: int, num_sms: int, seg_max: int = 64) -> int:
    return lib().sk_fixed_nseg(bs, num_kv_heads, num_sms, seg_max)


def sk_plan_capacity(bs: int, num_kv_heads: int, num_sms: int) -> int:
    """Smallest valid plan buffer length for a batch (computed by the library)."""
    return _check(lib().sk_plan_capacity(int(bs), int(num_kv_heads), int(num_sms)), "sk_plan_capacity")


plan_capacity = sk_plan_capacity


def sk_set_wait_limit(cycles: int) -> int:
    """Sets the attention kernels' abortable-wait limit in SM cycles (negative:
    the default, about two seconds) for later launches; returns the previous one.
    A test hook for the timeout path."""
    return int(lib().sk_set_wait_limit(int(cycles)))


def sk_plan_cache_reset() -> None:
    lib().sk_plan_cache_reset()


def sk_plan_launch_count() -> int:
    return lib().sk_plan_launch_count()


def sk_build_plan(seq_lens, cu_seqlens_q, num_kv_heads: int, plan, tok_nseg, num_sms: int,
                  seg_max: int = 64, stream=None) -> int:
    """Returns SK_OK (plan kernel enqueued) or SK_CACHED (cache hit)."""
    import torch
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q", 1)
    _need(plan, torch.int32, "plan", 1)
    _need(tok_nseg, torch.int32, "tok_nseg", 1)
    bs = seq_lens.numel()
    if cu_seqlens_q.numel() != bs + 1:
        raise ValueError(f"cu_seqlens_q has {cu_seqlens_q.numel()} entries, expected bs + 1 = {bs + 1}")
    _on_cuda(seq_lens=seq_lens, cu_seqlens_q=cu_seqlens_q, plan=plan, tok_nseg=tok_nseg)
    rc = lib().sk_build_plan(_ptr(seq_lens), seq_lens._version, _ptr(cu_seqlens_q),
                             cu_seqlens_q._version, bs, tok_nseg.numel(), num_kv_heads, num_sms,
                             seg_max, _ptr(plan), plan.numel(), _ptr(tok_nseg), _stream(stream))
    return _check(rc, "sk_build_plan")


def _kv_dtype(kv_pages) -> int:
    import torch
    if kv_pages.dtype == torch.bfloat16:
        return SK_KV_BF16
    if kv_pages.dtype in (torch.uint8, torch.float8_e4m3fn):
        return SK_KV_FP8_E4M3
    raise ValueError(f"kv_pages dtype {kv_pages.dtype}: expected bfloat16, uint8 or float8_e4m3fn")


def sk_paged_decode_attn(q, kv_pages, block_table, seq_lens, cu_seqlens_q, plan, part_o, part_m,
                         part_l, *, max_q_len: int, sm_scale: float, num_sms: int,
                         k_scale: float = 1.0, v_scale: float = 1.0, causal: bool = True,
                         stream=None) -> int:
    import torch
    _need(q, torch.bfloat16, "q", 3)
    _need(kv_pages, None, "kv_pages", 4)
    _need(block_table, torch.int32, "block_table", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q", 1)
    _need(part_o, torch.float32, "part_o", 4)
    _need(part_m, torch.float32, "part_m", 3)
    _need(part_l, torch.float32, "part_l", 3)
    if plan is not None:
        _need(plan, torch.int32, "plan", 1)
    nt, hq, d, nb, hkv, page, bs = _check_batch(q, kv_pages, block_table, seq_lens, cu_seqlens_q)
    seg_max = part_o.shape[1]
    _shape(part_o, (nt, seg_max, hq, d), "part_o")
    _shape(part_m, (nt, seg_max, hq), "part_m")
    _shape(part_l, (nt, seg_max, hq), "part_l")
    _on_cuda(q=q, kv_pages=kv_pages, block_table=block_table, seq_lens=seq_lens, cu_seqlens_q=cu_seqlens_q,
             plan=plan, part_o=part_o, part_m=part_m, part_l=part_l)
    rc = lib().sk_paged_decode_attn(
        _ptr(q), _ptr(kv_pages), _kv_dtype(kv_pages), float(k_scale), float(v_scale),
        _ptr(block_table), block_table.shape[1], nb, page, _ptr(seq_lens), _ptr(cu_seqlens_q),
        _ptr(plan), plan.numel() if plan is not None else 0, seq_lens.numel(), nt, int(max_q_len),
        hq, hkv, d, float(sm_scale), 1 if causal else 0, int(num_sms), seg_max,
        _ptr(part_o), _ptr(part_m), _ptr(part_l), _stream(stream))
    return _check(rc, "sk_paged_decode_attn")


def sk_merge_segments(part_o, part_m, part_l, tok_nseg, out, lse=None, fixed_nseg: int = 0,
                      stream=None) -> int:
    import torch
    _need(part_o, torch.float32, "part_o", 4)
    _need(part_m, torch.float32, "part_m", 3)
    _need(part_l, torch.float32, "part_l", 3)
    _need(out, torch.bfloat16, "out", 3)
    if tok_nseg is not None:
        _need(tok_nseg, torch.int32, "tok_nseg", 1)
    if lse is not None:
        _need(lse, torch.float32, "lse", 2)
    nt, seg_max, hq, d = part_o.shape
    _shape(part_m, (nt, seg_max, hq), "part_m")
    _shape(part_l, (nt, seg_max, hq), "part_l")
    _shape(out, (nt, hq, d), "out")
    _shape(lse, (nt, hq), "lse")
    if tok_nseg is not None and tok_nseg.numel() != nt:
        raise ValueError(f"tok_nseg has {tok_nseg.numel()} entries for {nt} tokens")
    _on_cuda(part_o=part_o, part_m=part_m, part_l=part_l, tok_nseg=tok_nseg, out=out, lse=lse)
    rc = lib().sk_merge_segments(_ptr(part_o), _ptr(part_m), _ptr(part_l), _ptr(tok_nseg),
                                 int(fixed_nseg), nt, hq, d, seg_max, _ptr(out), _ptr(lse),
                                 _stream(stream))
    return _check(rc, "sk_merge_segments")


def sk_reshape_and_cache(key, value, slot_mapping, kv_pages, *, k_scale: float = 1.0,
                         v_scale: float = 1.0, stream=None) -> int:
    """Writes this step's K/V rows ([num_tokens, num_kv_heads, head_dim] bf16) into
    ``kv_pages`` ([num_blocks, num_kv_heads, page, 2*head_dim], bf16 or e4m3) at
    ``slot_mapping`` (int64 [num_tokens], negative = no slot), in place."""
    import torch
    _need(key, torch.bfloat16, "key", 3)
    _need(value, torch.bfloat16, "value", 3)
    _need(slot_mapping, torch.int64, "slot_mapping", 1)
    _need(kv_pages, None, "kv_pages", 4)
    nt, hkv, d = key.shape
    if tuple(value.shape) != (nt, hkv, d) or slot_mapping.numel() != nt:
        raise ValueError("key, value and slot_mapping must agree on [num_tokens, num_kv_heads, head_dim]")
    nb, hkv2, page, d2 = kv_pages.shape
    if hkv2 != hkv or d2 != 2 * d:
        raise ValueError("kv_pages must be [num_blocks, num_kv_heads, page, 2 * head_dim]")
    _on_cuda(key=key, value=value, slot_mapping=slot_mapping, kv_pages=kv_pages)
    rc = lib().sk_reshape_and_cache(_ptr(key), _ptr(value), _ptr(slot_mapping), nt, hkv, d,
                                    _ptr(kv_pages), _kv_dtype(kv_pages), float(k_scale), float(v_scale),
                                    nb, page, _stream(stream))
    return _check(rc, "sk_reshape_and_cache")


def sk_std_to_shuffled(kv_pages, k_shuf, v_shuf, block_ids=None, stream=None) -> int:
    """Standard pages [NB, H, 16, 256] to shuffled K [NB, H, 128/x, 16, x] and
    V [NB, H, 16/x, 128, x] (x = 16 / element size), for ``block_ids`` (int32)
    or every block."""
    import torch
    _need(kv_pages, None, "kv_pages", 4)
    _need(k_shuf, kv_pages.dtype, "k_shuf", 5)
    _need(v_shuf, kv_pages.dtype, "v_shuf", 5)
    if block_ids is not None:
        _need(block_ids, torch.int32, "block_ids", 1)
    nb, hkv, page, d2 = kv_pages.shape
    d = d2 // 2
    x = 16 // kv_pages.element_size()
    if tuple(k_shuf.shape) != (nb, hkv, d // x, page, x) or tuple(v_shuf.shape) != (nb, hkv, page // x, d, x):
        raise ValueError("k_shuf must be [NB, H, D/x, page, x] and v_shuf [NB, H, page/x, D, x]")
    _on_cuda(kv_pages=kv_pages, k_shuf=k_shuf, v_shuf=v_shuf, block_ids=block_ids)
    rc = lib().sk_std_to_shuffled(_ptr(kv_pages), _kv_dtype(kv_pages), _ptr(block_ids),
                                  0 if block_ids is None else block_ids.numel(), nb, hkv, d, page,
                                  _ptr(k_shuf), _ptr(v_shuf), _stream(stream))
    return _check(rc, "sk_std_to_shuffled")


def sk_static_scratch_bytes() -> int:
    return lib().sk_static_scratch_bytes()


def sk_paged_decode_attention_static(q, kv_pages, block_table, seq_lens, cu_seqlens_q, out, lse=None,
                                     *, max_q_len: int, sm_scale: float, num_sms: int,
                                     k_scale: float = 1.0, v_scale: float = 1.0, causal: bool = True,
                                     seg_max: int = 64, use_plan: Optional[bool] = None,
                                     stream=None) -> int:
    """The whole call without device allocation: plan, per-token counts and
    partials live in the library's fixed 32 MiB device array.  For callers that
    cannot allocate; calls that overlap on the GPU race on that array.
    use_plan defaults to bs > 1, as in paged_decode_attention (bs == 1 takes the
    fixed split)."""
    import torch
    _need(q, torch.bfloat16, "q", 3)
    _need(kv_pages, None, "kv_pages", 4)
    _need(block_table, torch.int32, "block_table", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q", 1)
    _need(out, torch.bfloat16, "out", 3)
    if lse is not None:
        _need(lse, torch.float32, "lse", 2)
    nt, hq, d, nb, hkv, page, bs = _check_batch(q, kv_pages, block_table, seq_lens, cu_seqlens_q)
    _shape(out, (nt, hq, d), "out")
    _shape(lse, (nt, hq), "lse")
    if use_plan is None:
        use_plan = bs > 1
    _on_cuda(q=q, kv_pages=kv_pages, block_table=block_table, seq_lens=seq_lens, cu_seqlens_q=cu_seqlens_q,
             out=out, lse=lse)
    rc = lib().sk_paged_decode_attention_static(
        _ptr(q), _ptr(kv_pages), _kv_dtype(kv_pages), float(k_scale), float(v_scale),
        _ptr(block_table), block_table.shape[1], nb, page, _ptr(seq_lens), _ptr(cu_seqlens_q),
        1 if use_plan else 0, seq_lens.numel(), nt, int(max_q_len), hq, hkv, d, float(sm_scale),
        1 if causal else 0, int(num_sms), int(seg_max), _ptr(out), _ptr(lse), _stream(stream))
    return _check(rc, "sk_paged_decode_attention_static")


_ROPE_SCALING = {"plain": 0, "linear": 1, "base": 2, "bands": 3}


def _fits(t, dtype, shape, name, dev) -> int:
    """Checks one argument in one expression (calls of a decode step are short): its type, shape, layout and
    device ``dev`` (an ordinal, -1 for the CPU).  Returns its address."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _need(t, dtype, name, len(shape))
    _shape(t, shape, name)
    raise ValueError(f"{name} must be a CUDA tensor on the device of the other arguments, is on {t.device}")


def _pages(kv_pages, dev):
    """Address, type and shape of the pages."""
    if kv_pages is None or kv_pages.dim() != 4 or not kv_pages.is_contiguous():
        _need(kv_pages, None, "kv_pages", 4)
    if kv_pages.get_device() != dev:
        raise ValueError(f"kv_pages must be a CUDA tensor on the device of the other arguments, is on {kv_pages.device}")
    return kv_pages.data_ptr(), _kv_dtype(kv_pages), kv_pages.shape


def _launch(dev: int, stream, name, f, *args) -> int:
    """Calls ``f(*args, stream)`` with device ``dev`` current (streams and the status word are per device); the
    stream is that device's current one by default."""
    import torch
    if dev < 0:
        raise ValueError(f"{name}: the arguments must be CUDA tensors")
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return _launch(dev, stream, name, f, *args)
    if stream is None:
        st = torch._C._cuda_getCurrentRawStream(dev)
    else:
        st = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    rc = f(*args, st)
    return rc if rc >= 0 else _check(rc, name)


def _heads_view(t, name, dev):
    """[tokens, heads, 128] bf16 whose heads are contiguous; returns the address and the stride between tokens."""
    import torch
    if t.dtype is not torch.bfloat16 or t.dim() != 3:
        raise ValueError(f"{name} must be bfloat16 [num_tokens, heads, head_dim], is {t.dtype} {tuple(t.shape)}")
    nt, h, d = t.shape
    st, sh, sd = t.stride()
    if (sd != 1 and d != 1) or (sh != d and h != 1):
        raise ValueError(f"{name} must have contiguous heads, has strides {t.stride()}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the device of the other arguments, is on {t.device}")
    return t.data_ptr(), st if nt > 1 else max(st, h * d)


def sk_rope_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: str = "plain", factor: float = 1.0,
                        original_len: float = 0.0, low: float = 1.0, high: float = 32.0, device=None):
    """Rotary frequencies (float64 [rot_dim / 2] on ``device``) and their attention factor.
    ``scaling``: "plain", "linear" (w / factor), "base" (a larger base) or "bands" (by the turns a
    frequency makes in ``original_len`` positions: w / factor up to ``low``, w from ``high`` on)."""
    import torch
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"scaling {scaling!r}: expected one of {sorted(_ROPE_SCALING)}")
    out = (ctypes.c_double * max(1, int(rot_dim) // 2))()
    af = ctypes.c_double(1.0)
    _check(lib().sk_rope_frequencies(int(rot_dim), float(base), _ROPE_SCALING[scaling], float(factor),
                                     float(original_len), float(low), float(high), out, ctypes.byref(af)),
           "sk_rope_frequencies")
    return torch.tensor(list(out), dtype=torch.float64, device=device), af.value


def sk_rope_and_cache(q, key, value, positions, freqs, slot_mapping, kv_pages, q_out, *, interleaved: bool = False,
                      attn_factor: float = 1.0, k_scale: float = 1.0, v_scale: float = 1.0, acc_pages=None,
                      pos_pages=None, stream=None) -> int:
    """Turns q ([num_tokens, num_q_heads, 128] bf16) into ``q_out`` and key by the tokens' ``positions``
    (int64) and stores key and ``value`` ([num_tokens, num_kv_heads, 128] bf16) into ``kv_pages`` at
    ``slot_mapping`` (int64, negative = no slot).  q, key and value may be views with a stride between
    tokens.  ``freqs``: float64 [rot_dim / 2], radians per position (sk_rope_frequencies), rot_dim a
    multiple of 16; ``interleaved`` pairs (2i, 2i + 1) instead of halves.  ``acc_pages`` (fp32) and
    ``pos_pages`` (int32), both [num_blocks, num_kv_heads, page], receive 0 and the position of each
    stored token: the state that eviction works on."""
    import torch
    dev = q.get_device()
    (pq, qs), (pk, ks), (pv, vs) = _heads_view(q, "q", dev), _heads_view(key, "key", dev), _heads_view(value, "value", dev)
    nt, hq, d = q.shape
    hkv = key.shape[1]
    _shape(key, (nt, hkv, d), "key")
    _shape(value, (nt, hkv, d), "value")
    pp, dt, (nb, hkv2, page, d2) = _pages(kv_pages, dev)
    if hkv2 != hkv or d2 != 2 * d:
        raise ValueError("kv_pages must be [num_blocks, num_kv_heads, page, 2 * head_dim]")
    acc = None if acc_pages is None else _fits(acc_pages, torch.float32, (nb, hkv, page), "acc_pages", dev)
    pos = None if pos_pages is None else _fits(pos_pages, torch.int32, (nb, hkv, page), "pos_pages", dev)
    rot2 = freqs.numel()
    return _launch(dev, stream, "sk_rope_and_cache", lib().sk_rope_and_cache, pq, pk, pv, qs, ks, vs,
                   _fits(positions, torch.int64, (nt,), "positions", dev),
                   _fits(freqs, torch.float64, (rot2,), "freqs", dev), 2 * rot2, 1 if interleaved else 0, attn_factor,
                   _fits(slot_mapping, torch.int64, (nt,), "slot_mapping", dev), nt, hq, hkv, d,
                   _fits(q_out, torch.bfloat16, (nt, hq, d), "q_out", dev), pp, dt, k_scale, v_scale, nb, page, acc,
                   pos)


def _batch(q, kv_pages, block_table, seq_lens, cu_seqlens_q):
    """Addresses and sizes of a batch over the paged cache, its shapes and devices checked."""
    import torch
    dev = q.get_device()
    if q.dtype is not torch.bfloat16 or q.dim() != 3 or not q.is_contiguous():
        _need(q, torch.bfloat16, "q", 3)
    pp, dt, (nb, hkv, page, d2) = _pages(kv_pages, dev)
    if block_table.dim() != 2 or seq_lens.dim() != 1 or cu_seqlens_q.dim() != 1:
        raise ValueError("block_table must have 2 dimensions, seq_lens and cu_seqlens_q 1")
    nt, hq, d = q.shape
    shape, bs = block_table.shape, seq_lens.shape[0]
    if d2 != 2 * d or hkv < 1 or hq % hkv or shape[0] < bs or cu_seqlens_q.shape[0] != bs + 1:
        _check_batch(q, kv_pages, block_table, seq_lens, cu_seqlens_q)
    i32 = torch.int32
    return (dev, q.data_ptr(), pp, dt, _fits(block_table, i32, shape, "block_table", dev),
            _fits(seq_lens, i32, (bs,), "seq_lens", dev), _fits(cu_seqlens_q, i32, (bs + 1,), "cu_seqlens_q", dev), nt,
            hq, d, nb, hkv, page, bs, shape[1])


def sk_prefill_workspace_bytes(num_tokens: int, num_q_heads: int, kv_dtype: int) -> int:
    """Bytes of device workspace that sk_paged_prefill_attn needs on the current device (computed by the library)."""
    return _check(lib().sk_prefill_workspace_bytes(num_tokens, num_q_heads, kv_dtype), "sk_prefill_workspace_bytes")


def _raw_stream(device, stream):
    """The handle of ``stream``, by default of the current one of ``device``."""
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index) if device.type == "cuda" else 0
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_object(stream, device):
    import torch
    if stream is None:
        return torch.cuda.current_stream(device)
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)


def _owned_by(stream, device):
    """Context in which memory for a call on ``stream`` is taken: it belongs to that stream, so that it is not handed
    out again to another one while the call's kernels still use it."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(_stream_object(stream, device))


def _buffer(ws, key, need, device, stream):
    """A byte buffer of at least ``need`` bytes, kept in the workspace dict.  One that has become too small stays in
    the dict as well, for a captured graph may hold its address; sizes at least double, so that all of them together
    take no more than twice the last.  A call on another stream than the one that the buffer was taken on is recorded,
    so that its memory is not handed out again while that stream uses it."""
    import torch
    t = ws.get(key)
    raw = _raw_stream(device, stream)
    if t is None or t.numel() < need or t.device != device:
        if t is not None:
            ws.setdefault("outgrown", []).append(t)
            need = max(need, 2 * t.numel())
        with _owned_by(stream, device):
            t = ws[key] = torch.empty(need, dtype=torch.uint8, device=device)
        ws[key + "_streams"] = {raw}
    elif raw not in ws.setdefault(key + "_streams", set()):
        t.record_stream(_stream_object(stream, device))
        ws[key + "_streams"].add(raw)                # once is enough: it lasts until the memory is free
    return t.data_ptr()


def sk_paged_prefill_attn(q, kv_pages, block_table, seq_lens, cu_seqlens_q, out, lse=None, *, max_q_len: int,
                          sm_scale: float, max_seq_len: Optional[int] = None, k_scale: float = 1.0,
                          v_scale: float = 1.0, causal: bool = True, workspace=None, stream=None) -> int:
    """Attention of a chunk of new tokens over the paged cache into ``out`` (bf16 [num_tokens, num_q_heads, 128])
    and ``lse`` (fp32 [num_tokens, num_q_heads], or None).  ``max_seq_len`` bounds seq_lens (default: what the block
    table holds) and decides how the work is divided.  ``workspace`` is an optional dict that keeps the call's
    buffer (and those that it outgrew, which captured graphs may use); calls that may overlap need one each."""
    import torch
    dev, pq, pp, dt, pb, ps, pc, nt, hq, d, nb, hkv, page, bs, stride = _batch(q, kv_pages, block_table, seq_lens,
                                                                               cu_seqlens_q)
    po = _fits(out, torch.bfloat16, (nt, hq, d), "out", dev)
    pl = None if lse is None else _fits(lse, torch.float32, (nt, hq), "lse", dev)
    buf, need = None, 0
    if dev >= 0:
        if torch.cuda.current_device() == dev:
            need = sk_prefill_workspace_bytes(nt, hq, dt)
        else:
            with torch.cuda.device(dev):
                need = sk_prefill_workspace_bytes(nt, hq, dt)
        buf = _buffer(workspace if workspace is not None else {}, "prefill", need, q.device, stream)
    return _launch(dev, stream, "sk_paged_prefill_attn", lib().sk_paged_prefill_attn, pq, pp, dt, k_scale, v_scale, pb,
                   stride, nb, page, ps, pc, bs, nt, max_q_len, hq, hkv, d, sm_scale, 1 if causal else 0,
                   stride * page if max_seq_len is None else max_seq_len, buf, need, po, pl)


def paged_prefill_attention(q, kv_pages, block_table, seq_lens, cu_seqlens_q, *, max_q_len: int, sm_scale: float,
                            max_seq_len: Optional[int] = None, k_scale: float = 1.0, v_scale: float = 1.0,
                            causal: bool = True, workspace=None, out=None, lse=None, stream=None):
    """One attention call of a chunk of new tokens (prompts, chunks of prompts, follow-up turns; cross attention when
    not ``causal``) over the paged cache; arguments as sk_paged_prefill_attn.  Returns (out bf16 [NT, H_q, 128], lse
    fp32 [NT, H_q])."""
    import torch
    nt, hq, d = q.shape
    if out is None or lse is None:
        with _owned_by(stream, q.device):
            if out is None:
                out = torch.empty((nt, hq, d), dtype=torch.bfloat16, device=q.device)
            if lse is None:
                lse = torch.empty((nt, hq), dtype=torch.float32, device=q.device)
    sk_paged_prefill_attn(q, kv_pages, block_table, seq_lens, cu_seqlens_q, out, lse, max_q_len=max_q_len,
                          sm_scale=sm_scale, max_seq_len=max_seq_len, k_scale=k_scale, v_scale=v_scale, causal=causal,
                          workspace=workspace, stream=stream)
    return out, lse


def sk_accum_workspace_bytes(num_tokens: int, num_q_heads: int, num_kv_heads: int, max_q_len: int, kv_dtype: int) -> int:
    """Bytes of device workspace that sk_accum_attn_weights needs (computed by the library)."""
    return _check(lib().sk_accum_workspace_bytes(num_tokens, num_q_heads, num_kv_heads, max_q_len, kv_dtype),
                  "sk_accum_workspace_bytes")


def sk_accum_attn_weights(q, kv_pages, block_table, seq_lens, cu_seqlens_q, lse, acc_pages, *, max_q_len: int,
                          sm_scale: float, k_scale: float = 1.0, causal: bool = True, workspace=None,
                          stream=None) -> int:
    """Adds to ``acc_pages`` (fp32 [num_blocks, num_kv_heads, page]) the attention weight that each cached key
    receives from this step's query tokens: exp(score - lse) summed over the tokens that see it and the
    heads of its group, ``lse`` (fp32 [num_tokens, num_q_heads]) being what the attention call returned.
    ``workspace`` is an optional dict that keeps the call's buffer; calls that may overlap need one each."""
    import torch
    dev, pq, pp, dt, pb, ps, pc, nt, hq, d, nb, hkv, page, bs, stride = _batch(q, kv_pages, block_table, seq_lens,
                                                                               cu_seqlens_q)
    pl = _fits(lse, torch.float32, (nt, hq), "lse", dev)
    pa = _fits(acc_pages, torch.float32, (nb, hkv, page), "acc_pages", dev)
    buf, need = None, 0
    if dev >= 0:
        need = sk_accum_workspace_bytes(nt, hq, hkv, max_q_len, dt)
        if need:
            buf = _buffer(workspace if workspace is not None else {}, "accum", need, q.device, stream)
    return _launch(dev, stream, "sk_accum_attn_weights", lib().sk_accum_attn_weights, pq, pp, dt, k_scale, pb, stride,
                   nb, page, ps, pc, bs, nt, max_q_len, hq, hkv, d, sm_scale, 1 if causal else 0, pl, pa, buf, need)


def sk_evict_capacity(budget: int, max_seq_len: int) -> int:
    """Smallest length of the move lists (computed by the library)."""
    return _check(lib().sk_evict_capacity(int(budget), int(max_seq_len)), "sk_evict_capacity")


def sk_evict_select(acc_pages, pos_pages, block_table, seq_lens, next_pos, src_rows, dst_rows, counts, new_lens, *,
                    budget: int, recent: int = 0, max_seq_len: Optional[int] = None, stream=None) -> int:
    """Which ``budget`` rows of each (sequence, KV head) stay: the rows of the last ``recent`` positions, then
    those with the largest weight.  Writes the moves that bring the staying rows below row ``budget``
    (src_rows, dst_rows int32 [bs, num_kv_heads, capacity], counts int32 [bs, num_kv_heads]) and the
    new lengths; see sk_evict_move.  ``max_seq_len`` bounds the lengths (default: what the block table
    holds)."""
    import torch
    dev = acc_pages.get_device()
    _need(acc_pages, torch.float32, "acc_pages", 3)
    nb, hkv, page = acc_pages.shape
    bs, cap = seq_lens.numel(), src_rows.shape[-1]
    if block_table.dim() != 2 or block_table.shape[0] < bs:
        raise ValueError(f"block_table has shape {tuple(block_table.shape)} for {bs} sequences")
    stride = block_table.shape[1]
    if max_seq_len is None:
        max_seq_len = stride * page
    pl, pn = _fits(seq_lens, torch.int32, (bs,), "seq_lens", dev), _fits(new_lens, torch.int32, (bs,), "new_lens", dev)
    if pl == pn and bs:
        raise ValueError("new_lens must not be seq_lens itself")
    return _launch(dev, stream, "sk_evict_select", lib().sk_evict_select, acc_pages.data_ptr(),
                   _fits(pos_pages, torch.int32, (nb, hkv, page), "pos_pages", dev),
                   _fits(block_table, torch.int32, block_table.shape, "block_table", dev), stride, nb, page, pl,
                   _fits(next_pos, torch.int32, (bs,), "next_pos", dev), bs, hkv, budget, recent, max_seq_len, cap,
                   _fits(src_rows, torch.int32, (bs, hkv, cap), "src_rows", dev),
                   _fits(dst_rows, torch.int32, (bs, hkv, cap), "dst_rows", dev),
                   _fits(counts, torch.int32, (bs, hkv), "counts", dev), pn)


def sk_evict_move(src_rows, dst_rows, counts, block_table, kv_pages, acc_pages, pos_pages, *, stream=None) -> int:
    """Moves rows src_rows to dst_rows (sk_evict_select's lists) of ``kv_pages``, ``acc_pages`` and
    ``pos_pages``, in place.  Sequences with moves must not share blocks with others (a common prefix): copy those
    first."""
    import torch
    dev = src_rows.get_device()
    _need(src_rows, torch.int32, "src_rows", 3)
    bs, hkv, cap = src_rows.shape
    if block_table.dim() != 2 or block_table.shape[0] < bs:
        raise ValueError(f"block_table has shape {tuple(block_table.shape)} for {bs} sequences")
    pp, dt, (nb, hkv2, page, d2) = _pages(kv_pages, dev)
    if hkv2 != hkv:
        raise ValueError(f"kv_pages has {hkv2} KV heads, the move lists {hkv}")
    return _launch(dev, stream, "sk_evict_move", lib().sk_evict_move, src_rows.data_ptr(),
                   _fits(dst_rows, torch.int32, (bs, hkv, cap), "dst_rows", dev),
                   _fits(counts, torch.int32, (bs, hkv), "counts", dev), cap, bs, hkv, d2 // 2,
                   _fits(block_table, torch.int32, block_table.shape, "block_table", dev), block_table.shape[1], nb,
                   page, pp, dt, _fits(acc_pages, torch.float32, (nb, hkv, page), "acc_pages", dev),
                   _fits(pos_pages, torch.int32, (nb, hkv, page), "pos_pages", dev))


def _move_lists(ws, bs, hkv, cap, device, stream):
    """src_rows, dst_rows and counts of an eviction in the workspace dict: those that are there where they fit, else cut from
    a kept buffer."""
    import torch
    names, i32 = ("src_rows", "dst_rows", "counts"), torch.int32
    src, dst, counts = found = [ws.get(name) for name in names]
    shape = (bs, hkv, cap if src is None or src.dim() != 3 else max(cap, src.shape[2]))
    fit = all(t is not None and t.dtype is i32 and t.device == device and t.is_contiguous() for t in found) and \
        src.shape == shape and dst.shape == shape and counts.shape == shape[:2]
    own = ws.get("evict")
    if fit and (own is None or src.data_ptr() != own.data_ptr()):
        return src, dst, counts
    if not fit:
        if own is None:                              # lists of the caller's that are too small stay, as outgrown buffers do
            ws.setdefault("outgrown", []).extend(t for t in found if t is not None)
        shape = (bs, hkv, cap)
    n, m = shape[0] * shape[1] * shape[2], bs * hkv
    _buffer(ws, "evict", 4 * (2 * n + m), device, stream)
    if not fit:
        flat = ws["evict"][:4 * (2 * n + m)].view(i32)
        src, dst, counts = flat[:n].view(shape), flat[n:2 * n].view(shape), flat[2 * n:].view(bs, hkv)
        ws.update(zip(names, (src, dst, counts)))
    return src, dst, counts


def evict_rows(kv_pages, acc_pages, pos_pages, block_table, seq_lens, next_pos, *, budget: int, recent: int = 0,
               max_seq_len: Optional[int] = None, workspace=None, stream=None):
    """One eviction: sk_evict_select and sk_evict_move.  Every sequence longer than ``budget`` is cut down to
    ``budget`` rows per KV head, in place; such a sequence must not share blocks with others (a common prefix: copy
    those blocks first).  ``workspace`` is an optional dict that keeps the lists
    (src_rows, dst_rows, counts, of this call's shapes; ones put there beforehand are used where they fit); calls
    that may overlap need one each.  Returns the new lengths (int32 [bs], a new tensor); the pages past them can be
    handed out again."""
    import torch
    bs, hkv, page = seq_lens.numel(), kv_pages.shape[1], kv_pages.shape[2]
    dev = kv_pages.device
    if max_seq_len is None:
        max_seq_len = block_table.shape[1] * page
    src, dst, counts = _move_lists(workspace if workspace is not None else {}, bs, hkv,
                                   sk_evict_capacity(budget, max_seq_len), dev, stream)
    with _owned_by(stream, dev):
        new_lens = torch.empty_like(seq_lens)
    sk_evict_select(acc_pages, pos_pages, block_table, seq_lens, next_pos, src, dst, counts, new_lens, budget=budget,
                    recent=recent, max_seq_len=max_seq_len, stream=stream)
    sk_evict_move(src, dst, counts, block_table, kv_pages, acc_pages, pos_pages, stream=stream)
    return new_lens


def sk_get_device_status(stream=None, clear: bool = True) -> int:
    """Synchronises and returns the mask of SK_DEV_* bits (0 when clean), the
    timeout bit included: the C call reports a timeout as SK_ERR_TIMEOUT and
    keeps the mask for sk_last_device_status()."""
    L = lib()
    rc = L.sk_get_device_status(_stream(stream), 1 if clear else 0)
    if rc == SK_ERR_TIMEOUT:
        return int(L.sk_last_device_status())
    return _check(rc, "sk_get_device_status")


def paged_decode_attention(q, kv_pages, block_table, seq_lens, cu_seqlens_q, *, max_q_len: int,
                           sm_scale: float, num_sms: int, k_scale: float = 1.0,
                           v_scale: float = 1.0, causal: bool = True, seg_max: int = 64,
                           use_plan: Optional[bool] = None, workspace=None, out=None, lse=None,
                           stream=None) -> Tuple[object, object]:
    """One attention call: plan (bs > 1, or when use_plan is True), split-KV
    attention, LSE merge.  ``workspace`` is an optional dict of preallocated
    buffers (plan, tok_nseg, part_o, part_m, part_l) reused across calls.
    Returns (out bf16 [NT, H_q, D], lse fp32 [NT, H_q])."""
    import torch
    nt, hq, d = q.shape
    hkv = kv_pages.shape[1]
    bs = seq_lens.numel()
    dev = q.device
    ws = workspace if workspace is not None else {}
    if use_plan is None:
        use_plan = bs > 1
    if "part_o" not in ws:
        ws["part_o"] = torch.empty((nt, seg_max, hq, d), dtype=torch.float32, device=dev)
        ws["part_m"] = torch.empty((nt, seg_max, hq), dtype=torch.float32, device=dev)
        ws["part_l"] = torch.empty((nt, seg_max, hq), dtype=torch.float32, device=dev)
    if use_plan and "plan" not in ws:
        ws["plan"] = torch.empty(plan_capacity(bs, hkv, num_sms), dtype=torch.int32, device=dev)
        ws["tok_nseg"] = torch.empty(nt, dtype=torch.int32, device=dev)
    if out is None:
        out = torch.empty((nt, hq, d), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((nt, hq), dtype=torch.float32, device=dev)
    plan = ws["plan"] if use_plan else None
    if use_plan:
        sk_build_plan(seq_lens, cu_seqlens_q, hkv, plan, ws["tok_nseg"], num_sms, seg_max, stream)
    sk_paged_decode_attn(q, kv_pages, block_table, seq_lens, cu_seqlens_q, plan, ws["part_o"],
                         ws["part_m"], ws["part_l"], max_q_len=max_q_len, sm_scale=sm_scale,
                         num_sms=num_sms, k_scale=k_scale, v_scale=v_scale, causal=causal,
                         stream=stream)
    fixed = 0 if use_plan else sk_fixed_nseg(bs, hkv, num_sms, seg_max)
    sk_merge_segments(ws["part_o"], ws["part_m"], ws["part_l"], ws["tok_nseg"] if use_plan else None,
                      out, lse, fixed_nseg=fixed, stream=stream)
    return out, lse
