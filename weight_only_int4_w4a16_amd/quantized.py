"""A paged key-value cache in 8 bits with a scale for each block of tokens and head: rows are quantised as they are
written, read back, and attended to. Conventions of `mixers`, and

  codes   int8 or float8_e4m3fn [pages, page_size, heads, dim], strides as for the caches there
  scales  float32 [pages, page_size / block, heads], any strides; block 16, 32, 48 or 64; value = code * scale

quantized_kv_write makes the scales: 2^-126 or more, or NaN. One that comes from elsewhere must not be negative: its sign
would be lost on reading, and attention would give NaN.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import mixers
from .mixers import (_F32, _HALF, _I32, _P, _TYPES, _Strides, _check, _empty, _factor, _flat, _guard, _handle, _i32, _int32,
                     _library, _need, _rows, _scratch, _short)

__all__ = ["quantized_kv_write", "quantized_kv_read", "quantized_attention", "quantized_attention_workspace"]

_CODES = {torch.int8: 3, torch.float8_e4m3fn: 2}


class _Cache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_stride", _Strides), ("v_stride", _Strides), ("k_scale", _P), ("v_scale", _P),
                ("k_scale_stride", _Strides), ("v_scale_stride", _Strides), ("num_pages", _i32), ("page_size", _i32),
                ("heads", _i32), ("dim", _i32), ("block", _i32), ("type", _i32)]


def _cache_of(k_cache, v_cache, k_scale, v_scale, dev: int) -> _Cache:
    dev = _need(k_cache, "k_cache", tuple(_CODES), 4, dev)
    _need(v_cache, "v_cache", (k_cache.dtype,), 4, dev)
    _need(k_scale, "k_scale", _F32, 3, dev)
    _need(v_scale, "v_scale", _F32, 3, dev)
    shape, blocks = k_cache.shape, k_scale.shape[1]
    if shape != v_cache.shape:
        raise ValueError(f"k_cache {tuple(shape)} and v_cache {tuple(v_cache.shape)} differ in shape")
    if not blocks or shape[1] % blocks:
        raise ValueError(f"{blocks} blocks do not divide a page of {shape[1]}")
    strides = []
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        st = t.stride()
        if st[3] != 1:
            raise ValueError(f"{name} must have unit stride along its last dimension")
        strides.append(_Strides(*[st[i] if shape[i] > 1 else 0 for i in range(3)]))
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t.shape != (shape[0], blocks, shape[2]):
            raise ValueError(f"{name} must be {(shape[0], blocks, shape[2])}, got {tuple(t.shape)}")
        strides.append(_Strides(*t.stride()))
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), strides[0], strides[1], k_scale.data_ptr(), v_scale.data_ptr(),
                  strides[2], strides[3], shape[0], shape[1], shape[2], shape[3], shape[1] // blocks,
                  _CODES[k_cache.dtype])


def quantized_kv_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       k_scale: torch.Tensor, v_scale: torch.Tensor, slot_map: torch.Tensor, stream=None) -> None:
    """Quantises k and v [T, heads, dim] (bfloat16 or float16) to the slots slot_map int32 [T] of a cache of codes.

    Tokens with slots one after the other in a block are a run, and runs of one call lie in different blocks. A
    run that starts at a block's first slot starts the block anew, with the scale largest |x| / 127 (int8) or / 448
    (e4m3) of each head; another one raises the block's scale where it has to, and the codes that the block holds
    go over to it. A sequence is thus written from its first position on, in any number of calls (one that begins in a
    block's middle has the scale that the block had before, at least). Tokens whose slot is outside the cache are
    skipped. A value that is not finite makes NaN of its block and head, until the block is started anew."""
    if stream is None:
        _library()
        if _short(mixers._binding.quantized_kv_write(k, v, k_cache, v_cache, k_scale, v_scale, slot_map),
                  "w4a16_quantized_kv_write"):
            return
    dev = _need(k, "k", _HALF, 3, -1)
    _need(v, "v", (k.dtype,), 3, dev)
    _flat(slot_map, "slot_map", _I32, 1, dev)
    c = _cache_of(k_cache, v_cache, k_scale, v_scale, dev)
    T = slot_map.shape[0]
    if k.shape != v.shape or k.shape != (T, c.heads, c.dim):
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} must be [{T}, {c.heads}, {c.dim}]")
    ldk, hsk = _rows(k, "k")
    ldv, hsv = _rows(v, "v")
    with _guard(dev):
        _check(_library().w4a16_quantized_kv_write(k.data_ptr(), ldk, hsk, v.data_ptr(), ldv, hsv, T, _TYPES[k.dtype],
                                                   slot_map.data_ptr(), ctypes.addressof(c), _handle(stream, dev)),
               "w4a16_quantized_kv_write")


def quantized_kv_read(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                      slot_map: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                      out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, stream=None
                      ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The keys and values [T, heads, dim] that the slots slot_map int32 [T] stand for, rounded to `dtype` (bfloat16
    or float16; that of `out`, a pair, where given); zeros for a slot outside the cache. Slots may repeat."""
    if out is not None and stream is None:
        _library()
        if _short(mixers._binding.quantized_kv_read(k_cache, v_cache, k_scale, v_scale, slot_map, *out),
                  "w4a16_quantized_kv_read"):
            return out
    dev = _flat(slot_map, "slot_map", _I32, 1, -1)
    c = _cache_of(k_cache, v_cache, k_scale, v_scale, dev)
    T = slot_map.shape[0]
    with _guard(dev):
        if out is None:
            if dtype not in _HALF:
                raise TypeError(f"dtype must be {' or '.join(map(str, _HALF))}, got {dtype}")
            out = tuple(_empty((T, c.heads, c.dim), dtype, dev, stream) for _ in range(2))
        k, v = out
        _need(k, "out[0]", _HALF, 3, dev)
        _need(v, "out[1]", (k.dtype,), 3, dev)
        if k.shape != v.shape or k.shape != (T, c.heads, c.dim):
            raise ValueError(f"out {tuple(k.shape)} and {tuple(v.shape)} must be [{T}, {c.heads}, {c.dim}]")
        ldk, hsk = _rows(k, "out[0]")
        ldv, hsv = _rows(v, "out[1]")
        _check(_library().w4a16_quantized_kv_read(ctypes.addressof(c), slot_map.data_ptr(), T, _TYPES[k.dtype],
                                                  k.data_ptr(), ldk, hsk, v.data_ptr(), ldv, hsv, _handle(stream, dev)),
               "w4a16_quantized_kv_read")
    return out


def quantized_attention_workspace(q: torch.Tensor, k_cache: torch.Tensor) -> torch.Tensor:
    """Scratch memory for quantized_attention calls with these head counts and dim, any batch and length."""
    need = _library().w4a16_quantized_attention_workspace(q.shape[1], k_cache.shape[2], k_cache.shape[3])
    return torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)


def quantized_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                        v_scale: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                        scale: Optional[float] = None, window: int = 0, out: Optional[torch.Tensor] = None,
                        lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """paged_attention over a cache of codes: attention of one new token of each request over its cached tokens,
    itself included. q [B, Hq, dim] bfloat16 or float16; page_table int32 [B, max_pages], seq_lens int32 [B],
    window, scale, out and lse as there. `workspace` (quantized_attention_workspace) may be kept for all calls on
    one stream."""
    if out is not None and workspace is not None and stream is None:
        _library()
        if _short(mixers._binding.quantized_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                                                      _factor(scale, q), window, out, lse, workspace),
                  "w4a16_quantized_attention"):
            return out
    window = _int32(window, "window")
    dev = _need(q, "q", _HALF, 3, -1)
    c = _cache_of(k_cache, v_cache, k_scale, v_scale, dev)
    _need(page_table, "page_table", _I32, 2, dev)
    _flat(seq_lens, "seq_lens", _I32, 1, dev)
    B, Hq, dim = q.shape
    pages = page_table.shape[1]
    if page_table.shape[0] != B or seq_lens.shape[0] != B or c.dim != dim:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, cache {tuple(k_cache.shape)}, page_table "
                         f"{tuple(page_table.shape)}, seq_lens {tuple(seq_lens.shape)}")
    if pages > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table must have unit stride along its rows")
    ldq, hsq = _rows(q, "q")
    lib = _library()
    with _guard(dev):
        if out is None:
            out = _empty((B, Hq, dim), q.dtype, dev, stream)
        else:
            _need(out, "out", (q.dtype,), 3, dev)
            if out.shape != q.shape:
                raise ValueError(f"out must be {tuple(q.shape)}, got {tuple(out.shape)}")
        ldo, hso = _rows(out, "out")
        if lse is not None:
            _flat(lse, "lse", _F32, 2, dev)
            if lse.shape != (B, Hq):
                raise ValueError(f"lse must be {(B, Hq)}, got {tuple(lse.shape)}")
        need = 0 if workspace is not None else lib.w4a16_quantized_attention_workspace(Hq, c.heads, dim)
        workspace, at, room = _scratch(workspace, need, dev, stream)
        _check(lib.w4a16_quantized_attention(
            q.data_ptr(), ldq, hsq, _TYPES[q.dtype], ctypes.addressof(c), page_table.data_ptr(),
            page_table.stride(0) if B > 1 else pages, pages, seq_lens.data_ptr(), B, Hq,
            dim ** -0.5 if scale is None else scale, window, out.data_ptr(), ldo, hso,
            None if lse is None else lse.data_ptr(), at, room, _handle(stream, dev)), "w4a16_quantized_attention")
    return out
