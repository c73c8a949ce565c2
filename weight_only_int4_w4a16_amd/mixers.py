"""Token mixers of a decode or prompt step: page tables, the paged key-value cache, attention of one
new token over it, and linear attention with a decay for each head.

Like the rest of the package this only checks and marshals arguments; every step of the computation
runs in the HIP kernels of libw4a16.so, and there is no fallback. Calls whose outputs and scratch are
given, on the current device and stream, go through _binding (C++, a few microseconds less per call);
all others, and all refusals, through the code below.

Tensor conventions:
  caches      [pages, page_size, heads, dim], unit stride along dim, other strides free (a
              [pages, heads, page_size, dim] cache is passed as cache.permute(0, 2, 1, 3)); bfloat16,
              float16, or float8_e4m3fn with float32 [heads] scales (value = code * scale)
  page_table  int32 [B, max_pages]: the pages of each request, in order
  slot_map    int32 [T]: page * page_size + offset of each new token, -1 for none
  states      float32 [B or num_states, heads, Dk, Dv], contiguous
Work runs on `stream` (a torch.cuda.Stream, default: the current one); outputs and scratch that are not
given are allocated for that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import operator
from typing import NamedTuple, Optional

import torch

__all__ = ["PageTables", "page_tables", "page_tables_buffers", "paged_kv_write", "paged_attention",
           "paged_attention_workspace", "linear_attention", "linear_attention_workspace",
           "linear_attention_step"]

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}
_HALF = (torch.bfloat16, torch.float16)
_CACHE = (torch.bfloat16, torch.float16, torch.float8_e4m3fn)
_I32 = (torch.int32,)
_F32 = (torch.float32,)
_i64, _i32, _f32, _P = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p


class _Cache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_stride", _i64 * 3), ("v_stride", _i64 * 3),
                ("k_scale", _P), ("v_scale", _P), ("num_pages", _i32), ("page_size", _i32),
                ("heads", _i32), ("dim", _i32), ("type", _i32)]


_Strides = _i64 * 3
_lib = None
_binding = None


def _library():
    """libw4a16.so with the argument types of this module's entry points; loads _binding as well."""
    global _lib, _binding
    if _lib is None:
        from . import library
        lib = library()
        try:
            from . import _binding as binding
        except ImportError as e:
            raise ImportError("_binding.so is missing or does not load: build it with "
                              "`python -m weight_only_int4_w4a16_amd.build`") from e
        _binding = binding
        _binding.bind(*[ctypes.cast(getattr(lib, "w4a16_" + n), _P).value for n in (
            "page_tables", "paged_kv_write", "paged_attention", "linear_attention", "linear_attention_step")])
        _binding.bind_more(*[ctypes.cast(getattr(lib, "w4a16_" + n), _P).value for n in (
            "delta_rule", "delta_rule_step", "quantized_kv_write", "quantized_kv_read", "quantized_attention")])
        row = [_P, _i64, _i64]
        lib.w4a16_page_tables.argtypes = [_P, _P, _i32, _P, _i64, _i32, _P, _i32, _i32, _i32,
                                          _P, _P, _P, _P, _P, _P]
        lib.w4a16_paged_kv_write.argtypes = row + row + [_i32, _i32, _P, _P, _P]
        lib.w4a16_paged_attention.argtypes = row + [_i32, _P, _P, _i64, _i32, _P, _i32, _i32, _f32,
                                                    _i32] + row + [_P, _P, _i64, _P]
        lib.w4a16_paged_attention_workspace.argtypes = [_i32, _i32, _i32]
        lib.w4a16_paged_attention_workspace.restype = _i64
        lib.w4a16_linear_attention.argtypes = row * 4 + [_P] + [_i32] * 7 + [_f32, _P, _P] + row + [
            _P, _i64, _P]
        lib.w4a16_linear_attention_workspace.argtypes = [_i32] * 5
        lib.w4a16_linear_attention_workspace.restype = _i64
        lib.w4a16_linear_attention_step.argtypes = row * 4 + [_P] + [_i32] * 7 + [_f32, _P, _P] + row + [_P]
        lib.w4a16_delta_rule.argtypes = row * 5 + [_P] + [_i32] * 7 + [_f32, _P, _P] + row + [_P, _i64, _P]
        lib.w4a16_delta_rule_workspace.argtypes = [_i32] * 6
        lib.w4a16_delta_rule_workspace.restype = _i64
        lib.w4a16_delta_rule_step.argtypes = row * 5 + [_P] + [_i32] * 7 + [_f32, _P, _P] + row + [_P]
        lib.w4a16_quantized_kv_write.argtypes = row + row + [_i32, _i32, _P, _P, _P]
        lib.w4a16_quantized_kv_read.argtypes = [_P, _P, _i32, _i32] + row + row + [_P]
        lib.w4a16_quantized_attention.argtypes = lib.w4a16_paged_attention.argtypes
        lib.w4a16_quantized_attention_workspace.argtypes = [_i32, _i32, _i32]
        lib.w4a16_quantized_attention_workspace.restype = _i64
        for f in (lib.w4a16_page_tables, lib.w4a16_paged_kv_write, lib.w4a16_paged_attention,
                  lib.w4a16_linear_attention, lib.w4a16_linear_attention_step, lib.w4a16_delta_rule,
                  lib.w4a16_delta_rule_step, lib.w4a16_quantized_kv_write, lib.w4a16_quantized_kv_read,
                  lib.w4a16_quantized_attention):
            f.restype = ctypes.c_int
        _lib = lib
    return _lib


def _check(status: int, where: str):
    if status != 0:
        from . import W4A16Error
        raise W4A16Error(status, where)


def _need(t, name: str, types, ndim: int, dev: int) -> int:
    """Checks one tensor and returns its device's index (`dev` >= 0: the one it has to be on)."""
    if isinstance(t, torch.Tensor) and t.dtype in types and t.dim() == ndim:
        at = t.get_device()
        if at >= 0 and (dev < 0 or at == dev):
            if max(t.shape, default=0) >= 2 ** 31 and t.dtype != torch.uint8:   # a workspace may be longer
                raise ValueError(f"{name} is too long: {tuple(t.shape)}")
            return at
    _refuse(t, name, types, ndim, dev)


def _refuse(t, name: str, types, ndim: int, dev: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in types:
        raise TypeError(f"{name} must be {' or '.join(map(str, types))}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} must be on a GPU")
    raise ValueError(f"{name} is on GPU {at}, the other operands on GPU {dev}")


def _int32(x, name: str) -> int:
    """x as an int; ctypes would pass 2**32 + 16 on as 16."""
    x = operator.index(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


def _flat(t, name: str, types, ndim: int, dev: int) -> int:
    at = _need(t, name, types, ndim, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return at


_HERE = contextlib.nullcontext()


def _short(status: int, where: str) -> bool:
    """Whether the short way took a call: raises for a refusal of the C entry."""
    if status > 0:
        _check(status, where)
    return status == 0


def _factor(scale, t):
    """scale, or the default for rows like t's; None where neither can be told."""
    if scale is None and isinstance(t, torch.Tensor) and t.dim() == 3 and t.shape[2]:
        return t.shape[2] ** -0.5
    return scale


def _guard(dev: int):
    """Makes `dev` the current device for a launch and its allocations where it is not."""
    return _HERE if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _handle(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _empty(shape, dtype, dev: int, stream):
    """Memory for work on `stream`: its pool's, so that it is not handed out again before that work."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _rows(t, name: str):
    """Strides of [rows, heads, dim] with contiguous rows (a dimension of one has none)."""
    a, b, c = t.stride()
    n, m, d = t.shape
    if c != 1 and d > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return (a if n > 1 else 0), (b if m > 1 else 0)


def _cache_of(k_cache, v_cache, k_scale, v_scale, kind, dev: int) -> _Cache:
    types = (kind, torch.float8_e4m3fn)
    _need(k_cache, "k_cache", types, 4, dev)
    _need(v_cache, "v_cache", (k_cache.dtype,), 4, dev)
    shape = k_cache.shape
    if shape != v_cache.shape:
        raise ValueError(f"k_cache {tuple(shape)} and v_cache {tuple(v_cache.shape)} differ in shape")
    strides = []
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        st = t.stride()
        if st[3] != 1:
            raise ValueError(f"{name} must have unit stride along its last dimension")
        strides.append(_Strides(*[st[i] if shape[i] > 1 else 0 for i in range(3)]))
    scales = []
    for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if s is not None:
            if k_cache.dtype is not torch.float8_e4m3fn:
                raise ValueError(f"{name} goes with a float8_e4m3fn cache")
            _flat(s, name, _F32, 1, dev)
            if s.numel() != shape[2]:
                raise ValueError(f"{name} must have one value for each of {shape[2]} heads")
        scales.append(None if s is None else s.data_ptr())
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), strides[0], strides[1], scales[0], scales[1],
                  shape[0], shape[1], shape[2], shape[3], _TYPES[k_cache.dtype])


class PageTables(NamedTuple):
    """What `page_tables` writes: seq_lens [B], cu_new [B + 1], slot_map and positions [max_tokens],
    counts [2] (new tokens, pages taken), all int32."""
    seq_lens: torch.Tensor
    cu_new: torch.Tensor
    slot_map: torch.Tensor
    positions: torch.Tensor
    counts: torch.Tensor


def page_tables_buffers(batch: int, max_tokens: int, device=None, stream=None) -> PageTables:
    """The outputs of `page_tables` for `batch` requests and at most `max_tokens` new tokens."""
    dev = torch.cuda.current_device() if device is None else torch.device(device).index or 0
    return PageTables(*[_empty(n, torch.int32, dev, stream)
                        for n in (batch, batch + 1, max_tokens, max_tokens, 2)])


def page_tables(ctx_lens: torch.Tensor, new_lens: torch.Tensor, page_table: torch.Tensor,
                free_pages: torch.Tensor, page_size: int, max_tokens: Optional[int] = None,
                out: Optional[PageTables] = None, stream=None) -> PageTables:
    """Page tables and slot maps of one step from the requests' lengths, made on the device.

    Request b holds ctx_lens[b] cached tokens and gets new_lens[b] new ones (int32 [B]). The pages that it
    needs beyond those it has are taken from free_pages (int32) in order of the requests and written
    into its row of page_table (int32 [B, max_pages], in place). Returns, with the new tokens of all
    requests one after the other: the lengths after the step, the requests' first tokens, each
    token's slot and position (-1 past the last token, slot -1 where there is no page), and the
    counts of tokens and pages taken. Give max_tokens or `out`.

    The list is read from its start, and the lengths are not moved on. For the next step copy seq_lens to
    ctx_lens and drop counts[1] pages from the list, on the device (no host round trip, so in a graph as well):
    `at = torch.arange(n) + counts[1]; free.copy_(torch.where(at < n, free[at.clamp(max=n - 1)], -1))`."""
    if out is not None and max_tokens is None and stream is None:
        _library()
        if _short(_binding.page_tables(ctx_lens, new_lens, page_table, free_pages, page_size, *out),
                  "w4a16_page_tables"):
            return out
    page_size = _int32(page_size, "page_size")
    dev = _flat(ctx_lens, "ctx_lens", _I32, 1, -1)
    _flat(new_lens, "new_lens", _I32, 1, dev)
    _need(page_table, "page_table", _I32, 2, dev)
    _flat(free_pages, "free_pages", _I32, 1, dev)
    B = ctx_lens.shape[0]
    if new_lens.shape[0] != B or page_table.shape[0] != B:
        raise ValueError(f"lengths and page_table rows differ: {B}, {new_lens.shape[0]}, "
                         f"{page_table.shape[0]}")
    if page_table.shape[1] > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table must have unit stride along its rows")
    with _guard(dev):
        if out is None:
            if max_tokens is None:
                raise ValueError("give max_tokens or out")
            out = page_tables_buffers(B, max_tokens, dev, stream)
        for t, name in zip(out, PageTables._fields):
            _flat(t, name, _I32, 1, dev)
        seq_lens, cu_new, slot_map, positions, counts = out
        T = slot_map.shape[0]
        if (seq_lens.shape[0] != B or cu_new.shape[0] != B + 1 or counts.shape[0] != 2
                or positions.shape[0] != T or (max_tokens is not None and max_tokens != T)):
            raise ValueError("out does not fit the batch and max_tokens")
        pages = page_table.shape[1]
        _check(_library().w4a16_page_tables(
            ctx_lens.data_ptr(), new_lens.data_ptr(), B, page_table.data_ptr(),
            page_table.stride(0) if B > 1 else pages, pages, free_pages.data_ptr(),
            free_pages.shape[0], page_size, T, seq_lens.data_ptr(), cu_new.data_ptr(),
            slot_map.data_ptr(), positions.data_ptr(), counts.data_ptr(), _handle(stream, dev)),
            "w4a16_page_tables")
    return out


def paged_kv_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   slot_map: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                   v_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """Writes k and v [T, heads, dim] (bfloat16 or float16) to the slots slot_map int32 [T] of a paged
    cache of the same type, or of float8_e4m3fn after division by the head's scale (saturating, to
    nearest even). Tokens whose slot is outside the cache are skipped."""
    if stream is None:
        _library()
        if _short(_binding.paged_kv_write(k, v, k_cache, v_cache, k_scale, v_scale, slot_map),
                  "w4a16_paged_kv_write"):
            return
    dev = _need(k, "k", _HALF, 3, -1)
    _need(v, "v", (k.dtype,), 3, dev)
    _flat(slot_map, "slot_map", _I32, 1, dev)
    c = _cache_of(k_cache, v_cache, k_scale, v_scale, k.dtype, dev)
    T = slot_map.shape[0]
    if k.shape != v.shape or k.shape != (T, c.heads, c.dim):
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} must be [{T}, {c.heads}, {c.dim}]")
    ldk, hsk = _rows(k, "k")
    ldv, hsv = _rows(v, "v")
    with _guard(dev):
        _check(_library().w4a16_paged_kv_write(k.data_ptr(), ldk, hsk, v.data_ptr(), ldv, hsv, T,
                                               _TYPES[k.dtype], slot_map.data_ptr(), ctypes.addressof(c),
                                               _handle(stream, dev)), "w4a16_paged_kv_write")


def _scratch(workspace, need: int, dev: int, stream):
    """(tensor, address, bytes) of a call's scratch memory."""
    if workspace is None:
        workspace = _empty(max(need, 16), torch.uint8, dev, stream)
    else:
        _flat(workspace, "workspace", (torch.uint8,), 1, dev)
    return workspace, workspace.data_ptr(), workspace.shape[0]


def paged_attention_workspace(q: torch.Tensor, k_cache: torch.Tensor) -> torch.Tensor:
    """Scratch memory for paged_attention calls with these head counts and dim, any batch and length."""
    need = _library().w4a16_paged_attention_workspace(q.shape[1], k_cache.shape[2], k_cache.shape[3])
    return torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    page_table: torch.Tensor, seq_lens: torch.Tensor, scale: Optional[float] = None,
                    window: int = 0, k_scale: Optional[torch.Tensor] = None,
                    v_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Attention of one new token of each request over its cached tokens, itself included.

    q [B, Hq, dim] bfloat16 or float16; head h reads KV head h / (Hq / heads). Request b attends to its
    first seq_lens[b] positions (int32 [B]), or the last `window` of them if that is not 0. scale
    defaults to dim ** -0.5. Returns out, like q; lse, float32 [B, Hq], receives log sum exp of the scores.
    A request of length 0 gets zeros and -inf. `workspace` (paged_attention_workspace) may be kept
    for all calls on one stream."""
    if out is not None and workspace is not None and stream is None:
        _library()
        if _short(_binding.paged_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                                           _factor(scale, q), window, out, lse, workspace),
                  "w4a16_paged_attention"):
            return out
    window = _int32(window, "window")
    dev = _need(q, "q", _HALF, 3, -1)
    c = _cache_of(k_cache, v_cache, k_scale, v_scale, q.dtype, dev)
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
        workspace, at, room = _scratch(
            workspace, lib.w4a16_paged_attention_workspace(Hq, c.heads, dim) if workspace is None else 0,
            dev, stream)
        _check(lib.w4a16_paged_attention(
            q.data_ptr(), ldq, hsq, _TYPES[q.dtype], ctypes.addressof(c), page_table.data_ptr(),
            page_table.stride(0) if B > 1 else pages, pages, seq_lens.data_ptr(), B, Hq,
            dim ** -0.5 if scale is None else scale, window, out.data_ptr(), ldo, hso,
            None if lse is None else lse.data_ptr(), at, room, _handle(stream, dev)),
            "w4a16_paged_attention")
    return out


def _mixer(q, k, v, log_decay, dev_first: int = -1):
    """Checks what both linear forms share; returns (device, tokens, Hk, H, Dk, Dv, ldg, hsg)."""
    dev = _need(q, "q", _HALF, 3, dev_first)
    _need(k, "k", (q.dtype,), 3, dev)
    _need(v, "v", (q.dtype,), 3, dev)
    T, Hk, Dk = q.shape
    H, Dv = v.shape[1], v.shape[2]
    if k.shape != q.shape or v.shape[0] != T:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    if not isinstance(log_decay, torch.Tensor):
        raise TypeError("log_decay must be a torch.Tensor")
    per_token = log_decay.dim() == 2
    _need(log_decay, "log_decay", _F32, 2 if per_token else 1, dev)
    if log_decay.shape != ((T, H) if per_token else (H,)):
        raise ValueError(f"log_decay must be [{H}] or [{T}, {H}], got {tuple(log_decay.shape)}")
    st = log_decay.stride()
    return dev, T, Hk, H, Dk, Dv, (st[0] if per_token else 0), st[-1]


def _state(t, name: str, rows: int, H: int, Dk: int, Dv: int, dev: int):
    _flat(t, name, _F32, 4, dev)
    if t.shape != (rows, H, Dk, Dv):
        raise ValueError(f"{name} must be {(rows, H, Dk, Dv)}, got {tuple(t.shape)}")


def _mixed(out, v, dev: int, stream):
    if out is None:
        return _empty(tuple(v.shape), v.dtype, dev, stream)
    _need(out, "out", (v.dtype,), 3, dev)
    if out.shape != v.shape:
        raise ValueError(f"out must be {tuple(v.shape)}, got {tuple(out.shape)}")
    return out


def linear_attention_workspace(q: torch.Tensor, v: torch.Tensor, num_seqs: int = 1) -> torch.Tensor:
    """Scratch memory for linear_attention over the tokens of q and v in `num_seqs` sequences, or over fewer
    tokens or sequences."""
    need = _library().w4a16_linear_attention_workspace(q.shape[0], num_seqs, v.shape[1], q.shape[2],
                                                       v.shape[2])
    return torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)


def linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                     cu_seqlens: Optional[torch.Tensor] = None, state: Optional[torch.Tensor] = None,
                     state_out: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None):
    """Linear attention over packed sequences, for prompts: S_t = e^g_t S_{t-1} + k_t v_t^T,
    o_t = scale * q_t^T S_t.

    q, k [T, Hk, Dk] and v [T, H, Dv] bfloat16 or float16 (head h reads q and k of head h / (H / Hk));
    log_decay float32 [T, H], or [H] for decays fixed for each head; cu_seqlens int32 [num_seqs + 1] on the
    GPU, or None for one sequence; state float32 [num_seqs, H, Dk, Dv], or None for zeros. scale defaults
    to Dk ** -0.5. Returns (out [T, H, Dv], state_out), where state_out may be `state` itself."""
    if out is not None and state_out is not None and workspace is not None and stream is None:
        _library()
        if _short(_binding.linear_attention(q, k, v, log_decay, cu_seqlens, state, state_out,
                                            _factor(scale, q), out, workspace), "w4a16_linear_attention"):
            return out, state_out
    dev, T, Hk, H, Dk, Dv, ldg, hsg = _mixer(q, k, v, log_decay)
    seqs = 1
    if cu_seqlens is not None:
        _flat(cu_seqlens, "cu_seqlens", _I32, 1, dev)
        seqs = cu_seqlens.shape[0] - 1
    if state is not None:
        _state(state, "state", seqs, H, Dk, Dv, dev)
    ldq, hsq = _rows(q, "q")
    ldk, hsk = _rows(k, "k")
    ldv, hsv = _rows(v, "v")
    lib = _library()
    with _guard(dev):
        if state_out is None:
            state_out = _empty((max(seqs, 0), H, Dk, Dv), torch.float32, dev, stream)
        _state(state_out, "state_out", seqs, H, Dk, Dv, dev)
        out = _mixed(out, v, dev, stream)
        ldo, hso = _rows(out, "out")
        need = 0 if workspace is not None else lib.w4a16_linear_attention_workspace(T, seqs, H, Dk, Dv)
        workspace, at, room = _scratch(workspace, need, dev, stream)
        _check(lib.w4a16_linear_attention(
            q.data_ptr(), ldq, hsq, k.data_ptr(), ldk, hsk, v.data_ptr(), ldv, hsv,
            log_decay.data_ptr(), ldg, hsg, None if cu_seqlens is None else cu_seqlens.data_ptr(), seqs,
            T, Hk, H, Dk, Dv, _TYPES[q.dtype], Dk ** -0.5 if scale is None else scale,
            None if state is None else state.data_ptr(), state_out.data_ptr(), out.data_ptr(), ldo, hso,
            at, room, _handle(stream, dev)), "w4a16_linear_attention")
    return out, state_out


def linear_attention_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                          state: torch.Tensor, slots: Optional[torch.Tensor] = None,
                          state_out: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """linear_attention for one new token of each of B requests: q, k [B, Hk, Dk], v [B, H, Dv],
    log_decay [B, H] or [H]. state float32 [num_states, H, Dk, Dv] is updated in place unless state_out is
    given; request b's state is row slots[b] (int32 [B], all different; outside the pool: a zero row and
    no state) or, without slots, row b. Returns out [B, H, Dv]."""
    if out is not None and stream is None:
        _library()
        if _short(_binding.linear_attention_step(q, k, v, log_decay, state, slots,
                                                 state if state_out is None else state_out,
                                                 _factor(scale, q), out), "w4a16_linear_attention_step"):
            return out
    dev, B, Hk, H, Dk, Dv, ldg, hsg = _mixer(q, k, v, log_decay)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a [num_states, H, Dk, Dv] tensor")
    rows = state.shape[0]
    _state(state, "state", rows, H, Dk, Dv, dev)
    if state_out is None:
        state_out = state
    else:
        _state(state_out, "state_out", rows, H, Dk, Dv, dev)
    if slots is not None:
        _flat(slots, "slots", _I32, 1, dev)
        if slots.shape[0] != B:
            raise ValueError(f"slots must have {B} entries, got {slots.shape[0]}")
    ldq, hsq = _rows(q, "q")
    ldk, hsk = _rows(k, "k")
    ldv, hsv = _rows(v, "v")
    with _guard(dev):
        out = _mixed(out, v, dev, stream)
        ldo, hso = _rows(out, "out")
        _check(_library().w4a16_linear_attention_step(
            q.data_ptr(), ldq, hsq, k.data_ptr(), ldk, hsk, v.data_ptr(), ldv, hsv,
            log_decay.data_ptr(), ldg, hsg, None if slots is None else slots.data_ptr(), rows, B, Hk, H, Dk,
            Dv, _TYPES[q.dtype], Dk ** -0.5 if scale is None else scale, state.data_ptr(),
            state_out.data_ptr(), out.data_ptr(), ldo, hso, _handle(stream, dev)),
            "w4a16_linear_attention_step")
    return out
