"""The gated delta rule: linear attention whose state gives up what it holds for a key before it takes the new
value. Over packed prompts and for single tokens, with the conventions of `mixers`."""
from __future__ import annotations

from typing import Optional

import torch

from . import mixers
from .mixers import (_F32, _I32, _TYPES, _check, _empty, _factor, _flat, _guard, _handle, _library, _mixed, _mixer, _need,
                     _rows, _scratch, _short, _state)

__all__ = ["delta_rule", "delta_rule_workspace", "delta_rule_step"]


def _rates(beta, T: int, H: int, dev: int):
    """Strides of beta: float32 [T, H], or [H] where it is the same for every token."""
    if not isinstance(beta, torch.Tensor):
        raise TypeError("beta must be a torch.Tensor")
    per_token = beta.dim() == 2
    _need(beta, "beta", _F32, 2 if per_token else 1, dev)
    if beta.shape != ((T, H) if per_token else (H,)):
        raise ValueError(f"beta must be [{H}] or [{T}, {H}], got {tuple(beta.shape)}")
    st = beta.stride()
    return (st[0] if per_token and T > 1 else 0), st[-1]


def delta_rule_workspace(q: torch.Tensor, v: torch.Tensor, num_seqs: int = 1) -> torch.Tensor:
    """Scratch memory for delta_rule over the tokens of q and v in `num_seqs` sequences, or over fewer tokens or
    sequences: 31 KB for every 64 tokens and head (2 GB for 131072 tokens of 32 heads), and for every sequence and head."""
    need = _library().w4a16_delta_rule_workspace(q.shape[0], num_seqs, v.shape[1], q.shape[2], v.shape[2], _TYPES[q.dtype])
    return torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)


def delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, beta: torch.Tensor,
               cu_seqlens: Optional[torch.Tensor] = None, state: Optional[torch.Tensor] = None,
               state_out: Optional[torch.Tensor] = None, scale: Optional[float] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """The gated delta rule over packed sequences, for prompts: S_t = e^g_t S_{t-1} + k_t u_t^T,
    u_t = beta_t (v_t - e^g_t S_{t-1}^T k_t), o_t = scale * q_t^T S_t.

    q, k [T, Hk, Dk] and v [T, H, Dv] bfloat16 or float16 (head h reads q and k of head h / (H / Hk); keys
    of norm 1 are meant); log_decay and beta float32 [T, H], or [H] where fixed for each head; cu_seqlens int32
    [num_seqs + 1] on the GPU, or None for one sequence: not decreasing (linear_attention makes its own so, here tokens
    and states of a list that decreases are undefined), and clamped to the tokens; state float32 [num_seqs, H, Dk, Dv],
    or None for zeros. scale defaults to Dk ** -0.5. Returns (out [T, H, Dv], state_out), where state_out may be `state` itself.
    `workspace` (delta_rule_workspace, 31 KB for every 64 tokens and head) may be kept for all calls on one stream;
    without it a call allocates that much."""
    if out is not None and state_out is not None and workspace is not None and stream is None:
        _library()
        if _short(mixers._binding.delta_rule(q, k, v, log_decay, beta, cu_seqlens, state, state_out, _factor(scale, q),
                                             out, workspace), "w4a16_delta_rule"):
            return out, state_out
    dev, T, Hk, H, Dk, Dv, ldg, hsg = _mixer(q, k, v, log_decay)
    ldb, hsb = _rates(beta, T, H, dev)
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
        need = 0 if workspace is not None else lib.w4a16_delta_rule_workspace(T, seqs, H, Dk, Dv, _TYPES[q.dtype])
        workspace, at, room = _scratch(workspace, need, dev, stream)
        _check(lib.w4a16_delta_rule(
            q.data_ptr(), ldq, hsq, k.data_ptr(), ldk, hsk, v.data_ptr(), ldv, hsv, log_decay.data_ptr(), ldg, hsg,
            beta.data_ptr(), ldb, hsb, None if cu_seqlens is None else cu_seqlens.data_ptr(), seqs, T, Hk, H, Dk, Dv,
            _TYPES[q.dtype], Dk ** -0.5 if scale is None else scale, None if state is None else state.data_ptr(),
            state_out.data_ptr(), out.data_ptr(), ldo, hso, at, room, _handle(stream, dev)), "w4a16_delta_rule")
    return out, state_out


def delta_rule_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, beta: torch.Tensor,
                    state: torch.Tensor, slots: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """delta_rule for one new token of each of B requests: q, k [B, Hk, Dk], v [B, H, Dv], log_decay and beta
    [B, H] or [H]. state float32 [num_states, H, Dk, Dv] is updated in place unless state_out is given;
    request b's state is row slots[b] (int32 [B], all different; outside the pool: a zero row and no state) or,
    without slots, row b. Returns out [B, H, Dv]."""
    if out is not None and stream is None:
        _library()
        if _short(mixers._binding.delta_rule_step(q, k, v, log_decay, beta, state, slots,
                                                  state if state_out is None else state_out, _factor(scale, q), out),
                  "w4a16_delta_rule_step"):
            return out
    dev, B, Hk, H, Dk, Dv, ldg, hsg = _mixer(q, k, v, log_decay)
    ldb, hsb = _rates(beta, B, H, dev)
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
        _check(_library().w4a16_delta_rule_step(
            q.data_ptr(), ldq, hsq, k.data_ptr(), ldk, hsk, v.data_ptr(), ldv, hsv, log_decay.data_ptr(), ldg, hsg,
            beta.data_ptr(), ldb, hsb, None if slots is None else slots.data_ptr(), rows, B, Hk, H, Dk, Dv,
            _TYPES[q.dtype], Dk ** -0.5 if scale is None else scale, state.data_ptr(), state_out.data_ptr(),
            out.data_ptr(), ldo, hso, _handle(stream, dev)), "w4a16_delta_rule_step")
    return out
