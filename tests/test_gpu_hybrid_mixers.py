"""Every mixer call of the hybrid example against the float64 definitions, on the operands that it gets there."""
import os
import sys

import pytest
import torch

import mixer_oracle as mo
import weight_only_int4_w4a16_amd as w

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def check_attention(q, k_cache, v_cache, table, lens, k_scale=None, v_scale=None):
    out = w.paged_attention(q, k_cache, v_cache, table, lens, k_scale=k_scale, v_scale=v_scale)
    page = k_cache.shape[1]
    for b, n in enumerate(lens.tolist()):
        at = torch.arange(n, device="cuda")
        where = table[b].long()[at // page]
        rows = []
        for c, s in ((k_cache, k_scale), (v_cache, v_scale)):
            x = c.float()[where, at % page].double()
            rows.append((x if s is None else x * s.double()[:, None]).cpu())
        scale = q.shape[2] ** -0.5
        o, _, mag, qk, top = mo.attention(q[b].cpu().double(), *rows, scale)
        tol, _ = mo.attention_bounds(q.dtype, o, mag, qk, top, n, q.shape[2])
        assert bool(((out[b].cpu().double() - o).abs() <= tol).all()), f"token {b} of length {n}"
    return out


def check_sequence(q, k, v, g, s0, out, s1):
    o, S, mag, M = mo.linear(*(t.cpu().double() for t in (q, k, v, g, s0)), q.shape[2] ** -0.5)
    tol, tol_s = mo.linear_bounds(q.dtype, o, mag, M, q.shape[0])
    assert bool(((out.cpu().double() - o).abs() <= tol).all())
    assert bool(((s1.cpu().double() - S).abs() <= tol_s).all())


def check_linear(q, k, v, g, cu_seqlens, state, state_out):
    before = state.clone()
    out, end = w.linear_attention(q, k, v, g, cu_seqlens=cu_seqlens, state=state, state_out=state_out)
    cu = cu_seqlens.tolist()
    for b in range(len(cu) - 1):
        t = slice(cu[b], cu[b + 1])
        check_sequence(q[t], k[t], v[t], g[t], before[b], out[t], end[b])
    return out, end


def check_step(q, k, v, g, state):
    before = state.clone()
    out = w.linear_attention_step(q, k, v, g, state)
    for b in range(q.shape[0]):
        t = slice(b, b + 1)
        check_sequence(q[t], k[t], v[t], g[t], before[b], out[t], state[b])
    return out


def check_write(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None):
    raw = torch.uint8 if k_cache.dtype == torch.float8_e4m3fn else torch.int16
    want = [c.clone() for c in (k_cache, v_cache)]
    page = k_cache.shape[1]
    for c, x, s in ((want[0], k, k_scale), (want[1], v, v_scale)):
        if s is not None:
            x = (x.float() / s[:, None]).clamp(-448, 448)
        x = x.to(c.dtype)
        at = slots.long()
        assert bool((at >= 0).all())
        c.view(raw)[at // page, at % page] = x.contiguous().view(raw)
    w.paged_kv_write(k, v, k_cache, v_cache, slots, k_scale=k_scale, v_scale=v_scale)
    for c, got in zip(want, (k_cache, v_cache)):
        assert torch.equal(c.view(raw), got.view(raw))


class Checked:
    """The library with its mixers checked."""
    calls = dict(paged_attention=check_attention, linear_attention=check_linear, linear_attention_step=check_step,
                 paged_kv_write=check_write)

    def __init__(self):
        self.seen = set()

    def __getattr__(self, name):
        if name not in self.calls:
            return getattr(w, name)
        self.seen.add(name)
        return self.calls[name]


@pytest.mark.parametrize("cache_type", [torch.bfloat16, torch.float8_e4m3fn])
def test_mixers_of_the_example(cache_type, monkeypatch):
    import hybrid_decode
    lib = Checked()
    monkeypatch.setattr(hybrid_decode, "w", lib)
    model = hybrid_decode.HybridDecoder(requests=3, longest=160, pages=64, seed=6, cache_type=cache_type)
    gen = torch.Generator().manual_seed(7)
    prompts = [torch.randint(0, 1000, (n,), generator=gen).cuda() for n in (70, 3, 17)]
    model.generate(prompts, 4)
    assert lib.seen == set(Checked.calls)
