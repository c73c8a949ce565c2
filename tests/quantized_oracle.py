"""The 8-bit cache with a scale for each block and head, by its definition, on the CPU in float64.

A float64 quotient of a 16-bit value (or a code times a float32 scale) and a float32 scale is on the right side of
every border between two codes, and on it only where the exact one is: both sides of the comparison have at most 32
bits, so they are equal or 2^-32 apart. So are products of codes and scales, which are exact.
"""
import math

import numpy as np
import torch

LARGEST = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
LEAST = 2.0 ** -126


def values(codes):
    """What codes stand for, in units of the scale (float64)."""
    return codes.float().double() if codes.dtype == torch.float8_e4m3fn else codes.double()


def to_codes(x, kind):
    """float64 values in units of the scale -> nearest codes, ties to even."""
    x = x.clamp(-LARGEST[kind], LARGEST[kind])
    if kind == torch.int8:
        return x.round().to(torch.int8)
    _, e = np.frexp(x.numpy())
    unit = np.ldexp(1.0, np.maximum(e, -5) - 4)          # 4 bits, or multiples of 2^-9
    return torch.from_numpy(np.rint(x.numpy() / unit) * unit).to(torch.float32).to(kind)   # exact in both


def rounded(x, dtype):
    """float64 values -> bfloat16 or float16 in one rounding, as float64."""
    if dtype == torch.float16:
        with np.errstate(over="ignore"):
            return torch.from_numpy(x.numpy().astype(np.float16).astype(np.float64))
    _, e = np.frexp(x.numpy())
    unit = np.ldexp(1.0, np.maximum(e, -125) - 8)
    return torch.from_numpy(np.rint(x.numpy() / unit) * unit)


def write(x, codes, scale, slots):
    """Writes rows x [T, heads, dim] into codes [pages, page, heads, dim] and scale [pages, blocks, heads] (float32),
    both in place, by walking over runs."""
    page, blocks, kind = codes.shape[1], scale.shape[1], codes.dtype
    block = page // blocks
    n = codes.shape[0] * page
    t = 0
    while t < len(slots):
        s = slots[t]
        if not 0 <= s < n:
            t += 1
            continue
        end = t + 1
        while end < len(slots) and slots[end] == slots[end - 1] + 1 and slots[end] % block and slots[end] < n:
            end += 1
        p, b, off = s // page, s % page // block, s % block
        rows = x[t:end].double()
        for h in range(codes.shape[2]):
            r = rows[:, h]
            amax = float(r.abs().max())
            here = codes[p, b * block:(b + 1) * block, h]
            old = float(scale[p, b, h])
            if not math.isfinite(amax):
                new = math.nan
            else:
                new = max(float(np.float32(amax / LARGEST[kind])), LEAST)
                if off:
                    new = new if old <= new else old      # NaN stays
            if off and new > old:
                moved = to_codes(values(here) * old / new, kind)
                keep = torch.ones(block, dtype=torch.bool)
                keep[off:off + end - t] = False
                here.view(torch.uint8)[keep] = moved.view(torch.uint8)[keep]
            fresh = to_codes(r / new, kind) if new == new else torch.zeros_like(here[:end - t])
            here.view(torch.uint8)[off:off + end - t] = fresh.view(torch.uint8)
            scale[p, b, h] = new
        t = end


def spread(scale, page):
    """Scales [pages, blocks, heads] for every slot: [pages, page, heads, 1], float64."""
    return scale.double().repeat_interleave(page // scale.shape[1], 1)[..., None]


def read(codes, scale, slots, dtype):
    """The rounded values of the slots, zeros outside."""
    full = (values(codes) * spread(scale, codes.shape[1])).reshape(-1, *codes.shape[2:])
    out = torch.zeros(len(slots), *codes.shape[2:], dtype=torch.float64)
    for t, s in enumerate(slots):
        if 0 <= s < full.shape[0]:
            out[t] = full[s]
    return rounded(out, dtype)


def attention_bounds(dtype, out, mag, qk, top, n, D, weight, most):
    """Largest errors of out and lse of one request: scores are float32 sums of D products, times scales;
    weights (their product with the value's scale, at most `weight` of the normalised ones) are float16,
    2^-11 off or, far below the largest, 2^-40 of it, each with codes up to `most`; sums over n positions are float32."""
    u = torch.finfo(dtype).eps / 2
    F32 = 2.0 ** -24
    score = (D + 6) * F32 * qk + 10 * F32 * (top + 1) + 2.0 ** -32 * qk * D
    sums = (n + 64) * F32 + 2.0 ** -20
    tiny = 2.0 ** -24 if dtype == torch.float16 else 1e-30
    rel = 2.0 ** -11 + 2 * score + 2 * sums
    return u * out.abs() + (rel * mag + 2.0 ** -40 * n * weight * most) * (1 + u) + tiny, score + sums
