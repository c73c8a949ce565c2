"""Plain float64 definitions of the token mixers, on the CPU, with the bounds that their tests use.

Nothing here shares code with the HIP path. Roundings are counted as half a step of the type
(`half_step`) relative to the value; sums in float32 as one half step for each addition.
"""
import math

import torch

F32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def page_tables(ctx, new, table, free, page, max_tokens):
    """The lists that w4a16_page_tables writes, by walking over requests and tokens."""
    most = 2 ** 31 - 1
    table = [list(r) for r in table]
    seq, cu, slots, pos, taken = [], [0], [], [], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(c, 0), max(n, 0)
        p0, p1 = min(-(-c // page), len(table[b])), min(-(-(c + n) // page), len(table[b]))
        for j in range(p0, p1):
            table[b][j] = free[taken] if taken < len(free) else -1
            taken += 1
        seq.append(min(c + n, most))
        cu.append(min(cu[-1] + n, most))
        for i in range(c, c + n):
            if len(slots) >= max_tokens:
                break
            j = i // page
            held = table[b][j] if j < len(table[b]) else -1
            s = held * page + i % page
            slots.append(s if held >= 0 and s <= most else -1)
            pos.append(min(i, most))
    slots += [-1] * (max_tokens - len(slots))
    pos += [-1] * (max_tokens - len(pos))
    return seq, cu, slots, pos, [cu[-1], taken], table


def attention(q, k, v, scale, lo=0):
    """One request: q [Hq, D], k and v [n, Hkv, D] as float64 values, positions lo..n-1. Returns
    (out, lse, sum of p |v|, largest sum of |q k| * scale, largest |score|) with NaN kept out of nothing."""
    n, Hkv, D = k.shape
    Hq = q.shape[0]
    if n <= lo:
        z = torch.zeros(Hq, D, dtype=torch.float64)
        return z, torch.full((Hq,), -math.inf, dtype=torch.float64), z, 0.0, 0.0
    out, lse, mag, qk, top = [], [], [], 0.0, 0.0
    for h in range(Hq):
        g = h // (Hq // Hkv)
        s = (k[lo:, g] @ q[h]) * scale
        p = torch.softmax(s, 0)
        out.append(p @ v[lo:, g])
        mag.append(p @ v[lo:, g].abs())
        lse.append(torch.logsumexp(s, 0))
        qk = max(qk, float((k[lo:, g].abs() @ q[h].abs()).max()) * abs(scale))
        top = max(top, float(s.abs().max()))
    return torch.stack(out), torch.stack(lse), torch.stack(mag), qk, top


def attention_bounds(dtype, out, mag, qk, top, n, D):
    """Largest errors of out and lse: scores are float32 sums of D products (times a scale and log2 e,
    rounded), e^x is off by a few float32 steps, the probabilities are rounded to `dtype` for their
    product with v, sums over n positions are float32, out is rounded once."""
    u = half_step(dtype)
    score = (D + 4) * F32 * qk + 8 * F32 * (top + 1)
    sums = (n + 64) * F32 + 2.0 ** -20
    tiny = 2.0 ** -24 if dtype == torch.float16 else 1e-30   # fp16 subnormals: p, and out
    rel = u + 2 * score + 2 * sums
    return u * out.abs() + rel * mag * (1 + u) + tiny, score + sums


def linear(q, k, v, g, state, scale):
    """One sequence: q, k [T, Hk, Dk], v [T, H, Dv], g [T, H], state [H, Dk, Dv], all float64. Returns
    (out, final state) and the same sums with every term's magnitude."""
    T, Hk, _ = q.shape
    H = v.shape[1]
    share = H // Hk
    S, M = state.clone(), state.abs()
    out, mag = [], []
    for t in range(T):
        d = g[t].exp()[:, None, None]
        kt, qt = k[t].repeat_interleave(share, 0), q[t].repeat_interleave(share, 0) * scale
        S = d * S + kt[:, :, None] * v[t][:, None, :]
        M = d * M + (kt[:, :, None] * v[t][:, None, :]).abs()
        out.append((qt[:, :, None] * S).sum(1))
        mag.append((qt.abs()[:, :, None] * M).sum(1))
    if not T:
        z = torch.zeros(0, H, v.shape[2], dtype=torch.float64)
        return z, S, z, M
    return torch.stack(out), S, torch.stack(mag), M


def linear_bounds(dtype, out, mag, M, T):
    """The chunked form: decays and float32 sums as counted; operands of the products that only reach
    `out` are rounded to `dtype` (two of them per term, and q after its decay), those that reach the
    state are two `dtype` values (16 bits of a bfloat16 pair, 22 of a float16 one)."""
    u = half_step(dtype)
    noise = (T + 128) * F32 + 2.0 ** -20
    pair = 2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -20
    tiny = 2.0 ** -24 if dtype == torch.float16 else 1e-30
    return u * out.abs() + (3 * u + noise) * mag * (1 + u) + tiny, (pair + noise) * M + 1e-30


def step_bounds(dtype, out, mag, M, D):
    """The single-token form: float32 throughout, out rounded once."""
    u, noise = half_step(dtype), (D + 16) * F32
    tiny = 2.0 ** -24 if dtype == torch.float16 else 1e-30
    return u * out.abs() + noise * mag * (1 + u) + tiny, 8 * F32 * M + 1e-30
