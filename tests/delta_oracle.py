"""Float64 definition of the gated delta rule, on the CPU, and how far the library's results may be from it.

Errors are counted column by column of the state, as norms of a column: what a block of 64 tokens adds, and
what it passes on of an earlier error (the state's map is e^g (1 - beta k k^T), so by the product of its norms).
Float32 sums of n products are off by n half steps of the magnitudes, values kept as three bfloat16 by one.
"""
import torch

F32 = 2.0 ** -24
CHUNK = 64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def delta(q, k, v, g, beta, state, scale):
    """One sequence in float64: q, k [T, Hk, Dk], v [T, H, Dv], g, beta [T, H], state [H, Dk, Dv]. Returns (out
    [T, H, Dv], final state, u [T, H, Dv], states before every 64th token)."""
    share = v.shape[1] // q.shape[1]
    S, out, us, starts = state.clone(), [], [], []
    for t in range(q.shape[0]):
        if t % CHUNK == 0:
            starts.append(S)
        kt, qt = k[t].repeat_interleave(share, 0), q[t].repeat_interleave(share, 0)
        S = g[t].exp()[:, None, None] * S
        u = beta[t][:, None] * (v[t] - (kt[:, None, :] @ S)[:, 0])
        S = S + kt[:, :, None] * u[:, None, :]
        out.append(scale * (qt[:, None, :] @ S)[:, 0])
        us.append(u)
    if not out:
        z = torch.zeros(0, *v.shape[1:], dtype=torch.float64)
        return z, S, z, starts
    return torch.stack(out), S, torch.stack(us), starts


def bounds(dtype, q, k, v, g, beta, scale, out, u, starts, final):
    """Largest errors of out [T, H, Dv] and of the final state [H, Dk, Dv] of `delta`'s results."""
    share = v.shape[1] // q.shape[1]
    T, H = g.shape
    split = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -15   # scores: one bfloat16 value or two
    tiny = 2.0 ** -24 if dtype == torch.float16 else 1e-30
    E = torch.zeros(H, v.shape[2], dtype=torch.float64)
    tol = torch.zeros_like(out)
    for c, S0 in enumerate(starts):
        at = slice(c * CHUNK, min(T, (c + 1) * CHUNK))
        kk, qq = (x[at].repeat_interleave(share, 1).transpose(0, 1) for x in (k, q))      # [H, n, Dk]
        b = g[at].cumsum(0).T                                                             # [H, n]
        bt, n = beta[at].T.abs(), b.shape[1]
        nk, nq = kk.norm(dim=-1), qq.norm(dim=-1)
        low = torch.ones(n, n, dtype=torch.bool).tril()
        w = torch.where(low, b[:, :, None] - b[:, None, :], -torch.inf).exp()
        A = torch.where(low.tril(-1), beta[at].T[:, :, None] * w * (kk @ kk.transpose(1, 2)), 0.0)
        I = torch.eye(n, dtype=torch.float64)
        Ti = torch.linalg.solve_triangular(I + A, I.expand(H, n, n).contiguous(), upper=False).abs()
        most = torch.where(low.tril(-1), bt[:, :, None] * w * nk[:, :, None] * nk[:, None, :], 0.0)
        Tb, dT = Ti * bt[:, None, :], 300 * F32 * (Ti @ (I + most) @ Ti) * bt[:, None, :]
        s = S0.norm(dim=1) + E                                                            # [H, Dv]
        eb, ed = b.exp(), (b[:, -1:] - b).exp()
        rho = v[at].transpose(0, 1).abs() + (eb * nk)[..., None] * s[:, None]
        du = (272 * F32 * Tb + dT) @ rho
        uu = u[at].transpose(0, 1).abs()
        grow = torch.clamp((1 - bt * nk * nk).abs(), min=1.0).cumprod(1)                  # norms of the maps
        P = w * (qq @ kk.transpose(1, 2)).abs()
        Pn = w * nq[:, :, None] * nk[:, None, :]
        far = (eb * nq)[..., None] * ((2.0 ** -16 + 140 * F32) * s[:, None] + grow[..., None] * E[:, None])
        far = far + P @ (du + (split * (1 + 2.0 ** -8) + 2.0 ** -16 + 70 * F32) * uu) + 200 * F32 * (Pn @ uu)
        tol[at] = half_step(dtype) * out[at].abs() + (abs(scale) * far * (1 + half_step(dtype))).transpose(0, 1) + tiny
        E = (eb[:, -1] * grow[:, -1])[:, None] * E + ((ed * nk)[..., None] * (du + 80 * F32 * uu)).sum(1) \
            + 4 * F32 * eb[:, -1][:, None] * s
    return tol, (E + 2 * F32 * final.norm(dim=1))[:, None, :] + 1e-30


def step_bounds(dtype, q, k, v, g, beta, state, scale, out, final):
    """The single-token form, float32 throughout: requests [B, ...], state [B, H, Dk, Dv]."""
    share = v.shape[1] // q.shape[1]
    kk, qq = (x.repeat_interleave(share, 1) for x in (k, q))
    n = q.shape[2] + 16
    s = g.exp()[..., None] * state.norm(dim=2)
    nk, nq = kk.norm(dim=-1)[..., None], qq.norm(dim=-1)[..., None]
    rho = v.abs() + nk * s
    u = beta.abs()[..., None] * rho
    tiny = 2.0 ** -24 if dtype == torch.float16 else 1e-30
    far = abs(scale) * n * F32 * (nq * s + 3 * nq * nk * u)
    return (half_step(dtype) * out.abs() + far * (1 + half_step(dtype)) + tiny,
            (n * F32 * u)[..., None, :] * kk.abs()[..., None] + 8 * F32 * (state.abs() * g.exp()[..., None, None]
                                                                         + kk.abs()[..., None] * u[..., None, :]) + 1e-30)
