"""Paged attention beside a sink: one position far ahead of the others whose value is near zero."""
import math

import pytest
import torch

import mixer_oracle as mo
from test_gpu_paged_attention import Paged, ints

pytestmark = pytest.mark.gpu


def sink(p, ahead, scale, at=0):
    """Makes position `at` of every request `ahead` nats ahead of the rest, with a value of zero."""
    D = p.q.shape[2]
    p.q[:] = 0
    p.q[:, :, 0] = 1.0
    for b, n in enumerate(p.lens):
        for j in range(n):
            page, slot = p.table[b][j // p.page], j % p.page
            k = torch.zeros(p.k.shape[2], D)
            if j == at:
                k[:, 0] = ahead / scale
            p.k[page, slot] = k.to(p.k.dtype).cuda()
            p.rows[0][b][j] = k.to(p.k.dtype).double()
            if j == at:
                p.v[page, slot] = 0
                p.rows[1][b][j] = 0
    return p


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,at", [(30, 0), (700, 0), (700, 699), (4000, 2000)])
@pytest.mark.parametrize("ahead", [8.0, 11.0, 14.0, 17.0, 18.0, 22.0])
def test_positions_behind_a_sink(dtype, n, at, ahead):
    scale = 0.125
    p = Paged([n], 4, 2, 64, 16, dtype, seed=n, amp=0.5)
    for rows in p.rows[1]:   # values of one sign and some size, so that the outputs are normal
        rows.abs_().mul_(2.0 ** 14)
    p.v.copy_((p.v.float().abs() * 2.0 ** 14).to(dtype))
    sink(p, ahead, scale, at)
    out, sums = p.run(scale)
    # relative to the value: the weights' rounding (all alike here) and the output's, and float32 sums; half a
    # step of float16's subnormals for the output, and for each weight of at most 2^15 (2^-40 of the largest)
    o, lse, _, _, _ = mo.attention(p.q[0].double(), p.rows[0][0], p.rows[1][0], scale)
    off = (out[0].cpu().double() - o).abs()
    noise = (n + 64) * mo.F32 + 2.0 ** -20 + 8 * mo.F32 * (ahead + 1)
    tiny = 2.0 ** -25 + 2.0 ** -40 * float(p.rows[1][0].sum(0).max()) if dtype == torch.float16 else 0
    assert bool((off <= (2 * mo.half_step(dtype) + 2 * noise) * o.abs() + tiny).all())
    assert float((sums[0].cpu().double() - lse).abs().max()) <= noise


def test_lengths_and_windows_at_float16():
    """The reference of the weights does not show: empty requests, single positions, windows, several runs."""
    p = Paged([0, 1, 2, 129, 3000], 8, 2, 128, 16, torch.float16, seed=8)
    for window in (0, 1, 200):
        out, sums = p.run(0.09, window=window)
        p.check(out, sums, 0.09, window)
    assert math.isinf(float(sums[0, 0])) and bool((out[0] == 0).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("window", [0, 1, 500, 2 ** 31 - 1])
def test_lengths_below_zero(dtype, window):
    """Lengths down to the least integer are requests without positions, with any window."""
    p = Paged([5, 40, 9], 4, 2, 64, 16, dtype, seed=12)
    out, sums = p.run(0.125, window=window, lens=ints([-2 ** 31, 40, -1]))
    for b in (0, 2):
        assert bool((out[b] == 0).all()) and bool((sums[b] == -math.inf).all())
    p.lens = [0, 40, 0]
    p.rows = [[x[:n] for x, n in zip(rows, p.lens)] for rows in p.rows]
    p.check(out, sums, 0.125, window)
