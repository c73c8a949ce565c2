"""Attention over the 8-bit cache: digits of its results, and values and scales of every size."""
import math

import pytest
import torch

import mixer_oracle as mo
import quantized_oracle as qo
from test_gpu_quantized_attention import BF, E4, FP, I8, Attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_outputs_are_off_by_their_own_rounding(kind, dtype):
    """Many weights of like size. Held as two float16 values they are off by 2^-22; scores below 16 and logarithms of scales
    below 16, in powers of two, by a few half steps of 2^-21, sums of 1500 terms by less: below 2^-17 of the norm in all.
    What rounding leaves moves by twice that at most (where it changes the rounded value, both neighbours are half a step
    away but for that)."""
    x = Attend([1500, 700, 130], 16, 4, 128, 32, 16, kind, dtype, seed=30, spread=0.2)
    out, _ = x.run()
    full = [qo.values(c) * qo.spread(s, x.page) for c, s in zip(x.codes, x.scale)]
    want = []
    for b, n in enumerate(x.lens):
        pos = torch.arange(n)
        at = x.table[b, pos // x.page].long()
        want.append(mo.attention(x.q[b].double(), *(t[at, pos % x.page] for t in full), 128 ** -0.5)[0])
    want = torch.stack(want)
    own = float((qo.rounded(want, dtype) - want).norm() / want.norm())
    got = float((out.cpu().double() - want).norm() / want.norm())
    print(f"{own:.4g} {got:.4g}")
    assert got <= own + 2.0 ** -16


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("down", [100, 108, 114])
def test_values_near_the_least_scale(kind, down):
    """Values' scales down to 2^-126: results are those of the same codes with larger scales, times a power of two, but
    for half a step of bfloat16 below its normal numbers (2^-134)."""
    x = Attend([300, 40, 1, 700], 8, 2, 64, 32, 16, kind, BF, seed=31)
    larger = x.scale[1]
    x.scale[1] = (larger * 2.0 ** -down).clamp(min=2.0 ** -126)
    out, lse = x.run()
    x.scale[1] = x.scale[1] * 2.0 ** down
    assert float((x.scale[1] - larger).abs().max()) < 2.0 ** (down - 120)
    assert bool(out.any(-1).all())
    got = out.cpu().double() * 2.0 ** down
    x.check(got, lse)


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("dtype,base", [(FP, -10), (BF, -10), (BF, -45), (BF, 17)])
def test_weights_and_scales_far_apart(kind, dtype, base):
    """One block has the larger weights by 2^30, the other the larger values by 2^30, so that both count alike. Weights alone
    leave float16's range, and so do their products with the scales, which are 2^-45 or 2^17 here."""
    x = Attend([32], 1, 1, 64, 16, 16, kind, dtype, seed=32)
    x.q[:] = 1.0
    p = x.table[0, :2].long()
    x.codes[0] = torch.zeros_like(x.codes[0])
    x.codes[0][p[0], :, :, 0] = torch.tensor(96.0).to(kind)          # a value of both
    x.scale[0][:] = 1.0
    x.scale[1][p[0]], x.scale[1][p[1]] = 2.0 ** base, 2.0 ** (base + 30)
    scale = 30 * math.log(2) / 96
    out, lse = x.run(scale=scale)
    x.check(out, lse, scale=scale)
    x.codes[1][p[0]] = torch.zeros_like(x.codes[1][p[0]])             # the second block alone
    one, _ = x.run(scale=scale)
    assert bool((one != out).any()) and bool(one.any())
    x.check(one, lse, scale=scale)
