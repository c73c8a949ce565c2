"""Attention over the 8-bit cache: digits of its results, and values and scales of every size."""
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
