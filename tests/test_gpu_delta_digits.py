"""Digits of the delta rule's outputs, against float64.

Both parts of an output, q^T S and the scores' product with U, take two bfloat16 values of each of their operands
(half steps of 2^-8 of the value, squared: 2^-16) and leave out the product of both second ones (2^-16): each operand
and that product moves a term by 2^-16 of it at most, with a sign that does not follow the term's. Terms and their errors
then add alike, as squares, and the outputs are off by 3 * 2^-16 of their norm at most before they are rounded. An error x
moves what rounding leaves by 2 |x| at most: where it changes the rounded value, both neighbours are half a step away but
for |x|."""
import pytest
import torch

import delta_oracle as do
import quantized_oracle as qo
from test_gpu_delta_rule import BF, FP, Delta

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,rate,alike", [(60, 0.1, 0.0), (1920, 0.01, 0.0), (700, 0.5, 0.6)])
def test_outputs_are_off_by_their_own_rounding(dtype, n, rate, alike):
    x = Delta([n], 4, 2, 128, 128, dtype, seed=n, rate=rate, alike=alike)
    out, _ = x.run()
    o, _, _, _ = do.delta(x.q.double(), x.k.double(), x.v.double(), x.g.double(), x.beta.double(), x.state[0].double(), x.scale)
    own = float((qo.rounded(o, dtype) - o).norm() / o.norm())
    got = float((out.cpu().double() - o).norm() / o.norm())
    print(f"{own:.4g} {got:.4g}")
    assert got <= own + 6 * 2.0 ** -16
