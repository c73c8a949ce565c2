"""Linear attention over operands of every size: what a type's range or a rounding term could lose.

Bounds of single elements are mixer_oracle's. Those of a whole state are of its norm: with b the largest sum of
log decays that stands in an exponent, a factor e^b is off by b half steps of float32 (its exponent's rounding) and
two of the exponential, its product with v by one, what the terms of the type leave by one, and sums by fewer than
twelve, as they are rounded at random: (b + 16) 2^-24. (One bfloat16 term fewer is off by 40 of those.)
"""
import math

import pytest
import torch

import mixer_oracle as mo
import weight_only_int4_w4a16_amd as w
from test_gpu_linear_attention import Linear

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def check(x, out, state, exponent=0.0):
    """Elements by their bounds, each sequence's state also by its norm."""
    assert bool(out.isfinite().all()) and bool(state.isfinite().all())
    x.check(out, state)
    at = x.lead
    for s, n in enumerate(x.lens):
        g = x.g[at:at + n] if x.g.dim() == 2 else x.g.expand(n, x.H)
        S0 = torch.zeros(state.shape[1:]).double() if x.state is None else x.state[s].double()
        _, S, _, _ = mo.linear(x.q[at:at + n].double(), x.k[at:at + n].double(), x.v[at:at + n].double(), g.double(),
                               S0, x.scale)
        for h in range(x.H):
            off = float((state[s, h].cpu().double() - S[h]).norm() / S[h].norm())
            assert off <= (exponent + 16) * mo.F32, f"sequence {s}, head {h}: state off by {off:.3g} of its norm"
        at += n


@pytest.mark.parametrize("n", [1, 40, 200])
@pytest.mark.parametrize("size,v_size", [(32.0, 0.01), (100.0, 1e-3)])
def test_scores_past_the_range_of_float16(n, size, v_size):
    """Scores of 1e5 and more with small values: outputs that float16 holds."""
    torch.manual_seed(n)
    x = Linear([n], 2, 1, 128, 64, FP16, seed=n, rate=0.2)
    x.scale = 32.0 / size
    x.q = (size * (1 + 0.1 * torch.randn(x.q.shape))).to(FP16)
    x.k = (size * (1 + 0.1 * torch.randn(x.k.shape))).to(FP16)
    x.v = (v_size * torch.randn(x.v.shape)).to(FP16)
    x.v[:, :, 0] = 0
    x.state *= v_size * size
    out, state = x.run(scale=x.scale)
    check(x, out, state)
    if n == 40:   # token by token, in float32
        q, k, v, g, s = (t.cuda() for t in (x.q, x.k, x.v, x.g, x.state))
        rows = torch.cat([w.linear_attention_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], s, scale=x.scale)
                          for t in range(n)])
        x.check(rows, s)


def test_rows_of_every_size():
    """Neighbouring queries and keys that differ by powers of two, scores among float16's subnormals and below."""
    x = Linear([200], 2, 2, 64, 64, FP16, seed=3, rate=0.02, initial=False)
    t = torch.arange(200)
    x.q = (x.q.float() * (2.0 ** -(t % 16))[:, None, None]).to(FP16)
    x.k = (x.k.float() * (2.0 ** -(8 + t % 3))[:, None, None]).to(FP16)
    x.v = (x.v.float() * 1000).to(FP16)
    x.scale = 1.0
    check(x, *x.run(scale=1.0))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("amp", [1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("n", [200, 700])
def test_small_queries_and_keys(dtype, amp, n):
    x = Linear([n], 2, 1, 128, 128, dtype, seed=n, rate=0.02, initial=False)
    x.q, x.k = ((t.float() * amp).to(dtype) for t in (x.q, x.k))
    x.scale = 0.1 / amp ** 2
    check(x, *x.run(scale=x.scale))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("n", [200, 700])
def test_small_values(dtype, n):
    """Values among float16's subnormals, beside keys that bring them up; then large ones."""
    torch.manual_seed(n)
    x = Linear([n], 2, 1, 128, 128, dtype, seed=n, rate=0.02, initial=False, amp=30.0)
    x.v = (x.v.float() / 30 * 1e-6).to(dtype)
    check(x, *x.run())
    x.v[150:] = (torch.randn(x.v[150:].shape) * 100).to(dtype)
    x.q = (x.q.float() * 1e-3).to(dtype)
    check(x, *x.run())
    x.v = x.v.flip(0)
    check(x, *x.run())


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("n,growth,cleared", [(64, 0.1, ()), (130, 0.3, ()), (1500, 0.01, ()), (2500, 0.02, ()),
                                              (700, 0.05, (100, 300, 520))])
def test_growth(dtype, n, growth, cleared):
    """Positive log decays: factors of e^6 to e^50 stand before values of hundreds."""
    torch.manual_seed(n)
    x = Linear([n], 2, 1, 64, 64, dtype, seed=n)
    x.v = (x.v.float() * 200).to(dtype)
    x.g = growth * (0.9 + 0.2 * torch.rand(x.g.shape))
    x.g[list(cleared)] = -math.inf
    total = n * growth
    x.scale = 0.1 * math.exp(-total)
    check(x, *x.run(scale=x.scale), exponent=1.1 * total * 1.443)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("lens", [[200], [1500, 70], [3, 64, 129]])
def test_digits_of_states(dtype, lens):
    """States to float32's digits: every term of the products that return them counts."""
    x = Linear(lens, 2, 1, 128, 128, dtype, seed=sum(lens), rate=0.02, initial=False)
    check(x, *x.run())
    x = Linear(lens, 2, 1, 128, 128, dtype, seed=sum(lens), rate=0.0)
    check(x, *x.run())


@pytest.mark.parametrize("dtype,n,size,growth", [
    (BF16, 60, 1e30, 80.0), (BF16, 130, 1e30, 80.0), (BF16, 700, 1e30, 80.0), (BF16, 700, 1e37, 20.0),
    (FP16, 130, 1e37, 20.0), (FP16, 700, 1e37, 20.0),
])
@pytest.mark.parametrize("g0", [-math.inf, -1e4])
def test_cleared_before_growth(dtype, n, size, growth, g0):
    """A decay of zero counts as such when the ones after it grow."""
    x = Linear([n], 2, 2, 64, 64, dtype, seed=n)
    x.g = torch.full((n, 2), growth / (n - 1))
    x.g[0] = g0
    x.k[:-1] = 0
    x.state *= size
    x.check(*x.run())


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_large_first_state(dtype):
    """A first state of 1e30 beside ordinary tokens, which decays away."""
    x = Linear([500, 70], 2, 2, 64, 128, dtype, seed=9, rate=2.0)
    x.state *= 1e30
    x.scale = 1e-30
    check(x, *x.run(scale=x.scale), exponent=700.0)
