"""Linear attention over operands of every size: what a type's range could lose. Bounds are mixer_oracle's."""
import pytest
import torch

import weight_only_int4_w4a16_amd as w
from test_gpu_linear_attention import Linear

pytestmark = pytest.mark.gpu

FP16 = torch.float16


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
    x.check(out, state)
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
    x.check(*x.run(scale=1.0))
