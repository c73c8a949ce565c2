"""One workspace, made for the largest prompt, for all shorter ones."""
import pytest
import torch

import weight_only_int4_w4a16_amd as w
from test_gpu_linear_attention import Linear

pytestmark = pytest.mark.gpu


def test_one_workspace_for_every_length():
    big = Linear([4128], 8, 8, 64, 64, seed=1)
    work = w.linear_attention_workspace(big.q.cuda(), big.v.cuda(), 3)
    x = Linear([4096], 8, 8, 64, 64, seed=2, rate=0.02)   # takes more segments than 4128 tokens do
    out, state = x.run(workspace=work)
    again, state2 = x.run()
    assert torch.equal(out, again) and torch.equal(state, state2)
    for lens in ([700], [300, 0, 129], [1, 513], [255]):
        y = Linear(lens, 8, 8, 64, 64, seed=sum(lens))
        y.check(*y.run(workspace=work))
    with pytest.raises(w.W4A16Error, match="workspace"):
        x.run(workspace=work[:work.numel() // 8])
