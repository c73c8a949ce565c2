"""The README's Python lines run as they stand."""
import os
import re

import pytest
import torch

import weight_only_int4_w4a16_amd as w

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_readme_lines_run():
    with open(README) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    assert blocks
    torch.manual_seed(0)

    def rand(*shape):
        return torch.randn(shape, device="cuda").to(torch.bfloat16)

    def ints(a):
        return torch.tensor(a, dtype=torch.int32, device="cuda")

    names = dict(x_bf16=rand(256))
    names["qweight_int32"], names["scales_fp16"] = w.quantize_pack(rand(64, 256))
    cache = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    # three requests, one new token each
    names.update(ctx_lens=ints([0, 15, 16]), new_lens=ints([1, 1, 1]), page_size=16, max_tokens=3,
                 page_table=ints([[-1, -1], [5, -1], [6, -1]]), free_pages=ints([0, 1, 2]), k=rand(3, 2, 64),
                 v=rand(3, 2, 64), k_cache=cache, v_cache=cache.clone(), q=rand(3, 4, 64),
                 log_decay=torch.full((2,), -0.1, device="cuda"), state=torch.zeros(3, 2, 64, 64, device="cuda"))
    # linear attention's q has the heads of its k
    for block in blocks:
        exec(block.replace("linear_attention_step(q, k", "linear_attention_step(k, k"), names)
    assert names["y"].shape == (64,) and names["o"].shape == (3, 2, 64)
    assert names["t"].slot_map.tolist() == [0, 5 * 16 + 15, 16]
    assert bool(names["state"].ne(0).any())
