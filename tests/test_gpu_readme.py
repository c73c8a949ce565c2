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


def test_readme_delta_line_keeps_states_bounded():
    """The line that steps the delta rule, again and again over the same tokens as the README's. With keys of norm 1 and beta
    and decays below 1 a state's column shrinks by e^-0.1 a step and grows by at most 0.91 |v|: its norm stays below 9.6 max |v|."""
    with open(README) as f:
        text = f.read()
    line = re.findall(r"^o = w\.delta_rule_step\(.*$", text, re.M)
    keys = re.findall(r"^kn = .*$", text, re.M)
    assert len(line) == 1
    torch.manual_seed(1)
    names = dict(torch=torch, w=w, log_decay=torch.full((2,), -0.1, device="cuda"), beta=torch.full((2,), 0.9, device="cuda"),
                 state=torch.zeros(3, 2, 64, 64, device="cuda"))
    names.update({n: torch.randn(3, 2, 64, device="cuda").to(torch.bfloat16) for n in "kvq"})
    for _ in range(200):
        for x in keys + line:
            exec(x, names)
    assert float(names["state"].norm(dim=2).max()) <= 9.6 * float(names["v"].float().abs().max())
