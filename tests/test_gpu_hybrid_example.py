"""The hybrid decoder example: prompts at once and token by token have to give the same logits."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def run(cuts, cache_type):
    """Logits of all tokens of three requests, given in pieces: cuts[i][b] tokens of request b each."""
    from hybrid_decode import HybridDecoder
    model = HybridDecoder(requests=3, longest=160, pages=64, seed=3, cache_type=cache_type)
    gen = torch.Generator().manual_seed(4)
    text = [torch.randint(0, 1000, (sum(c[b] for c in cuts),), generator=gen).cuda() for b in range(3)]
    at, rows = [0] * 3, [[] for _ in range(3)]
    for cut in cuts:
        logits = model.forward(torch.cat([text[b][at[b]:at[b] + cut[b]] for b in range(3)]), cut)
        for part, b in zip(logits.split(cut), range(3)):
            rows[b].append(part)
            at[b] += cut[b]
    return [torch.cat(r).float() for r in rows], model


@pytest.mark.parametrize("cache_type", [torch.bfloat16, torch.float8_e4m3fn])
def test_prompts_and_single_tokens_agree(cache_type):
    whole, _ = run([(70, 17, 33)], cache_type)
    parts, model = run([(60, 5, 32), (7, 10, 0), (1, 1, 0), (1, 1, 1), (1, 0, 0)], cache_type)
    assert model.lens.tolist() == [70, 17, 33]
    for a, b in zip(whole, parts):
        # bfloat16 activations: each of the two layers' sums is rounded about ten times on its way to
        # logits of unit size, half a step of 2^-8 each; routers may flip where two weights are equal
        off = (a - b).abs()
        assert float(off.mean()) <= 20 * 2.0 ** -9
        assert float((off.amax(1) > 0.5).float().mean()) <= 0.1


def test_generate_is_repeatable():
    from hybrid_decode import HybridDecoder
    prompts = [torch.arange(n, device="cuda") % 1000 for n in (3, 40, 16)]
    a = HybridDecoder(requests=3, seed=5).generate(prompts, 5)
    b = HybridDecoder(requests=3, seed=5).generate(prompts, 5)
    assert a.shape == (3, 5) and torch.equal(a, b)
