"""Writes of so many rows that a wave takes several runs (from 8192 of tokens times heads on, 16 tokens to a wave from 65536
on), and reads of rows of more than 256 pieces of 8 values, bit for bit as the definition has them."""
import pytest
import torch

from test_gpu_quantized_kv import BF, FP, KINDS, Cache, rows

pytestmark = pytest.mark.gpu


def runs(T, pages, page, block, gen):
    """T slots: runs of 1 to a few blocks, each from a block that no other has touched, from its first slot on or from
    its middle, with slots of no page between them here and there."""
    def upto(n):
        return int(torch.randint(n, (1,), generator=gen))

    slots, at, end = [], 0, pages * page
    while len(slots) < T:
        kind = upto(8)
        if kind == 0:
            slots += [(-1, end, 2 ** 31 - 1, -2 ** 31)[upto(4)]] * (1 + upto(3))
            continue
        first = at * block + (0 if kind < 4 else upto(block))
        n = 1 + upto(3) if kind < 6 else 1 + upto(3 * block)
        n = min(n, T - len(slots), end - first)
        slots += range(first, first + n)
        at = (first + n - 1) // block + 1
    return slots[:T]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,heads,dim,page,block,dtype,layout", [
    (3000, 8, 64, 48, 16, BF, "nhd"),      # 5 tokens to a wave
    (2100, 33, 64, 64, 64, FP, "kv"),      # 16
    (9001, 8, 64, 32, 16, BF, "hnd"),      # 16
    (4100, 17, 128, 48, 48, BF, "nhd"),    # 16
])
def test_runs_inside_and_across_a_waves_tokens(kind, T, heads, dim, page, block, dtype, layout):
    gen = torch.Generator().manual_seed(T)
    pages = 8 * T // page
    slots = runs(T, pages, page, block, gen)
    inside = [s for s in slots if 0 <= s < pages * page]
    assert len(set(inside)) == len(inside)
    c = Cache(pages, page, heads, dim, block, kind, layout, seed=heads)
    k, v = rows(T, heads, dim, dtype, seed=T, amp=1.5)
    size = 2.0 ** torch.randint(-3, 3, (T, 1, 1), generator=gen).float()      # some scales grow, others do not
    c.write((k.float() * size).to(dtype), (v.float() / size).to(dtype), slots)
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_one_long_prompt(kind):
    """3000 tokens of 8 heads of 256 that begin in a block's middle, then again from another place in it."""
    c = Cache(25, 128, 8, 256, 64, kind, "nhd", seed=1)
    k, v = rows(3000, 8, 256, BF, seed=2)
    c.write(k, v, list(range(37, 3037)))
    c.check()
    c.write(v * 2, k * 2, list(range(64 + 5, 3069)))
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,dim", [(17, 256), (33, 128), (64, 64), (65, 64)])
def test_rows_of_more_than_256_pieces(kind, heads, dim):
    c = Cache(5, 32, heads, dim, 32, kind, "hnd", seed=heads)
    order = torch.randperm(c.slots, generator=torch.Generator().manual_seed(3)).tolist()
    c.read(order + [-1, c.slots, order[0]], BF)
    c.read(order[:7], FP)
