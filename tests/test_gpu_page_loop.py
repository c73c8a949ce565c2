"""Steps that follow one another without the host: lengths and the free list move on by device operations."""
import os
import sys

import pytest
import torch

import mixer_oracle as mo
import weight_only_int4_w4a16_amd as w

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def test_a_captured_step_takes_other_pages_each_time():
    B, page, pages = 5, 4, 40
    ctx, new = ints([3, 0, 8, 5, 1]), ints([2, 1, 5, 0, 3])
    table = [[30 + 2 * b, 31 + 2 * b] + [-1] * 10 for b in range(B)]
    view, free, rank = ints(table), ints(list(range(pages - 12))), torch.arange(pages - 12, device="cuda")
    n = free.numel()
    out = w.page_tables_buffers(B, 14)

    def step():
        w.page_tables(ctx, new, view, free, page, out=out)
        ctx.copy_(out.seq_lens)
        at = rank + out.counts[1]
        free.copy_(torch.where(at < n, free[at.clamp(max=n - 1)], -1))

    state = [t.clone() for t in (ctx, view, free)]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((ctx, view, free), state):
        t.copy_(s)
    lens, left = ctx.tolist(), free.tolist()
    for _ in range(13):   # past the end of the list
        graph.replay()
        torch.cuda.synchronize()
        seq, cu, slots, pos, counts, table = mo.page_tables(lens, new.tolist(), table, left, page, 14)
        lens, left = seq, left[counts[1]:]
        assert out.slot_map.tolist() == slots and out.positions.tolist() == pos and view.tolist() == table
        assert ctx.tolist() == lens and free.tolist() == left + [-1] * (n - len(left))
        (ctx + 1).sum().item()   # other work and synchronizations between replays


def test_the_example_does_not_wait_for_the_host():
    from hybrid_decode import HybridDecoder
    model = HybridDecoder(requests=3, longest=160, pages=32, seed=3)
    taken = model.free.tolist()
    new = ints([20, 3, 1])
    model.place(new, 24)
    torch.cuda.synchronize()
    mode = torch.cuda.get_sync_debug_mode()
    torch.cuda.set_sync_debug_mode("error")
    try:
        model.place(new, 24)
    finally:
        torch.cuda.set_sync_debug_mode(mode)
    assert model.lens.tolist() == [40, 6, 2]
    assert model.table[:, :3].tolist() == [[taken[0], taken[1], taken[4]], [taken[2], -1, -1], [taken[3], -1, -1]]
    assert model.free.tolist() == taken[5:] + [-1] * 5
