"""Page tables whose operands share memory are refused before anything is enqueued."""
import pytest
import torch

import weight_only_int4_w4a16_amd as w

pytestmark = pytest.mark.gpu


def operands():
    room = torch.zeros(4000, dtype=torch.int32, device="cuda")
    at = lambda i, n: room[i:i + n]   # noqa: E731
    ctx, new, free = at(0, 40), at(40, 40), at(80, 200)
    table = at(1000, 1200).view(40, 30)[:, :12]
    out = w.PageTables(at(300, 40), at(340, 41), at(381, 100), at(481, 100), at(581, 2))
    new.fill_(2)
    free.copy_(torch.arange(200))
    table.fill_(-1)
    return room, ctx, new, table, free, out


def test_neighbours_are_fine():
    room, ctx, new, table, free, out = operands()
    in_gap = room[1012:1030]   # between two rows of the table
    in_gap.fill_(7)
    for short in (True, False):   # with max_tokens the call goes the long way
        r = w.page_tables(ctx, new, table, free, 16, out=out, **({} if short else dict(max_tokens=100)))
        assert r.seq_lens.tolist() == [2] * 40 and r.counts.tolist() == [80, 40]
    w.page_tables(ctx, new, table, in_gap, 16, out=out)
    w.page_tables(new, new, table, free, 16, out=out)   # only read


@pytest.mark.parametrize("change", [
    dict(seq_lens="ctx"), dict(seq_lens="new"), dict(cu_new=(20, 41)), dict(counts=(0, 2)), dict(slot_map=(150, 100)),
    dict(positions=(279, 100)), dict(seq_lens=(1000, 40)), dict(seq_lens=(2150, 40)), dict(positions=(381, 100)),
    dict(slot_map=(901, 100)), dict(free=(1000, 200)),
])
def test_shared_operands_are_refused(change):
    room, ctx, new, table, free, out = operands()
    for name, where in change.items():
        t = {"ctx": ctx, "new": new}[where] if isinstance(where, str) else room[where[0]:where[0] + where[1]]
        if name == "free":
            free = t
        else:
            out = out._replace(**{name: t})
    before = room.clone()
    for kw in ({}, dict(max_tokens=100)):
        with pytest.raises(w.W4A16Error, match="share memory"):
            w.page_tables(ctx, new, table, free, 16, out=out, **kw)
    assert torch.equal(room, before)
