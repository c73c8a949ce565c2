"""Page tables, slot maps and paged cache writes on the GPU against the plain definitions."""
import numpy as np
import pytest
import torch

import mixer_oracle as mo
import weight_only_int4_w4a16_amd as w

pytestmark = pytest.mark.gpu


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def check_tables(ctx, new, table, free, page, max_tokens, stream=None):
    got_table = ints(table)
    r = w.page_tables(ints(ctx), ints(new), got_table, ints(free), page, max_tokens=max_tokens, stream=stream)
    torch.cuda.synchronize()
    seq, cu, slots, pos, counts, want = mo.page_tables(ctx, new, table, free, page, max_tokens)
    assert r.seq_lens.tolist() == seq and r.cu_new.tolist() == cu and r.counts.tolist() == counts
    assert r.positions.tolist() == pos and r.slot_map.tolist() == slots
    assert got_table.tolist() == want


def drawn_step(rng, B, most_ctx, most_new, page, spare):
    """Requests with their old pages in the table, and a free list of what they need plus `spare`."""
    ctx = rng.integers(0, most_ctx + 1, B)
    new = rng.integers(0, most_new + 1, B)
    ctx[rng.random(B) < 0.2] = 0
    new[rng.random(B) < 0.2] = 0
    old = -(-ctx // page)
    need = -(-(ctx + new) // page) - old
    width = int((old + need).max()) + 2
    perm = rng.permutation(int(old.sum() + need.sum()) + 20)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :old[b]] = perm[at:at + old[b]]
        at += old[b]
    free = perm[at:at + max(0, int(need.sum()) + spare)]
    return ctx.tolist(), new.tolist(), table.tolist(), free.tolist(), int(new.sum())


@pytest.mark.parametrize("B,most_ctx,most_new,page", [
    (1, 5, 1, 16), (1, 0, 1000, 1), (3, 40, 9, 16), (64, 500, 1, 16), (65, 300, 70, 48), (257, 100, 300, 7),
    (700, 50, 40, 64), (1500, 20, 3, 16), (9000, 9, 2, 4), (16384, 3, 2, 16),
])
def test_page_tables(B, most_ctx, most_new, page):
    rng = np.random.default_rng(B)
    ctx, new, table, free, total = drawn_step(rng, B, most_ctx, most_new, page, 5)
    check_tables(ctx, new, table, free, page, total + 3)


def test_page_tables_edges():
    rng = np.random.default_rng(1)
    ctx, new, table, free, total = drawn_step(rng, 40, 100, 50, 16, -9)      # the list is too short
    check_tables(ctx, new, table, free, 16, total)
    check_tables(ctx, new, table, [], 16, total)
    check_tables(ctx, new, table, free, 16, total // 2)                      # fewer tokens than there are
    check_tables(ctx, new, table, free, 16, 0)
    check_tables(ctx, new, [r[:3] for r in table], free, 16, total)          # rows too short for the lengths
    check_tables([0] * 5, [0] * 5, [[-1] * 2] * 5, [1, 2], 16, 4)            # nothing to do
    check_tables([-3, 10, -1], [4, -7, 2], [[-1] * 2, [5, 6], [-1] * 2], [1, 2], 8, 9)   # negative lengths
    check_tables([2, 2], [1, 1], [[2 ** 31 - 1], [2 ** 27]], [], 16, 2)      # pages whose slots pass 2^31
    # sums that saturate, in a table that holds a few pages of them
    check_tables([2 ** 31 - 1, 5], [2 ** 31 - 1, 2 ** 31 - 1], [[-1] * 3, [4, -1, -1]], [7, 8, 9, 10], 65536, 6)


def test_page_tables_strided_table_stream_and_graph():
    rng = np.random.default_rng(2)
    ctx, new, table, free, total = drawn_step(rng, 33, 90, 60, 16, 0)
    wide = torch.full((33, 64), -5, dtype=torch.int32, device="cuda")
    view = wide[:, 3:3 + len(table[0])]
    view.copy_(ints(table))
    c, n, f = ints(ctx), ints(new), ints(free)
    out = w.page_tables_buffers(33, total + 70)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w.page_tables(c, n, view, f, 16, out=out, stream=side)
    side.synchronize()
    want = mo.page_tables(ctx, new, table, free, 16, total + 70)
    assert out.slot_map.tolist() == want[2] and view.tolist() == want[5]
    assert (wide[:, :3] == -5).all() and (wide[:, 3 + view.shape[1]:] == -5).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.page_tables(c, n, view, f, 16, out=out)
    for rep in range(4):
        fewer = [max(0, x - rep) for x in new]
        n.copy_(ints(fewer))
        view.copy_(ints(table))
        g.replay()
        torch.cuda.synchronize()
        want = mo.page_tables(ctx, fewer, table, free, 16, total + 70)
        assert out.slot_map.tolist() == want[2] and out.positions.tolist() == want[3]
        assert out.cu_new.tolist() == want[1] and view.tolist() == want[5]


def new_cache(pages, page, heads, dim, dtype, layout):
    shape = (pages, heads, page, dim) if layout == "hnd" else (pages, page, heads, dim)
    x = torch.randn(shape, device="cuda").to(dtype)
    return x.permute(0, 2, 1, 3) if layout == "hnd" else x


def bits(t):
    """The bit patterns of a tensor, in its own shape, on the host."""
    return t.contiguous().view(torch.uint8).cpu()


def written(cache, x, slots, scale):
    """The cache after the plain write of x [T, heads, dim]."""
    c = cache.contiguous().cpu().clone()
    page = c.shape[1]
    raw = torch.uint8 if c.dtype == torch.float8_e4m3fn else torch.int16
    for t, s in enumerate(slots):
        if 0 <= s < c.shape[0] * page:
            row = x[t].cpu()
            if raw is torch.uint8:   # one float32 division, one rounding (torch's cast: nearest even)
                row = (row.float() / scale.cpu()[:, None]).clamp(-448, 448).to(c.dtype)
            c.view(raw)[s // page, s % page] = row.view(raw)
    return c


@pytest.mark.parametrize("T,heads,dim,page,dtype,fp8,layout", [
    (1, 1, 64, 1, torch.bfloat16, False, "nhd"), (7, 8, 128, 16, torch.bfloat16, False, "hnd"),
    (33, 3, 80, 5, torch.float16, False, "nhd"), (1025, 2, 256, 64, torch.bfloat16, True, "hnd"),
    (1, 4, 128, 16, torch.float16, True, "nhd"), (130, 5, 1024, 3, torch.float16, True, "hnd"),
    (300, 1, 16, 48, torch.bfloat16, True, "nhd"),
])
def test_kv_write(T, heads, dim, page, dtype, fp8, layout):
    torch.manual_seed(T)
    pages = -(-T // page) + 2
    kind = torch.float8_e4m3fn if fp8 else dtype
    kc, vc = (new_cache(pages, page, heads, dim, kind, layout) for _ in range(2))
    k = torch.randn(T, heads, dim, device="cuda").to(dtype) * 3
    v = torch.randn(T, heads, dim, device="cuda").to(dtype)
    k[0, 0, 0], v[0, 0, 1], v[0, 0, 2] = float("nan"), float("inf"), -float("inf")
    ks = torch.rand(heads, device="cuda") * 0.01 + 0.004 if fp8 else None   # some values saturate
    vs = torch.rand(heads, device="cuda") + 0.5 if fp8 else None
    slots = torch.randperm(pages * page)[:T].tolist()
    for i, bad in ((2, -1), (3, pages * page), (5, 2 ** 31 - 1), (6, -2 ** 31)):
        if i < T:
            slots[i] = bad
    want_k, want_v = written(kc, k, slots, ks), written(vc, v, slots, vs)
    w.paged_kv_write(k, v, kc, vc, ints(slots), k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    for got, want in ((kc, want_k), (vc, want_v)):
        if fp8:   # any NaN code will do
            a, b = got.contiguous().cpu().float(), want.float()
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(9e9), b.nan_to_num(9e9))
        else:
            assert torch.equal(bits(got), bits(want))


def test_kv_write_strides_and_offsets_past_32_bits():
    heads, dim, page = 2, 64, 16
    fused = torch.randn(9, 6 * heads, dim, device="cuda").to(torch.bfloat16)      # q, k and v of one product
    k, v = fused[:, 4 * heads::2][:, :heads], fused[:, 1:1 + heads]
    both = torch.zeros(5, 2, heads, page, dim, dtype=torch.bfloat16, device="cuda")   # K and V in one buffer
    kc, vc = both[:, 0].permute(0, 2, 1, 3), both[:, 1].permute(0, 2, 1, 3)
    slots = [3, 79, 40, 41, -1, 0, 16, 32, 64]
    want_k, want_v = written(kc, k, slots, None), written(vc, v, slots, None)
    w.paged_kv_write(k, v, kc, vc, ints(slots))
    assert torch.equal(bits(kc), bits(want_k)) and torch.equal(bits(vc), bits(want_v))
    big = torch.zeros(1 << 21, page, 1, 128, dtype=torch.float8_e4m3fn, device="cuda")   # 2^32 elements
    x = torch.randn(2, 1, 128, device="cuda").to(torch.float16)
    last = (1 << 25) - 1
    w.paged_kv_write(x, x, big, big, ints([last, 5]))
    flat = big.view(torch.uint8).reshape(-1, 128)
    want = x.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)[:, 0]
    assert torch.equal(flat[last], want[0]) and torch.equal(flat[5], want[1])
    assert int(flat[last - 1].sum()) == 0 and int(flat[(last * 128 % 2 ** 32) // 128 // 2].sum()) == 0


def test_kv_write_empty_and_refusals():
    c = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    w.paged_kv_write(x, x, c, c, ints([]))
    y = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="must be"):
        w.paged_kv_write(y, y, c, c, ints([1, 2]))
    with pytest.raises(ValueError, match="float8"):
        w.paged_kv_write(y, y, c, c, ints([1, 2, 3]), k_scale=torch.ones(2, device="cuda"))
    with pytest.raises(TypeError, match="k_cache"):
        w.paged_kv_write(y, y, c.half(), c.half(), ints([1, 2, 3]))
    with pytest.raises(w.W4A16Error, match="misaligned"):
        w.paged_kv_write(torch.zeros(3, 2, 68, dtype=torch.bfloat16, device="cuda")[..., :64],
                         y, c, c, ints([1, 2, 3]))
