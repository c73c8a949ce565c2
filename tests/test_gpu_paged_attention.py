"""Paged attention of one token on the GPU against the float64 definition, within counted roundings."""
import math

import pytest
import torch

import mixer_oracle as mo
import weight_only_int4_w4a16_amd as w

pytestmark = pytest.mark.gpu


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Paged:
    """A cache filled for requests of the given lengths; slots outside them hold NaN."""

    def __init__(self, lens, Hq, Hkv, D, page, dtype=torch.bfloat16, fp8=False, layout="hnd", seed=0, amp=1.0,
                 extra=2):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.dtype = lens, page, dtype
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        kind = torch.float8_e4m3fn if fp8 else dtype
        perm = torch.randperm(pages, generator=gen).tolist()
        self.table = [[perm.pop() for _ in range(n)] + [-1] * (max(need) + extra - n) for n in need]
        self.scales = [torch.rand(Hkv, generator=gen) + 0.5 for _ in range(2)] if fp8 else [None, None]
        self.rows, caches = [], []
        for s in self.scales:
            host = torch.full((pages, page, Hkv, D), math.nan).to(kind)
            raw = host.view(torch.uint8) if fp8 else host
            rows = []
            for b, n in enumerate(lens):
                x = (torch.randn(n, Hkv, D, generator=gen) * amp).to(kind)
                rows.append(x.double() * (s.double()[:, None] if fp8 else 1.0))
                at = torch.arange(n)
                where = torch.tensor(self.table[b], dtype=torch.long)[at // page]
                raw[where, at % page] = x.view(torch.uint8) if fp8 else x
            self.rows.append(rows)
            if layout == "hnd":
                caches.append(host.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3))
            else:
                caches.append(host.cuda())
        self.k, self.v = caches
        self.q = torch.randn(len(lens), Hq, D, generator=gen).to(dtype)

    def run(self, scale, window=0, lse=True, **kw):
        sums = torch.empty(self.q.shape[:2], device="cuda") if lse else None
        ks, vs = (None if s is None else s.cuda() for s in self.scales)
        out = w.paged_attention(kw.pop("q", self.q.cuda()), self.k, self.v, kw.pop("table", ints(self.table)),
                                kw.pop("lens", ints(self.lens)), scale=scale, window=window, k_scale=ks, v_scale=vs,
                                lse=sums, **kw)
        torch.cuda.synchronize()
        return out, sums

    def check(self, out, sums, scale, window=0):
        for b, n in enumerate(self.lens):
            lo = max(0, n - window) if window else 0
            o, l, mag, qk, top = mo.attention(self.q[b].double(), self.rows[0][b], self.rows[1][b], scale, lo)
            tol, tol_l = mo.attention_bounds(self.dtype, o, mag, qk, top, n, self.q.shape[2])
            err = (out[b].cpu().double() - o).abs()
            assert bool((err <= tol).all()), f"request {b} of length {n}: off by {float((err / tol).max()):.3g} bounds"
            if sums is not None:
                got = sums[b].cpu().double()
                assert torch.equal(got.isinf(), l.isinf())
                if n > lo:
                    assert float((got - l).abs().max()) <= tol_l, f"request {b}: lse"


LENS = [1, 0, 17, 64, 129, 5, 300, 33, 16]


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype,fp8,layout", [
    (8, 2, 128, 16, torch.bfloat16, False, "hnd"), (1, 1, 64, 16, torch.float16, False, "nhd"),
    (28, 4, 128, 64, torch.float16, True, "nhd"), (16, 1, 256, 32, torch.bfloat16, False, "nhd"),
    (12, 4, 96, 48, torch.bfloat16, False, "hnd"), (10, 2, 192, 1, torch.float16, False, "hnd"),
    (40, 1, 64, 7, torch.bfloat16, True, "hnd"), (6, 6, 128, 24, torch.bfloat16, True, "nhd"),
    (5, 1, 96, 8, torch.float16, True, "nhd"), (34, 2, 192, 16, torch.bfloat16, True, "hnd"),
    (16, 2, 256, 100, torch.float16, True, "hnd"), (33, 1, 128, 128, torch.float16, False, "hnd"),
])
def test_heads_dims_types_and_pages(Hq, Hkv, D, page, dtype, fp8, layout):
    p = Paged(LENS, Hq, Hkv, D, page, dtype, fp8, layout, seed=D + page)
    out, sums = p.run(D ** -0.5)
    p.check(out, sums, D ** -0.5)
    again, sums2 = p.run(D ** -0.5)
    assert torch.equal(out, again) and torch.equal(sums, sums2)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 1000, 2049, 9000])
def test_single_request_lengths(n):
    p = Paged([n], 8, 2, 128, 16, seed=n)
    out, sums = p.run(0.09)
    p.check(out, sums, 0.09)


@pytest.mark.parametrize("window", [1, 15, 16, 100, 5000])
def test_window(window):
    p = Paged([0, 1, 40, 700, 16, 2100], 8, 4, 64, 16, torch.float16, seed=window)
    out, sums = p.run(0.125, window=window)
    p.check(out, sums, 0.125, window)


@pytest.mark.parametrize("B,longest", [(40, 900), (300, 60), (1000, 3), (3, 20000)])
def test_ragged_batches(B, longest):
    gen = torch.Generator().manual_seed(B)
    lens = torch.randint(0, longest + 1, (B,), generator=gen).tolist()
    lens[0] = longest
    p = Paged(lens, 4, 2, 64, 16, seed=B)
    out, sums = p.run(0.125)
    p.check(out, sums, 0.125)


def test_large_scores_and_large_values():
    """Scores of several hundred, one position taking all the weight, and cold starts at -hundreds."""
    for scale in (3.0, -3.0):
        p = Paged([600, 70], 8, 2, 128, 16, torch.float16, seed=4, amp=3.0)
        out, sums = p.run(scale)
        p.check(out, sums, scale)
    p = Paged([200], 4, 1, 64, 16, torch.bfloat16, seed=5, amp=1e4)   # values far past float16's range
    p.q = p.q * 1e-5
    out, sums = p.run(0.125)
    p.check(out, sums, 0.125)


def test_infinite_scores_are_not_turned_into_nan():
    """A score of -inf takes no weight, and a request whose scores are all -inf has an empty row."""
    p = Paged([50, 20], 2, 1, 64, 16, torch.float16, seed=6)
    p.q[:] = 60000.0
    where = torch.tensor(p.table[0])[torch.arange(50) // 16]
    keep = torch.ones(50, dtype=torch.bool)
    keep[::3] = False
    bad = torch.where(keep)[0]
    p.k[where[bad].cuda(), (bad % 16).cuda()] = -math.inf
    p.rows[0][0][keep] = -math.inf
    p.rows[0][0][~keep] = 0.0
    good = torch.where(~keep)[0]
    p.k[where[good].cuda(), (good % 16).cuda()] = 0.0
    page1 = torch.tensor(p.table[1])[torch.arange(20) // 16].cuda()
    p.k[page1, (torch.arange(20) % 16).cuda()] = -math.inf
    out, sums = p.run(0.125)
    want = p.rows[1][0][~keep].mean(0)
    tol = mo.half_step(torch.float16) * 4 * p.rows[1][0].abs().max()
    assert float((out[0].cpu().double() - want).abs().max()) <= tol
    assert torch.allclose(sums[0].cpu(), torch.full((2,), math.log(17.0)), atol=1e-5)
    assert torch.equal(out[1], torch.zeros_like(out[1])) and bool((sums[1] == -math.inf).all())


def test_bad_pages_contribute_nothing():
    """Entries that are no page of the cache, and lengths past the table, are left out."""
    p = Paged([64, 40, 33], 4, 2, 64, 16, seed=7, extra=0)
    table = [list(r) for r in p.table]
    table[0][1] = -1
    table[1][0] = p.k.shape[0]
    table[2] = [2 ** 31 - 1, -2 ** 31, 10 ** 6] + table[2][3:]
    keep = [[*range(16), *range(32, 64)], list(range(16, 40)), []]
    lens = [2 ** 31 - 1 if i == 0 else n for i, n in enumerate(p.lens)]   # past the row's four pages
    out, sums = p.run(0.125, table=ints(table), lens=ints(lens))
    p.rows = [[r[b][keep[b]] for b in range(3)] for r in p.rows]
    p.lens = [len(x) for x in keep]
    p.check(out, sums, 0.125)


def test_strides_streams_and_preallocated_outputs():
    p = Paged([100, 7, 260], 6, 2, 128, 16, seed=8)
    wide = torch.zeros(3, 2 * 6 + 4, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, ::2][:, :6] = p.q.cuda()
    q = wide[:, ::2][:, :6]
    big = torch.full((3, 50), 7, dtype=torch.int32, device="cuda")
    table = big[:, 5:5 + len(p.table[0])]
    table.copy_(ints(p.table))
    room = torch.full((3, 9, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    out = room[:, 1:7, 128:]
    work = w.paged_attention_workspace(q, p.k)
    work.fill_(255)                                            # NaN patterns: contents do not matter
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, sums = p.run(0.09, q=q, table=table, out=out, workspace=work, stream=side)
    assert got.data_ptr() == out.data_ptr()
    p.check(got, sums, 0.09)
    assert bool((room[:, 0] == 5).all() and (room[:, 7:] == 5).all() and (room[:, :, :128] == 5).all())
    alone, _ = p.run(0.09)
    assert torch.equal(alone, got)


def test_graph_replays_match_eager_calls():
    p = Paged([1000, 3, 170, 0, 64], 8, 2, 128, 16, seed=9)
    q, lens, table = p.q.cuda(), ints(p.lens), ints(p.table)
    out, work = torch.empty_like(q), w.paged_attention_workspace(q, p.k)
    sums = torch.empty(q.shape[:2], device="cuda")

    def call():
        w.paged_attention(q, p.k, p.v, table, lens, scale=0.09, out=out, lse=sums, workspace=work)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(4):
        now = [max(0, n - 61 * rep) for n in p.lens]
        lens.copy_(ints(now))
        q.copy_(torch.randn(q.shape).to(q.dtype))
        g.replay()
        torch.cuda.synchronize()
        a, b = out.clone(), sums.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(b, sums)


def test_offsets_past_32_bits():
    """Pages whose first element lies past 2^32, in a cache of 2^21 pages."""
    page, D = 16, 128
    k = torch.zeros(1 << 21, page, 1, D, dtype=torch.float8_e4m3fn, device="cuda")
    last = [(1 << 21) - 1, (1 << 21) - 2, 1 << 20]
    x = torch.randn(40, D).to(torch.float8_e4m3fn)
    for i in range(40):
        k.view(torch.uint8)[last[i // page], i % page, 0] = x[i].cuda().view(torch.uint8)
    q = torch.randn(1, 4, D).to(torch.bfloat16)
    out = w.paged_attention(q.cuda(), k, k, ints([last]), ints([40]), scale=0.09)
    rows = x.double()[:, None]
    o, _, mag, qk, top = mo.attention(q[0].double(), rows, rows, 0.09)
    tol, _ = mo.attention_bounds(torch.bfloat16, o, mag, qk, top, 40, D)
    assert bool(((out[0].cpu().double() - o).abs() <= tol).all())


def test_empty_batch_and_refusals():
    p = Paged([5], 4, 2, 64, 16)
    none = w.paged_attention(p.q[:0].cuda(), p.k, p.v, ints(p.table)[:0], ints([]))
    assert none.shape == (0, 4, 64)
    with pytest.raises(ValueError, match="shape mismatch"):
        w.paged_attention(p.q.cuda(), p.k, p.v, ints(p.table), ints([5, 5]))
    with pytest.raises(ValueError, match="differ in shape"):
        w.paged_attention(p.q.cuda(), p.k, p.v[1:], ints(p.table), ints([5]))
    with pytest.raises(w.W4A16Error, match="shape"):
        w.paged_attention(p.q[:, :3].cuda(), p.k, p.v, ints(p.table), ints([5]))
    with pytest.raises(w.W4A16Error, match="workspace"):
        w.paged_attention(p.q.cuda(), p.k, p.v, ints(p.table), ints([5]),
                          workspace=torch.empty(0, dtype=torch.uint8, device="cuda").new_empty(8))


def test_short_way_refuses_like_the_long_one():
    """With outputs and scratch given, calls go through the C++ binding: same results, same refusals."""
    p = Paged([90, 3], 4, 2, 64, 16, torch.float16, True, "nhd", seed=11)
    q, table, lens = p.q.cuda(), ints(p.table), ints(p.lens)
    out, work = torch.empty_like(q), w.paged_attention_workspace(q, p.k)
    ks, vs = (s.cuda() for s in p.scales)

    def call(**kw):
        a = dict(q=q, k_cache=p.k, v_cache=p.v, page_table=table, seq_lens=lens, scale=0.125, k_scale=ks, v_scale=vs,
                 out=out, workspace=work)
        a.update(kw)
        return w.paged_attention(**a)

    p.check(call(), None, 0.125)
    long, _ = p.run(0.125, lse=False)
    assert torch.equal(long, out)
    assert torch.equal(call(scale=None), call(scale=64 ** -0.5))
    for kw, kind, text in (
            (dict(seq_lens=lens.long()), TypeError, "seq_lens"), (dict(seq_lens=lens[:1]), ValueError, "mismatch"),
            (dict(q=q.float()), TypeError, "q must"), (dict(out=out[:1]), ValueError, "out must"),
            (dict(k_scale=ks[:1]), ValueError, "one value"), (dict(v_cache=p.v[..., :32]), ValueError, "differ"),
            (dict(workspace=work[:100]), w.W4A16Error, "workspace"), (dict(window=-1), w.W4A16Error, "shape"),
            (dict(page_table=table.cpu()), ValueError, "GPU"), (dict(out=out.transpose(1, 2).contiguous().transpose(1, 2)),
                                                                ValueError, "unit stride")):
        with pytest.raises(kind, match=text):
            call(**kw)
