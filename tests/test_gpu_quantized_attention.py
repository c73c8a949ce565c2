"""Attention over the 8-bit cache with a scale for each block and head, against float64."""
import math

import pytest
import torch

import mixer_oracle as mo
import quantized_oracle as qo
import weight_only_int4_w4a16_amd as w

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
I8, E4 = torch.int8, torch.float8_e4m3fn


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Attend:
    def __init__(self, lens, Hq, heads, dim, page=16, block=16, kind=I8, dtype=BF, layout="hnd", seed=0, amp=1.0, spread=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.dtype, self.kind = lens, page, dtype, kind
        each = [-(-max(n, 0) // page) for n in lens]
        pages = sum(each) + 3
        perm = torch.randperm(pages, generator=gen).tolist()
        self.table = torch.full((len(lens), max(each + [1]) + 1), -1, dtype=torch.int32)
        for b, n in enumerate(each):
            self.table[b, :n] = torch.tensor(perm[:n], dtype=torch.int32)
            perm = perm[n:]
        shape = (pages, page, heads, dim)
        if kind == I8:
            self.codes = [torch.randint(-127, 128, shape, generator=gen, dtype=I8) for _ in range(2)]
        else:
            self.codes = [(torch.randn(shape, generator=gen) * 120).clamp(-448, 448).to(E4) for _ in range(2)]
        self.scale = [(1 + 2 * torch.rand(pages, page // block, heads, generator=gen)) / qo.LARGEST[kind]
                      * 2.0 ** (spread * torch.randn(pages, page // block, heads, generator=gen)) for _ in range(2)]
        self.q = (torch.randn(len(lens), Hq, dim, generator=gen) * amp).to(dtype)
        self.layout = layout

    def device(self):
        if self.layout == "hnd":
            return [c.transpose(1, 2).contiguous().cuda().transpose(1, 2) for c in self.codes]
        return [c.cuda() for c in self.codes]

    def run(self, **kw):
        lse = torch.full(self.q.shape[:2], 9.0, device="cuda")
        out = w.quantized_attention(kw.pop("q", self.q.cuda()), *self.device(), *[s.cuda() for s in self.scale],
                                    self.table.cuda(), ints(self.lens), lse=lse, **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, scale=None, window=0, skip=()):
        B, Hq, D = self.q.shape
        scale = D ** -0.5 if scale is None else scale
        full = [qo.values(c).nan_to_num(0.0) * qo.spread(s, self.page) for c, s in zip(self.codes, self.scale)]
        vs = qo.spread(self.scale[1], self.page)
        for b, n in enumerate(self.lens):
            if b in skip:
                continue
            n = max(n, 0)
            lo = max(0, n - window) if window else 0
            pos = torch.arange(lo, n)
            at = self.table[b, pos // self.page].long()
            pos, at = pos[at >= 0], at[at >= 0]
            k, v = (x[at, pos % self.page] for x in full)
            o, l, mag, qk, top = mo.attention(self.q[b].double(), k, v, scale)
            weight = 0.0
            share = Hq // k.shape[1]
            for h in range(Hq if len(pos) else 0):
                p = torch.softmax((k[:, h // share] @ self.q[b, h].double()) * scale, 0)
                weight = max(weight, float((p * vs[at, pos % self.page, h // share, 0]).max()))
            tol, tol_l = qo.attention_bounds(self.dtype, o, mag, qk, top, max(1, len(pos)), D, weight, qo.LARGEST[self.kind])
            err = (out[b].cpu().double() - o).abs()
            assert bool((err <= tol).all()), f"request {b} of {n}: off by {float((err / tol).max()):.3g} bounds"
            got = lse[b].cpu().double()
            assert torch.equal(torch.isinf(got), torch.isinf(l))
            fine = ~torch.isinf(l)
            assert bool(((got - l).abs()[fine] <= tol_l + 2.0 ** -23 * l.abs()[fine]).all()), f"request {b}: lse"


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 257, 1000, 4100])
@pytest.mark.parametrize("kind", [I8, E4])
def test_lengths(n, kind):
    x = Attend([n], 4, 2, 64, kind=kind, seed=n)
    x.check(*x.run())


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind,dtype,layout,page,block,Hq,heads", [
    (I8, BF, "hnd", 16, 16, 8, 2), (I8, FP, "nhd", 64, 32, 7, 7), (E4, BF, "nhd", 48, 48, 20, 1), (E4, FP, "hnd", 128, 64, 10, 2),
    (I8, BF, "nhd", 96, 16, 34, 2),
])
def test_dims_types_and_heads(dim, kind, dtype, layout, page, block, Hq, heads):
    x = Attend([300, 0, 1, 77, -3, 513], Hq, heads, dim, page, block, kind, dtype, layout, seed=dim)
    out, lse = x.run()
    x.check(out, lse)
    again, lse2 = x.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window", [1, 15, 100, 128, 129, 100000])
def test_windows(window):
    x = Attend([700, 90, 128, 5, 0], 4, 2, 64, 32, 16, seed=window)
    x.check(*x.run(window=window), window=window)


def test_many_requests_and_few_long_ones():
    x = Attend([(37 * i) % 200 for i in range(150)], 4, 1, 64, seed=1)
    x.check(*x.run())
    x = Attend([20000, 3, 9000], 8, 2, 128, 64, 64, E4, FP, "nhd", seed=2)
    x.check(*x.run())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kind", [I8, E4])
def test_scales_and_scores_of_all_sizes(dtype, kind):
    """Blocks whose values are many orders apart, weights that hang on one position, large and small queries."""
    x = Attend([500, 260], 4, 2, 64, 16, 16, kind, dtype, seed=3, spread=6.0, amp=0.01)
    for s in x.scale[0:1]:
        s.clamp_(max=0.2)
    x.check(*x.run())
    x = Attend([300], 4, 2, 64, 16, 16, kind, dtype, seed=4, amp=6.0)
    x.check(*x.run())
    x = Attend([300], 2, 2, 64, 16, 16, kind, dtype, seed=5)
    x.q = (x.q.float() * (60000.0 if dtype == FP else 1e30) / x.q.float().abs().max()).to(dtype)
    tiny = 2e-5 if dtype == FP else 1e-30
    x.check(*x.run(scale=tiny), scale=tiny)
    x.q = (x.q.float() * 1e-9).to(dtype) if dtype == FP else (x.q.float() * 1e-60).to(dtype)
    x.check(*x.run(scale=1.0), scale=1.0)


def test_a_small_block_behind_a_large_one():
    """The largest weight has values of little size, another block larger ones by 2^30 and a weight of 2^-30: both count."""
    x = Attend([32], 1, 1, 64, 16, 16, I8, FP, seed=6)
    x.q[:] = 1.0
    x.codes[0][:] = 0
    p = x.table[0, :2].long()
    x.codes[0][p[0], :, :, 0] = 100
    x.scale[0][:] = 1.0
    x.scale[1][p[0]], x.scale[1][p[1]] = 2.0 ** -10, 2.0 ** -10 * 2.0 ** 20
    scale = 20 * math.log(2) / 100
    x.check(*x.run(scale=scale), scale=scale)


def test_what_is_not_read_may_be_anything():
    """NaN scales and codes behind the end, before the window, and on pages that belong to nobody."""
    x = Attend([200, 40], 4, 2, 64, 32, 16, E4, BF, seed=7)
    out, lse = x.run(window=50)
    x.check(out, lse, window=50)
    used = torch.zeros_like(x.scale[0][..., 0], dtype=torch.bool)
    held = torch.zeros(x.codes[0].shape[:2], dtype=torch.bool)
    for b, n in enumerate(x.lens):
        for j in range(max(0, n - 50), n):
            used[x.table[b, j // 32], j % 32 // 16] = True
            held[x.table[b, j // 32], j % 32] = True
    for c, s in zip(x.codes, x.scale):
        s[~used] = math.nan
        c.view(torch.uint8)[~held] = 0x7F
    out2, lse2 = x.run(window=50)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_a_block_that_is_not_a_number():
    """Requests and heads that read a position of it get NaN, others what they had."""
    x = Attend([100, 60], 4, 2, 64, 16, 16, I8, BF, seed=8)
    out, lse = x.run()
    x.scale[1][x.table[0, 2], 0, 1] = math.nan                  # values: head 1 of the first request
    out2, lse2 = x.run()
    assert bool(out2[0, 2:].isnan().all()) and torch.equal(out2[0, :2], out[0, :2]) and torch.equal(out2[1], out[1])
    assert torch.equal(lse, lse2)
    x.scale[0][x.table[1, 3], 0, 0] = math.nan                  # keys: head 0 of the second
    out2, lse2 = x.run()
    assert bool(out2[1, :2].isnan().all()) and bool(lse2[1, :2].isnan().all()) and torch.equal(out2[1, 2:], out[1, 2:])


def test_pages_that_are_none():
    x = Attend([100, 50, 33], 4, 2, 64, 16, 16, I8, FP, "nhd", seed=9)
    x.table[0, 2], x.table[0, 6], x.table[1, 0] = -1, -1, -1
    x.table[2, :3] = -1
    out, lse = x.run()
    x.check(out, lse)
    assert not bool(out[2].any()) and bool(torch.isinf(lse[2]).all())
    x.table[0, 2] = 10 ** 6
    out2, lse2 = x.run()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_lengths_past_the_table():
    x = Attend([64, 20], 2, 1, 64, 16, 16, seed=10)
    x.table = x.table[:, :4].contiguous()
    out, lse = x.run()
    x.lens = [2 ** 31 - 1, 20]
    out2, lse2 = x.run()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_strides_ways_in_and_streams():
    x = Attend([90, 170], 4, 2, 64, 32, 32, I8, BF, "nhd", seed=11)
    want, lse = x.run()
    wide = torch.zeros(2, 9, 64, dtype=BF, device="cuda")
    wide[:, 2:6].copy_(x.q)
    got = torch.full((2, 4, 2, 64), 3.0, dtype=BF, device="cuda")
    x.run(q=wide[:, 2:6], out=got[:, :, 1])
    assert torch.equal(got[:, :, 1], want) and bool((got[:, :, 0] == 3).all())
    dev = x.device()
    scales = [torch.empty(2, 1, dev[0].shape[0], device="cuda").permute(2, 1, 0).copy_(s) for s in x.scale]
    table = torch.full((2, 40), -1, dtype=torch.int32, device="cuda")
    table[:, :x.table.shape[1]] = x.table.cuda()
    work = w.quantized_attention_workspace(x.q, dev[0])
    work = work.cuda() if not work.is_cuda else work
    out = torch.empty_like(want)
    o = w.quantized_attention(x.q.cuda(), *dev, *scales, table[:, :x.table.shape[1]], ints(x.lens), out=out, workspace=work)
    assert o is out and torch.equal(out, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o = w.quantized_attention(x.q.cuda(), *dev, *scales, table[:, :x.table.shape[1]], ints(x.lens), stream=side)
    side.synchronize()
    assert torch.equal(o, want)
    none = w.quantized_attention(x.q[:0].cuda(), *dev, *scales, table[:0], ints([]))
    assert none.shape == (0, 4, 64)
    with pytest.raises(ValueError, match="differ in shape"):
        w.quantized_attention(x.q.cuda(), dev[0], dev[1][:1], *scales, table, ints(x.lens))
    with pytest.raises(w.W4A16Error):
        w.quantized_attention(x.q.cuda(), *dev, *scales, table, ints(x.lens), workspace=work[:16])


def test_offsets_past_32_bits():
    """Pages whose first element lies past 2^32, in a cache of 2^21 pages."""
    page, D = 16, 128
    k = torch.zeros(1 << 21, page, 1, D, dtype=I8, device="cuda")
    scale = torch.zeros(1 << 21, 1, 1, device="cuda")
    last = [(1 << 21) - 1, (1 << 21) - 2, 1 << 20]
    gen = torch.Generator().manual_seed(1)
    x, s = torch.randint(-127, 128, (48, D), generator=gen, dtype=I8), torch.rand(3, generator=gen) * 0.02 + 0.01
    for i, p in enumerate(last):
        k[p, :, 0] = x[16 * i:16 * i + 16].cuda()
        scale[p] = float(s[i])
    q = torch.randn(1, 4, D, generator=gen).to(BF)
    out = w.quantized_attention(q.cuda(), k, k, scale, scale, ints([last]), ints([40]), scale=0.09)
    rows = (x.double() * s.double().repeat_interleave(16)[:, None])[:40, None]
    o, _, mag, qk, top = mo.attention(q[0].double(), rows, rows, 0.09)
    tol, _ = qo.attention_bounds(BF, o, mag, qk, top, 40, D, float(s.max()), 127.0)
    assert bool(((out[0].cpu().double() - o).abs() <= tol).all())


def test_graph_with_lengths_that_grow():
    """One captured call, replayed while requests grow, begin and end."""
    x = Attend([300, 5, 0, 64], 4, 2, 64, 32, 32, seed=12)
    dev, scales, table = x.device(), [s.cuda() for s in x.scale], x.table.cuda()
    q, lens = x.q.cuda(), ints([1, 5, 0, 0])
    out, work = torch.empty_like(q), w.quantized_attention_workspace(q, dev[0])

    def call(**kw):
        return w.quantized_attention(q, *dev, *scales, table, lens, **kw)

    call(out=out, workspace=work)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out=out, workspace=work)
    for now in ([1, 5, 0, 0], [300, 0, 0, 64], [129, 5, 0, 1], [0, 0, 0, 0], [300, 5, 0, 64]):
        lens.copy_(ints(now))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call())
