"""Writes into and reads from the 8-bit cache with a scale for each block and head: codes, scales and values bit for
bit as the definition has them."""
import math

import pytest
import torch

import quantized_oracle as qo
import weight_only_int4_w4a16_amd as w

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
KINDS = [torch.int8, torch.float8_e4m3fn]


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def some_codes(shape, kind, gen):
    if kind == torch.int8:
        return torch.randint(-127, 128, shape, generator=gen, dtype=torch.int8)
    return (torch.randn(shape, generator=gen) * 100).clamp(-448, 448).to(kind)


class Cache:
    """Codes and scales on both sides; `layout` of the device's."""

    def __init__(self, pages, page, heads, dim, block, kind, layout="nhd", seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.codes = [some_codes((pages, page, heads, dim), kind, gen) for _ in range(2)]
        self.scale = [torch.rand(pages, page // block, heads, generator=gen) * 0.02 + 0.005 for _ in range(2)]
        if layout == "hnd":
            self.dev = [c.transpose(1, 2).contiguous().cuda().transpose(1, 2) for c in self.codes]
        elif layout == "kv":      # both in one buffer
            both = torch.stack(self.codes, 2).cuda()
            self.dev = [both[:, :, 0], both[:, :, 1]]
        else:
            self.dev = [c.cuda() for c in self.codes]
        self.dev_scale = [s.cuda() for s in self.scale]
        self.slots = pages * page

    def write(self, k, v, slots, **kw):
        w.quantized_kv_write(k.cuda(), v.cuda(), *self.dev, *self.dev_scale, ints(slots), **kw)
        for x, c, s in zip((k, v), self.codes, self.scale):
            qo.write(x, c, s, slots)

    def check(self):
        torch.cuda.synchronize()
        for name, c, s, dc, ds in zip("kv", self.codes, self.scale, self.dev, self.dev_scale):
            got = ds.cpu()
            assert torch.equal(got.view(torch.int32)[~got.isnan()], s.view(torch.int32)[~s.isnan()]), f"scales of {name}"
            assert torch.equal(got.isnan(), s.isnan())
            a, b = dc.cpu().contiguous().view(torch.uint8), c.view(torch.uint8)
            if c.dtype == torch.float8_e4m3fn:   # the sign of a zero is free
                a, b = torch.where(a == 128, 0, a), torch.where(b == 128, 0, b)
            bad = torch.nonzero(a != b)
            assert not len(bad), f"codes of {name}: {len(bad)} differ, first at {bad[0].tolist()}"

    def read(self, slots, dtype, **kw):
        got = w.quantized_kv_read(*self.dev, *self.dev_scale, ints(slots), dtype=dtype, **kw)
        torch.cuda.synchronize()
        for x, c, s in zip(got, self.codes, self.scale):
            want = qo.read(c, s, slots, x.dtype)
            x = x.cpu().double()
            assert torch.equal(x.nan_to_num(7.0), want.nan_to_num(7.0)) and torch.equal(x.isnan(), want.isnan())
        return got


def rows(T, heads, dim, dtype, seed=0, amp=1.0):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(T, heads, dim, generator=gen) * amp).to(dtype) for _ in range(2)]


SHAPES = [(16, 16, 1, 64), (64, 32, 3, 128), (48, 48, 2, 96), (128, 64, 2, 256), (32, 16, 4, 192)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("page,block,heads,dim", SHAPES)
@pytest.mark.parametrize("layout", ["nhd", "hnd", "kv"])
def test_prompts_and_single_tokens(kind, dtype, page, block, heads, dim, layout):
    """Whole blocks, blocks begun and ended, single tokens into held ones, skipped tokens: one call."""
    c = Cache(9, page, heads, dim, block, kind, layout, seed=page + dim)
    slots = list(range(2 * page, 3 * page)) + list(range(5 * page, 5 * page + page // 2 + 3))   # a prompt over two pages
    slots += [-1, -1, c.slots, 7 * page + 1, 2 ** 31 - 1, 8 * page + block - 1]                 # single tokens, and none
    slots += list(range(3, min(block, 11)))                                                    # a few into a held block
    k, v = rows(len(slots), heads, dim, dtype, seed=block, amp=0.8)
    c.write(k, v, slots)
    c.check()
    c.read(list(range(c.slots)), dtype)
    c.read([5, -1, c.slots, 5, 2 ** 31 - 1, -2 ** 31, 0, 7 * page + 1], FP if dtype == BF else BF)


@pytest.mark.parametrize("kind", KINDS)
def test_token_by_token(kind):
    """Scales that grow now and then, and codes that go over to them again and again."""
    c = Cache(4, 32, 2, 64, 16, kind, seed=3)
    order = [2, 0, 3]
    for t in range(70):
        k, v = rows(1, 2, 64, BF, seed=t, amp=2.0 ** ((t * 7) % 5 - 2))
        c.write(k, v, [order[t // 32] * 32 + t % 32])
        if t % 16 in (0, 1, 7, 15):
            c.check()
    c.check()


def test_back_and_forward_again():
    """A sequence taken back into a block, and continued; then from the block's start."""
    c = Cache(2, 16, 1, 64, 16, torch.int8, seed=4)
    for n, (lo, hi) in enumerate([(0, 16), (5, 9), (9, 16), (0, 3), (3, 4)]):
        k, v = rows(hi - lo, 1, 64, BF, seed=n, amp=2.0 ** n)
        c.write(k, v, list(range(16 + lo, 16 + hi)))
        c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_values_on_borders(kind, dtype):
    """Small whole numbers and simple fractions over scales made of them: quotients on borders, or next to
    them by the scale's last bit."""
    gen = torch.Generator().manual_seed(7)
    c = Cache(40, 16, 4, 128, 16, kind, seed=7)
    T = 640
    x = torch.randint(-64, 65, (T, 4, 128), generator=gen).float() * 2.0 ** torch.randint(-9, 3, (T, 4, 128), generator=gen)
    k = x.to(dtype)
    v = (torch.randint(-255, 256, (T, 4, 128), generator=gen).float() / 4).to(dtype)
    c.write(k, v, list(range(T)))
    c.check()
    # the same over held blocks, whose old codes go over to new scales that divide the old ones simply
    for s in c.scale:
        s.copy_(torch.ones_like(s) * 2.0 ** -4)
    c.dev_scale = [s.cuda() for s in c.scale]
    c.write((x[:40] * 3).to(dtype), v[:40], [16 * i + 8 for i in range(40)])
    c.check()
    c.read(list(range(T)), dtype)


@pytest.mark.parametrize("kind", KINDS)
def test_sizes_of_values(kind):
    """Zeros, the smallest and the largest values of the types; a scale has a least value."""
    c = Cache(8, 16, 1, 64, 16, kind, seed=8)
    k = torch.zeros(96, 1, 64, dtype=BF)
    v = torch.zeros(96, 1, 64, dtype=BF)
    for i, amp in enumerate([0.0, 2.0 ** -133, 2.0 ** -120, 2.0 ** -70, 1.0, 3.38e38]):
        k[16 * i:16 * i + 16] = (torch.randn(16, 1, 64, generator=torch.Generator().manual_seed(i)).clamp(-1, 1) * amp).to(BF)
        v[16 * i:16 * i + 16, :, 3] = amp
    c.write(k, v, list(range(96)))
    c.check()
    c.read(list(range(96)), BF)
    c = Cache(2, 16, 1, 64, 16, kind, seed=9)
    k = torch.randn(32, 1, 64, generator=torch.Generator().manual_seed(5))
    k[:16] *= 65504.0 / k[:16].abs().max()
    k[16:] *= 2.0 ** -22
    c.write(k.to(FP), k.to(FP), list(range(32)))
    c.check()
    c.read(list(range(32)), FP)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_finite(kind, bad):
    """They make NaN of their block and head, until it is started anew; nothing else changes."""
    c = Cache(3, 16, 2, 64, 16, kind, seed=10)
    k, v = rows(20, 2, 64, BF, seed=1)
    k[3, 1, 60] = bad
    v[17, 0, 0] = bad
    c.write(k, v, list(range(20)))
    c.check()
    got = c.read(list(range(20)), BF)
    assert bool(got[0][:16, 1].isnan().all()) and bool(got[1][16:, 0].isnan().all())
    k, v = rows(2, 2, 64, BF, seed=2)
    c.write(k[:1], v[:1], [20])               # stays
    c.check()
    c.write(k[1:], v[1:], [16])               # anew
    c.check()
    assert not bool(c.dev_scale[1][1, 0].isnan().any())


def test_every_code():
    for kind in KINDS:
        codes = torch.arange(256, dtype=torch.uint8).view(kind).reshape(1, 16, 1, 16).repeat(1, 1, 2, 4)
        c = Cache(1, 16, 2, 64, 16, kind, seed=11)
        c.codes = [codes.clone(), codes.clone()]
        c.dev = [x.cuda() for x in c.codes]
        for scale in (1.0, 0.3, 1e-3, 700.0, 2.0 ** -126, 1.0039062):
            c.scale = [torch.full((1, 1, 2), scale), torch.full((1, 1, 2), scale / 3).clamp(min=2.0 ** -126)]
            c.dev_scale = [s.cuda() for s in c.scale]
            for dtype in (BF, FP):
                c.read(list(range(16)), dtype)


def test_strides():
    """Keys and values as parts of one projection, scales in another order, outputs inside a wider buffer."""
    c = Cache(3, 32, 2, 64, 16, torch.int8, "kv", seed=12)
    c.dev_scale = [torch.empty(2, 3, 2, device="cuda").permute(1, 2, 0).copy_(s) for s in c.scale]
    qkv = torch.randn(21, 6, 64, generator=torch.Generator().manual_seed(3)).to(BF)
    dev = qkv.cuda()
    slots = list(range(40, 61))
    w.quantized_kv_write(dev[:, 2:4], dev[:, 4:6], *c.dev, *c.dev_scale, ints(slots))
    for i, at in enumerate((2, 4)):
        qo.write(qkv[:, at:at + 2], c.codes[i], c.scale[i], slots)
    c.check()
    wide = torch.full((96, 5, 64), 9.0, dtype=BF, device="cuda")
    c.read(list(range(96)), BF, out=(wide[:, 0:2], wide[:, 3:5]))
    assert bool((wide[:, 2] == 9).all())


def test_large_calls():
    """Slots past 2^31 bytes of the cache, with the codes of a small one from the first whole block on."""
    heads, dim, page = 8, 256, 128
    pages = (1 << 31) // (heads * dim * page) + 9
    codes = torch.zeros(2, pages, page, heads, dim, dtype=torch.int8, device="cuda")
    scale = torch.ones(2, pages, page // 64, heads, device="cuda")
    T = 3000
    k, v = rows(T, heads, dim, BF, seed=13)
    first = pages * page - T
    slots = torch.arange(first, first + T, dtype=torch.int32, device="cuda")
    w.quantized_kv_write(k.cuda(), v.cuda(), codes[0], codes[1], scale[0], scale[1], slots)
    got = w.quantized_kv_read(codes[0], codes[1], scale[0], scale[1], slots)
    small = Cache(T // page + 2, page, heads, dim, 64, torch.int8)
    near = list(range(small.slots - T, small.slots))
    small.write(k, v, near)
    want = w.quantized_kv_read(*small.dev, *small.dev_scale, ints(near))
    assert torch.equal(got[0][60:], want[0][60:]) and torch.equal(got[1][60:], want[1][60:])
    assert not bool(codes[:, :pages - T // page - 1].any())


def test_more_threads_than_one_axis_holds():
    """2^26 tokens of 17 heads, one row for all, most of them with no slot."""
    T, heads = 1 << 26, 17
    c = Cache(3, 16, heads, 64, 16, torch.int8, seed=21)
    k, v = rows(1, heads, 64, BF, seed=21)
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    slots[5], slots[T // 2], slots[T - 1] = 0, 16, 32
    w.quantized_kv_write(k.cuda().expand(T, -1, -1), v.cuda().expand(T, -1, -1), *c.dev, *c.dev_scale, slots)
    got = w.quantized_kv_read(*c.dev, *c.dev_scale, ints([0, 16, 32]))
    small = Cache(3, 16, heads, 64, 16, torch.int8, seed=21)
    small.write(k.expand(3, -1, -1), v.expand(3, -1, -1), [0, 16, 32])
    want = w.quantized_kv_read(*small.dev, *small.dev_scale, ints([0, 16, 32]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [1, 2, 17, 1000])
def test_many_runs(T):
    """Every token in a block of its own, and runs that cross all places of a wave's share of the tokens."""
    c = Cache(T + 2, 16, 1, 64, 16, torch.int8, seed=T)
    k, v = rows(T, 1, 64, BF, seed=T)
    perm = torch.randperm(T, generator=torch.Generator().manual_seed(T)).tolist()
    c.write(k, v, [16 * p + (5 * p) % 16 for p in perm])
    c.check()
    c = Cache(T + 2, 16, 1, 64, 16, torch.float8_e4m3fn, seed=T)
    c.write(k, v, list(range(9, 9 + T)))
    c.check()


def test_ways_in_streams_and_refusals():
    c = Cache(2, 16, 2, 64, 16, torch.int8, seed=14)
    k, v = rows(5, 2, 64, BF, seed=14)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.write(k, v, list(range(5)), stream=side)
    side.synchronize()
    c.check()
    a = w.quantized_kv_read(*c.dev, *c.dev_scale, ints(list(range(5))))
    out = (torch.empty_like(a[0]), torch.empty_like(a[1]))
    assert w.quantized_kv_read(*c.dev, *c.dev_scale, ints(list(range(5))), out=out)[0] is out[0]
    assert torch.equal(a[0], out[0]) and torch.equal(a[1], out[1])
    none = w.quantized_kv_read(*c.dev, *c.dev_scale, ints([]))
    assert none[0].shape == (0, 2, 64)
    w.quantized_kv_write(k[:0].cuda(), v[:0].cuda(), *c.dev, *c.dev_scale, ints([]))
    with pytest.raises(ValueError, match="k_scale"):
        w.quantized_kv_write(k.cuda(), v.cuda(), *c.dev, c.dev_scale[0][:1], c.dev_scale[1], ints([0] * 5))
    with pytest.raises(ValueError, match="do not divide"):
        w.quantized_kv_write(k.cuda(), v.cuda(), *c.dev, *[torch.ones(2, 3, 2, device="cuda")] * 2, ints([0] * 5))
    with pytest.raises(w.W4A16Error):
        w.quantized_kv_write(k.cuda(), v.cuda(), *c.dev, *[torch.ones(2, 2, 2, device="cuda")] * 2, ints([0] * 5))
    with pytest.raises(TypeError, match="dtype"):
        w.quantized_kv_read(*c.dev, *c.dev_scale, ints([0]), dtype=torch.float32)
    with pytest.raises(TypeError, match="k_cache"):
        w.quantized_kv_read(k[None].cuda(), k[None].cuda(), *c.dev_scale, ints([0]))


def test_runs_that_meet_in_a_block_touch_nothing_else():
    """What their block then holds is not said; all other blocks and heads are as they were."""
    c = Cache(4, 32, 2, 64, 16, torch.int8, seed=15)
    before = [x.clone() for x in c.dev + c.dev_scale]
    k, v = rows(6, 2, 64, BF, seed=15)
    w.quantized_kv_write(k.cuda(), v.cuda(), *c.dev, *c.dev_scale, ints([40, 41, 45, 40, 33, 40]))
    for x, y in zip(c.dev + c.dev_scale, before):
        if x.dim() == 4:
            x, y = x.reshape(8, 16, 2, 64), y.reshape(8, 16, 2, 64)
        else:
            x, y = x.reshape(8, 2), y.reshape(8, 2)
        rest = [0, 1, 3, 4, 5, 6, 7]
        assert torch.equal(x[rest], y[rest])


def test_graph_of_a_step():
    """A captured write and read, replayed over slots that move on, against the same calls made eagerly."""
    a, b = (Cache(6, 16, 2, 64, 16, torch.float8_e4m3fn, seed=16) for _ in range(2))
    k, v = (t.cuda() for t in rows(3, 2, 64, BF, seed=16))
    slots = ints([16, 40, -1])
    out = tuple(torch.empty(96, 2, 64, dtype=BF, device="cuda") for _ in range(2))
    every = ints(list(range(96)))

    def step(c):
        w.quantized_kv_write(k, v, *c.dev, *c.dev_scale, slots)
        return w.quantized_kv_read(*c.dev, *c.dev_scale, every, out=out)

    keep = [x.clone() for x in a.dev + a.dev_scale]
    step(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    for x, y in zip(a.dev + a.dev_scale, keep):
        x.copy_(y)
    for i in range(5):
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step(b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.equal(x.float(), y.float()) for x, y in zip(a.dev + a.dev_scale, b.dev + b.dev_scale))
        slots += torch.tensor([1, 1, 0], dtype=torch.int32, device="cuda")
        k.mul_(-1.5)
        v.mul_(1.25)
