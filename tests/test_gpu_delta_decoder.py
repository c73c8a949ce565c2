"""The delta rule and the 8-bit cache as a decoder uses them: in the hybrid example, each call against its float64
definition on the operands that it gets there, and in captured steps."""
import os
import sys

import pytest
import torch

import delta_oracle as do
import mixer_oracle as mo
import quantized_oracle as qo
import weight_only_int4_w4a16_amd as w

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

KINDS = [torch.int8, torch.float8_e4m3fn]


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def check_sequence(q, k, v, g, beta, s0, out, s1):
    x = [t.cpu().double() for t in (q, k, v, g, beta)]
    scale = q.shape[2] ** -0.5
    o, S, u, starts = do.delta(*x, s0.cpu().double(), scale)
    tol, tol_s = do.bounds(q.dtype, *x, scale, o, u, starts, S)
    assert bool(((out.cpu().double() - o).abs() <= tol).all())
    assert bool(((s1.cpu().double() - S).abs() <= tol_s).all())


def check_delta(q, k, v, g, beta, cu_seqlens, state, state_out):
    before = state.clone()
    out, end = w.delta_rule(q, k, v, g, beta, cu_seqlens=cu_seqlens, state=state, state_out=state_out)
    cu = cu_seqlens.tolist()
    for b in range(len(cu) - 1):
        t = slice(cu[b], cu[b + 1])
        check_sequence(q[t], k[t], v[t], g[t], beta[t], before[b], out[t], end[b])
    return out, end


def check_step(q, k, v, g, beta, state):
    before = state.clone()
    out = w.delta_rule_step(q, k, v, g, beta, state)
    for b in range(q.shape[0]):
        t = slice(b, b + 1)
        check_sequence(q[t], k[t], v[t], g[t], beta[t], before[b], out[t], state[b])
    return out


def check_write(k, v, k_cache, v_cache, k_scale, v_scale, slot_map):
    codes, scales = [k_cache.cpu(), v_cache.cpu()], [k_scale.cpu(), v_scale.cpu()]
    for x, c, s in zip((k, v), codes, scales):
        qo.write(x.cpu(), c, s, slot_map.tolist())
    w.quantized_kv_write(k, v, k_cache, v_cache, k_scale, v_scale, slot_map)
    for c, got in zip(codes + scales, (k_cache, v_cache, k_scale, v_scale)):
        assert torch.equal(c.float(), got.cpu().float())


def check_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens):
    out = w.quantized_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)
    page, scale = k_cache.shape[1], q.shape[2] ** -0.5
    full = [qo.values(c.cpu()) * qo.spread(s.cpu(), page) for c, s in ((k_cache, k_scale), (v_cache, v_scale))]
    weight = float(qo.spread(v_scale.cpu(), page).max())
    for b, n in enumerate(seq_lens.tolist()):
        at = torch.arange(n)
        k, v = (x[page_table[b].cpu().long()[at // page], at % page] for x in full)
        o, _, mag, qk, top = mo.attention(q[b].cpu().double(), k, v, scale)
        tol, _ = qo.attention_bounds(q.dtype, o, mag, qk, top, n, q.shape[2], weight, qo.LARGEST[k_cache.dtype])
        assert bool(((out[b].cpu().double() - o).abs() <= tol).all()), f"token {b} of length {n}"
    return out


class Checked:
    """The library with its delta rule and 8-bit cache checked."""
    calls = dict(quantized_attention=check_attention, delta_rule=check_delta, delta_rule_step=check_step,
                 quantized_kv_write=check_write)

    def __init__(self):
        self.seen = set()

    def __getattr__(self, name):
        if name not in self.calls:
            return getattr(w, name)
        self.seen.add(name)
        return self.calls[name]


@pytest.mark.parametrize("kind", KINDS)
def test_calls_of_the_example(kind, monkeypatch):
    import hybrid_decode
    lib = Checked()
    monkeypatch.setattr(hybrid_decode, "w", lib)
    model = hybrid_decode.HybridDecoder(requests=3, longest=160, pages=64, seed=6, cache_type=kind, delta=True, block=16)
    gen = torch.Generator().manual_seed(7)
    prompts = [torch.randint(0, 1000, (n,), generator=gen).cuda() for n in (70, 3, 17)]
    model.generate(prompts, 4)
    assert lib.seen == set(Checked.calls)


def run(cuts, kind):
    from hybrid_decode import HybridDecoder
    model = HybridDecoder(requests=3, longest=160, pages=64, seed=3, cache_type=kind, delta=True, block=16)
    gen = torch.Generator().manual_seed(4)
    text = [torch.randint(0, 1000, (sum(c[b] for c in cuts),), generator=gen).cuda() for b in range(3)]
    at, rows = [0] * 3, [[] for _ in range(3)]
    for cut in cuts:
        logits = model.forward(torch.cat([text[b][at[b]:at[b] + cut[b]] for b in range(3)]), cut)
        for part, b in zip(logits.split(cut), range(3)):
            rows[b].append(part)
            at[b] += cut[b]
    return [torch.cat(r).float() for r in rows], model


@pytest.mark.parametrize("kind", KINDS)
def test_prompts_and_single_tokens_agree(kind):
    whole, _ = run([(70, 17, 33)], kind)
    parts, model = run([(60, 5, 32), (7, 10, 0), (1, 1, 0), (1, 1, 1), (1, 0, 0)], kind)
    assert model.lens.tolist() == [70, 17, 33]
    # bfloat16 activations as in the other form of the example: about ten roundings in each of two layers, half a step
    # of 2^-8 each. Codes: in both runs half a step off, in pieces once more where a scale grows, and the scales
    # differ; a step is 1 / 127 of a block's largest value (3.5 times its size), e4m3 2^-3 of the value.
    code = 3.5 / 127 if kind == torch.int8 else 2.0 ** -3
    for a, b in zip(whole, parts):
        off = (a - b).abs()
        assert float(off.mean()) <= 20 * 2.0 ** -9 + 1.5 * code
        assert float((off.amax(1) > 0.5 + 4 * code).float().mean()) <= 0.1


class Step:
    """A decode step of all new operators over buffers of its own: pages, cache write, attention, delta rule."""

    def __init__(self, kind, work, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        B, Hq, heads, dim, pages, page = 5, 8, 2, 64, 40, 32

        def rand(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")

        self.gen, self.B, self.page = gen, B, page
        self.qkv = rand(B, Hq + 2 * heads, dim).to(torch.bfloat16)
        self.mix = rand(B, 6, dim).to(torch.bfloat16)
        self.gates = -rand(2, B, 2).abs() * 0.3
        self.codes = torch.zeros(2, pages, page, heads, dim, dtype=kind, device="cuda")
        self.scales = torch.ones(2, pages, page // 16, heads, device="cuda")
        self.table = torch.full((B, 6), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        self.lens = ints([30, 0, 63, 64, 5])
        self.new = ints([1] * B)
        self.state = rand(B, 2, dim, dim)
        self.attended = torch.empty(B, Hq, dim, dtype=torch.bfloat16, device="cuda")
        self.mixed = torch.empty(B, 2, dim, dtype=torch.bfloat16, device="cuda")
        self.prompt, self.prompt_state = torch.empty_like(self.mixed), torch.empty_like(self.state)
        self.tables = w.page_tables_buffers(B, B)
        self.back = [torch.empty(B, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.work, self.delta_work = work
        self.cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        # what was there before: the cached tokens of each request
        first = w.page_tables(torch.zeros_like(self.lens), self.lens, self.table, self.free, page, max_tokens=200)
        x = rand(2, 200, heads, dim).to(torch.bfloat16)
        w.quantized_kv_write(x[0], x[1], *self.codes, *self.scales, first.slot_map)
        self.free = self.free[int(first.counts[1]):].contiguous()

    def __call__(self):
        t = w.page_tables(self.lens, self.new, self.table, self.free, self.page, out=self.tables)
        w.quantized_kv_write(self.qkv[:, 8:10], self.qkv[:, 10:], *self.codes, *self.scales, t.slot_map)
        w.quantized_attention(self.qkv[:, :8], *self.codes, *self.scales, self.table, t.seq_lens, out=self.attended,
                              workspace=self.work)
        w.quantized_kv_read(*self.codes, *self.scales, t.slot_map, out=tuple(self.back))
        q, k, v = self.mix[:, :2], self.mix[:, 2:4], self.mix[:, 4:]
        w.delta_rule(q, k, v, self.gates[0], self.gates[1].exp(), cu_seqlens=self.cu, state=self.state,
                     state_out=self.prompt_state, out=self.prompt, workspace=self.delta_work)
        w.delta_rule_step(q, k, v, self.gates[0], self.gates[1].exp(), self.state, out=self.mixed)

    def results(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (self.attended, self.mixed, self.state, self.codes.view(torch.uint8), self.scales,
                                    self.prompt, self.prompt_state, *self.back)]

    def move(self, seed):
        """The next token's inputs; lengths and the free list go on."""
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for x in (self.qkv, self.mix):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda") * (1 + seed % 3))
        self.lens.copy_(self.tables.seq_lens)
        taken = int(self.tables.counts[1])
        self.free.copy_(torch.cat([self.free[taken:], torch.full_like(self.free[:taken], -1)]))


@pytest.mark.parametrize("kind", KINDS)
def test_two_captured_steps_share_workspaces(kind):
    """Both replayed in turn on one stream, with eager steps of other objects between them: every replay gives what the
    same step gives eagerly."""
    one = torch.zeros(1, 8, 64, dtype=torch.bfloat16, device="cuda")
    work = (w.quantized_attention_workspace(one, torch.zeros(1, 16, 2, 64, dtype=kind, device="cuda")),
            w.delta_rule_workspace(torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda"), one.expand(5, 8, 64)[:, :2], 5))
    steps, eager, graphs = [Step(kind, work, s) for s in (1, 2)], [Step(kind, work, s) for s in (1, 2)], []
    for s in steps:
        before = [x.clone() for x in (s.codes.view(torch.uint8), s.scales, s.state, s.table)]
        s()                                     # loads the library
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s()
        graphs.append(g)
        for x, y in zip((s.codes.view(torch.uint8), s.scales, s.state, s.table), before):
            x.copy_(y)
    for i in range(4):
        for s, e, g in zip(steps, eager, graphs):
            g.replay()
            e()
            for x, y in zip(s.results(), e.results()):
                assert torch.equal(x, y)
            s.move(10 * i + 3)
            e.move(10 * i + 3)


def test_a_request_taken_over_by_another_pool():
    """Keys and values read back from one cache and written to another: the same attention but for a rounding of each
    value to bfloat16 (2^-8 of it) and its new code (half a step)."""
    gen = torch.Generator().manual_seed(9)
    n, heads, dim = 75, 2, 64
    k, v = (torch.randn(n, heads, dim, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(1, 8, dim, generator=gen).to(torch.bfloat16).cuda()
    pools = [[torch.zeros(9, page, heads, dim, dtype=torch.int8, device="cuda") for _ in range(2)]
             + [torch.ones(9, page // 16, heads, device="cuda") for _ in range(2)] for page in (16, 32)]
    slots = [ints([p * 16 + i for p in (3, 8, 0, 5, 1) for i in range(16)][:n]), ints([p * 32 + i for p in (7, 2, 4)
                                                                                       for i in range(32)][:n])]
    tables = [ints([[3, 8, 0, 5, 1]]), ints([[7, 2, 4]])]
    w.quantized_kv_write(k, v, *pools[0], slots[0])
    w.quantized_kv_write(*w.quantized_kv_read(*pools[0], slots[0]), *pools[1], slots[1])
    a, b = (w.quantized_attention(q, *p, t, ints([n])) for p, t in zip(pools, tables))
    x, y = (w.quantized_kv_read(*p, s) for p, s in zip(pools, slots))
    step = float(max(p.max() for p in pools[0][2:]))
    for c, d in zip(x, y):
        assert float((c.float() - d.float()).abs().max()) <= 0.51 * step + 2.0 ** -7 * float(c.float().abs().max())
    qk = float((q.float().abs().sum(-1)).max()) * dim ** -0.5
    most = float(v.float().abs().max())
    off = 0.51 * step + 2.0 ** -8 * most                            # of a key's or a value's element
    assert float((a.float() - b.float()).abs().max()) <= off + 2 * most * qk * off + 2.0 ** -7 * most
