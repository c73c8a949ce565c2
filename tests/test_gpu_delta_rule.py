"""The gated delta rule on the GPU, packed and single-token, against the float64 recurrence."""
import math

import pytest
import torch

import delta_oracle as do
import weight_only_int4_w4a16_amd as w

pytestmark = pytest.mark.gpu

DIMS = [(64, 64), (64, 128), (128, 64), (128, 128)]
BF, FP = torch.bfloat16, torch.float16


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Delta:
    def __init__(self, lens, H, Hk, Dk, Dv, dtype=BF, decay="token", initial=True, seed=0, rate=0.1, lead=0, beta=(0.0, 1.0),
                 norm=1.0, alike=0.0):
        gen = torch.Generator().manual_seed(seed)
        T = sum(lens) + lead
        self.lens, self.lead, self.T, self.dtype, self.H = lens, lead, T, dtype, H

        def rand(*shape):
            return torch.randn(shape, generator=gen)

        self.q = (rand(T, Hk, Dk)).to(dtype)
        k = rand(T, Hk, Dk) * (1 - alike) + rand(Hk, Dk) * alike * Dk ** 0.5
        self.k = (torch.nn.functional.normalize(k, dim=-1) * norm).to(dtype)
        self.v = rand(T, H, Dv).to(dtype)
        self.g = -torch.rand(T, H, generator=gen) * rate if decay == "token" else -torch.rand(H, generator=gen) * rate
        self.beta = beta[0] + (beta[1] - beta[0]) * torch.rand(T, H, generator=gen)
        self.state = rand(len(lens), H, Dk, Dv) if initial else None
        self.scale = Dk ** -0.5

    def run(self, **kw):
        cu = [self.lead]
        for n in self.lens:
            cu.append(cu[-1] + n)
        args = dict(cu_seqlens=ints(cu), state=None if self.state is None else self.state.cuda())
        args.update(kw)
        out, state = w.delta_rule(*[args.pop(x, getattr(self, x).cuda()) for x in ("q", "k", "v", "g", "beta")], **args)
        torch.cuda.synchronize()
        return out, state

    def check(self, out, state):
        at = self.lead
        for s, n in enumerate(self.lens):
            rows = slice(at, at + n)
            g = (self.g[rows] if self.g.dim() == 2 else self.g.expand(n, self.H)).double()
            S0 = torch.zeros(state.shape[1:]).double() if self.state is None else self.state[s].double()
            x = [self.q[rows].double(), self.k[rows].double(), self.v[rows].double(), g, self.beta[rows].double()]
            o, S, u, starts = do.delta(*x, S0, self.scale)
            tol, tol_s = do.bounds(self.dtype, *x, self.scale, o, u, starts, S)
            err = (out[rows].cpu().double() - o).abs()
            bad = ~(err <= tol)
            assert not bool(bad.any()), (f"sequence {s} of {n}: out off by {float((err / tol).max()):.3g} bounds, "
                                         f"first at {torch.nonzero(bad)[0].tolist()}")
            err = (state[s].cpu().double() - S).abs()
            assert bool((err <= tol_s).all()), f"sequence {s} of {n}: state off by {float((err / tol_s).max()):.3g} bounds"
            at += n


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 33, 47, 49, 63, 64, 65, 127, 128, 129, 200, 257, 400])
def test_single_sequence_lengths(n):
    x = Delta([n], 2, 2, 128, 128, seed=n)
    x.check(*x.run())


@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("dtype,decay,initial,H,Hk", [
    (BF, "token", True, 4, 2), (FP, "head", False, 3, 3), (FP, "token", True, 3, 1), (BF, "head", True, 2, 2),
])
def test_dims_types_and_decays(Dk, Dv, dtype, decay, initial, H, Hk):
    x = Delta([70, 0, 1, 130, 64, 3], H, Hk, Dk, Dv, dtype, decay, initial, seed=Dk + Dv)
    out, state = x.run()
    x.check(out, state)
    again, state2 = x.run()
    assert torch.equal(out, again) and torch.equal(state, state2)


@pytest.mark.parametrize("n,rate", [(1500, 0.02), (2500, 0.5), (4099, 0.002)])
def test_long_sequences(n, rate):
    x = Delta([n, 70], 2, 1, 64, 64, seed=n, rate=rate)
    x.check(*x.run())
    x = Delta([n], 1, 1, 128, 128, FP, "head", False, seed=n, rate=rate)
    x.check(*x.run())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_error_of_long_sequences(dtype):
    """States keep float32's digits: 24 bits of every operand, sums of up to 128 terms per 64 tokens (random
    signs: a few half steps), 60 blocks: 2^-24 * sqrt(60) * 4 is 2e-6 of the norm. Outputs: their own rounding,
    and two terms of that size or less (half_step / sqrt 3 each)."""
    x = Delta([3840], 2, 2, 128, 128, dtype, seed=5, rate=0.01)
    out, state = x.run()
    o, S, _, _ = do.delta(x.q.double(), x.k.double(), x.v.double(), x.g.double(), x.beta.double(), x.state[0].double(), x.scale)
    assert float((state[0].cpu().double() - S).norm() / S.norm()) < 2e-6
    assert float((out.cpu().double() - o).norm() / o.norm()) < do.half_step(dtype)


def test_decays_at_their_ends():
    x = Delta([150], 2, 2, 64, 64, seed=1, rate=0.0)
    x.check(*x.run())
    x = Delta([200], 2, 2, 64, 128, seed=2, rate=300.0)         # most weights vanish
    x.check(*x.run())
    x = Delta([260, 90], 2, 2, 128, 64, seed=3)
    x.g[[0, 5, 63, 64, 100, 128, 190, 261, 349]] = -math.inf      # the state is cleared there
    out, state = x.run()
    assert bool(torch.isfinite(out).all() and torch.isfinite(state).all())
    x.g[torch.isinf(x.g)] = -193.0
    x.check(out, state)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("beta,alike,norm", [((0.0, 0.0), 0.0, 1.0), ((1.0, 1.0), 1.0, 1.0), ((1.9, 2.0), 0.9, 1.0),
                                             ((0.0, 1.0), 0.7, 1.0), ((0.5, 1.0), 0.3, 0.01), ((0.0, 0.02), 0.5, 8.0)])
def test_betas_and_alike_keys(dtype, beta, alike, norm):
    """From no update at all to the same key over and over with the largest step, short and long keys."""
    x = Delta([200, 33], 2, 1, 128, 64, dtype, seed=11, beta=beta, alike=alike, norm=norm, rate=0.05)
    x.check(*x.run())


def test_states_and_values_of_all_sizes():
    x = Delta([100, 40], 2, 2, 64, 64, seed=21)
    x.state *= torch.logspace(-20, 20, 64)                        # columns forty orders apart
    x.v = (x.v.float() * torch.logspace(-15, 15, 64)).to(BF)
    x.check(*x.run())
    x = Delta([100], 2, 2, 64, 64, FP, seed=22)
    x.state *= torch.logspace(-8, 8, 64)
    x.v = (x.v.float() * torch.logspace(-5, 3, 64)).to(FP)
    x.scale, x.q = 2.0 ** -12, (x.q.float() * 300).to(FP)
    out, state = x.run(scale=x.scale, v=x.v.cuda(), q=x.q.cuda())
    fine = torch.isfinite(out.float()).all(0)                     # columns that float16 can hold
    assert bool(fine[:, :48].all())
    x.v, x.state, keep = x.v[..., :48], x.state[..., :48], slice(0, 48)
    x.check(out[..., keep], state[..., keep])


def test_strides_and_untouched_rows():
    """Rows of a wider buffer, heads swapped, the sequences not at its start: nothing else is written."""
    x = Delta([90, 65], 4, 2, 64, 128, seed=31, lead=7)
    wide = torch.zeros(x.T, 2 * 64 * 2 + 4 * 128, dtype=BF, device="cuda")
    q = wide[:, :128].view(-1, 2, 64)
    k = wide[:, 128:256].view(-1, 2, 64)
    v = wide[:, 256:].view(-1, 128, 4).transpose(1, 2)
    vt = torch.empty(4, x.T, 128, dtype=BF, device="cuda").transpose(0, 1)   # [T, H, Dv], heads far apart
    q.copy_(x.q), k.copy_(x.k), vt.copy_(x.v)
    assert v.stride(2) != 1
    g = torch.empty(4, x.T, device="cuda").T
    g.copy_(x.g)
    beta = torch.empty(x.T, 4, 3, device="cuda")[..., 1]
    beta.copy_(x.beta)
    out = torch.full((x.T + 3, 4, 2, 128), 5.0, dtype=BF, device="cuda")
    o, state = x.run(q=q, k=k, v=vt, g=g, beta=beta, out=out[:x.T, :, 0])
    x.check(o, state)
    assert bool((out[:, :, 1] == 5).all() and (out[x.T:] == 5).all() and (out[:7] == 5).all())
    with pytest.raises(ValueError, match="unit stride"):
        x.run(v=v)


def test_one_beta_per_head_and_broadcast_decays():
    x = Delta([77], 3, 3, 64, 64, seed=41)
    x.beta = x.beta[:1].expand(77, 3)
    out, state = x.run(beta=x.beta[0].cuda())
    x.check(out, state)
    out2, state2 = x.run(beta=x.beta[0].cuda().expand(77, 3))
    assert torch.equal(out, out2) and torch.equal(state, state2)


def test_state_in_place_and_none():
    x = Delta([70, 0, 5], 2, 2, 64, 64, seed=51)
    out, state = x.run()
    s = x.state.cuda()
    out2, got = x.run(state=s, state_out=s)
    assert got is s and torch.equal(s, state) and torch.equal(out, out2)
    assert torch.equal(state[1].cpu(), x.state[1])               # no tokens: as it came
    x.state = None
    out, state = x.run()
    x.check(out, state)
    assert not bool(state[1].any())


def test_many_sequences():
    """More sequences than lanes of a wave, most of them short, some empty."""
    lens = [(7 * i) % 23 if i % 50 else 130 for i in range(300)]
    x = Delta(lens, 1, 1, 64, 64, seed=61)
    x.check(*x.run())
    one = Delta([0] * 70 + [65] + [0] * 70, 1, 1, 64, 64, seed=62)
    one.check(*one.run())


def test_no_tokens():
    x = Delta([0, 0], 2, 2, 64, 128, seed=63)
    out, state = x.run()
    assert out.shape == (0, 2, 128) and torch.equal(state.cpu(), x.state)


def test_prompt_in_pieces_and_single_tokens():
    """A prompt at once, in two calls, and token by token give the same within both forms' bounds."""
    x = Delta([100], 4, 2, 128, 128, seed=71)
    out, state = x.run()
    dev = [t.cuda() for t in (x.q, x.k, x.v, x.g, x.beta)]
    o1, s = w.delta_rule(*[t[:37] for t in dev], state=x.state.cuda())
    o2, s = w.delta_rule(*[t[37:64] for t in dev], state=s)
    rows = [w.delta_rule_step(*[t[i:i + 1] for t in dev], s) for i in range(64, 100)]
    x.check(torch.cat([o1, o2] + rows), s)


@pytest.mark.parametrize("what", ["v", "k", "beta", "decay", "q"])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_what_is_not_finite_reaches_later_tokens_only(what, dtype, bad):
    """Token 70 of the first sequence; the second one, and all tokens before, are as without it."""
    x = Delta([150, 60], 2, 2, 64, 64, dtype, seed=81)
    out, state = x.run()
    if what == "v":
        x.v[70, 1, 5] = bad
    elif what in ("k", "q"):
        getattr(x, what)[70, 1, 3] = bad
    elif what == "beta":
        x.beta[70, 1] = bad
    else:
        x.g[70, 1] = bad
    out2, state2 = x.run()
    assert torch.equal(out2[:70], out[:70]) and torch.equal(out2[150:], out[150:]) and torch.equal(state2[1], state[1])
    assert torch.equal(out2[:, 0], out[:, 0]) and torch.equal(state2[0, 0], state[0, 0])
    if what == "q":
        assert not bool(torch.isfinite(out2[70, 1]).any())
        assert torch.equal(out2[71:], out[71:]) and torch.equal(state2, state)
    elif what == "v":
        assert not bool(torch.isfinite(out2[70:150, 1, 5]).any()) and not bool(torch.isfinite(state2[0, 1, :, 5]).any())
        rest = [i for i in range(64) if i != 5]
        assert torch.equal(out2[:, :, rest], out[:, :, rest]) and torch.equal(state2[..., rest], state[..., rest])
    else:
        assert not bool(torch.isfinite(out2[70:150, 1]).any()) and not bool(torch.isfinite(state2[0, 1]).any())


def test_sequence_bounds_outside_the_tokens():
    """Entries are clamped to the tokens there are; what lies in no sequence is not written."""
    x = Delta([40, 30], 1, 1, 64, 64, seed=91)
    out = torch.full_like(x.v, 7.0).cuda()
    o, state = x.run(cu_seqlens=ints([-5, 40, 1000]), out=out)
    x.check(o, state)
    out = torch.full_like(x.v, 7.0).cuda()
    x.run(cu_seqlens=ints([10, 20, 30]), out=out)
    assert bool((out[:10] == 7).all() and (out[30:] == 7).all() and (out[10:30] != 7).any())


@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B,H,Hk", [(1, 4, 2), (7, 3, 1), (40, 4, 4)])
def test_step(Dk, Dv, dtype, B, H, Hk):
    x = Delta([B], H, Hk, Dk, Dv, dtype, seed=B + Dk, rate=1.0)
    state = torch.randn(B, H, Dk, Dv, generator=torch.Generator().manual_seed(1))
    kk = x.k.double().repeat_interleave(H // Hk, 1)
    S = x.g.double().exp()[..., None, None] * state.double()
    u = x.beta.double()[..., None] * (x.v.double() - (kk[..., None, :] @ S)[..., 0, :])
    S = S + kk[..., :, None] * u[..., None, :]
    o = x.scale * (x.q.double().repeat_interleave(H // Hk, 1)[..., None, :] @ S)[..., 0, :]
    tol, tol_s = do.step_bounds(dtype, x.q.double(), x.k.double(), x.v.double(), x.g.double(), x.beta.double(),
                                state.double(), x.scale, o, S)
    dev = [t.cuda() for t in (x.q, x.k, x.v, x.g, x.beta)]
    s = state.cuda()
    other = torch.empty_like(s)
    out = w.delta_rule_step(*dev, s, state_out=other)
    assert torch.equal(s.cpu(), state)
    assert bool(((out.cpu().double() - o).abs() <= tol).all()) and bool(((other.cpu().double() - S).abs() <= tol_s).all())
    again = w.delta_rule_step(*dev, s, out=torch.empty_like(out))
    assert torch.equal(again, out) and torch.equal(s, other)


def test_step_slots():
    x = Delta([5], 2, 1, 64, 64, seed=101)
    pool = torch.randn(6, 2, 64, 64, generator=torch.Generator().manual_seed(2)).cuda()
    before = pool.clone()
    dev = [t.cuda() for t in (x.q, x.k, x.v, x.g, x.beta)]
    rows = [4, -1, 0, 6, 2]
    out = w.delta_rule_step(*dev, pool, slots=ints(rows))
    want = before[[4, 0, 2]].clone()
    o = w.delta_rule_step(*[t[[0, 2, 4]].contiguous() for t in dev], want)
    assert torch.equal(out[[0, 2, 4]], o) and torch.equal(pool[[4, 0, 2]], want)
    assert not bool(out[[1, 3]].any()) and torch.equal(pool[[1, 3, 5]], before[[1, 3, 5]])
    none = w.delta_rule_step(*[t[:0] for t in dev], pool)
    assert none.shape == (0, 2, 64)


def test_both_ways_into_the_library_and_another_stream():
    x = Delta([130, 20], 2, 2, 64, 64, seed=111)
    out, state = x.run()
    work = w.delta_rule_workspace(x.q.cuda(), x.v.cuda(), 2)
    o2, s2 = x.run(out=torch.empty_like(out), state_out=torch.empty_like(state), workspace=work)
    assert torch.equal(out, o2) and torch.equal(state, s2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o3, s3 = x.run(stream=side)
    assert torch.equal(out, o3) and torch.equal(state, s3)
    with pytest.raises(w.W4A16Error):
        x.run(out=torch.empty_like(out), state_out=torch.empty_like(state), workspace=work[:8])
    with pytest.raises(ValueError, match="beta"):
        x.run(beta=x.beta[:5].cuda())
    with pytest.raises(TypeError, match="beta"):
        x.run(beta=x.beta.double().cuda())


def test_offsets_past_32_bits():
    n, ld = 130, 2 ** 24 - 8   # the longest strides: a chunk's rows lie up to 2^31 bytes apart
    x = Delta([n], 2, 1, 128, 64, seed=990)

    def far(t, dtype):
        big = torch.empty((n - 1) * ld + t[0].numel(), dtype=dtype, device="cuda")
        return big.as_strided(t.shape, (ld,) + t.stride()[1:])

    kw = {}
    for name in ("q", "k", "v", "g", "beta"):
        t = getattr(x, name)
        kw[name] = far(t, t.dtype)
        kw[name].copy_(t)
    out = far(x.v, x.dtype)
    x.check(*x.run(out=out, **kw))


@pytest.mark.parametrize("n", [1, 70, 130])
@pytest.mark.parametrize("ld", [0, 8, 40])
def test_rows_that_share_memory(n, ld):
    """Rows closer than their length, or all in one place: rows behind the sequence's end are read as well, and count
    for nothing."""
    x = Delta([n], 1, 1, 64, 64, seed=n + ld, norm=0.2)

    def close(t, width):
        big = (torch.randn((n + 63) * ld + width, generator=torch.Generator().manual_seed(ld)) * 0.1).to(t.dtype)
        big[(n - 1) * ld + width:] = math.nan                     # not the sequence's
        return big.as_strided((n, 1, width), (ld, width, 1))

    x.q, x.k, x.v = (close(t, 64) for t in (x.q, x.k, x.v))
    dev = []
    for t in (x.q, x.k, x.v):
        big = torch.empty((n + 63) * ld + 64, dtype=t.dtype, device="cuda")
        big.copy_(t.as_strided((big.numel(),), (1,)))
        dev.append(big.as_strided((n, 1, 64), (ld, 64, 1)))
    x.check(*x.run(q=dev[0], k=dev[1], v=dev[2]))


def test_more_threads_than_one_axis_holds():
    """16384 sequences of 130 heads, most without a token: their states are zeros, the others' those of a call alone."""
    seqs, H, at, lens = 16384, 130, [0, 9001, 16383], [70, 1, 130]
    x = Delta(lens, H, 65, 64, 64, seed=77, initial=False)
    want, states = x.run()
    cu = torch.zeros(seqs + 1, dtype=torch.int32)
    for s, n in zip(at, lens):
        cu[s + 1:] += n
    big = torch.full((seqs, H, 64, 64), 7.0, device="cuda")
    out, big = w.delta_rule(x.q.cuda(), x.k.cuda(), x.v.cuda(), x.g.cuda(), x.beta.cuda(), cu_seqlens=cu.cuda(),
                            state_out=big)
    assert torch.equal(out, want) and torch.equal(big[at], states)
    big[at] = 0
    assert not any(bool(part.any()) for part in big.split(1024))


def test_states_that_are_not_finite():
    """An infinity or NaN in a first state stays in its column and head."""
    x = Delta([70, 3], 2, 1, 64, 64, seed=78)
    out, state = x.run()
    for bad in (math.nan, math.inf, -math.inf):
        first = x.state.clone()
        first[0, 1, 5, 9] = bad
        o, s = x.run(state=first.cuda())
        assert not bool(torch.isfinite(o[:70, 1, 9]).any()) and not bool(torch.isfinite(s[0, 1, 5, 9]))
        o[:70, 1, 9], s[0, 1, :, 9] = out[:70, 1, 9], state[0, 1, :, 9]
        assert torch.equal(o, out) and torch.equal(s, state)


def test_two_streams_at_once():
    """Calls side by side with workspaces of their own."""
    xs = [Delta([300, 70], 4, 2, 128, 64, seed=s) for s in (1, 2)]
    want = [x.run() for x in xs]
    dev = [[t.cuda() for t in (x.q, x.k, x.v, x.g, x.beta, x.state)] for x in xs]
    cu = ints([0, 300, 370])
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [w.delta_rule(*d[:5], cu_seqlens=cu, state=d[5], stream=s) for d, s in zip(dev, streams)]
        torch.cuda.synchronize()
        for (o, s), (o2, s2) in zip(got, want):
            assert torch.equal(o, o2) and torch.equal(s, s2)


def test_heads_on_every_place():
    """Head counts that the 8 XCDs divide and do not divide, shared and own keys, one sequence and several."""
    for lens, H, Hk in [([70], 1, 1), ([70], 3, 3), ([65, 2], 6, 2), ([66], 16, 2), ([5, 70, 1], 8, 8), ([70], 24, 8), ([64] * 9, 2, 1)]:
        x = Delta(lens, H, Hk, 64, 64, seed=H + Hk)
        x.check(*x.run())
