"""Linear attention on the GPU, packed and single-token, against the float64 recurrence."""
import math

import pytest
import torch

import mixer_oracle as mo
import weight_only_int4_w4a16_amd as w

pytestmark = pytest.mark.gpu

DIMS = [(64, 64), (64, 128), (128, 64), (128, 128)]


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Linear:
    def __init__(self, lens, H, Hk, Dk, Dv, dtype=torch.bfloat16, decay="token", initial=True, seed=0, amp=1.0,
                 rate=0.1, lead=0):
        gen = torch.Generator().manual_seed(seed)
        T = sum(lens) + lead
        self.lens, self.lead, self.T, self.dtype, self.H, self.Dk = lens, lead, T, dtype, H, Dk

        def rand(*shape):
            return (torch.randn(shape, generator=gen) * amp).to(dtype)

        self.q, self.k, self.v = rand(T, Hk, Dk), rand(T, Hk, Dk), rand(T, H, Dv)
        if decay == "token":
            self.g = -torch.rand(T, H, generator=gen) * rate
        else:
            self.g = -torch.rand(H, generator=gen) * rate
        self.state = torch.randn(len(lens), H, Dk, Dv, generator=gen) if initial else None
        self.scale = Dk ** -0.5

    def run(self, **kw):
        cu = [self.lead]
        for n in self.lens:
            cu.append(cu[-1] + n)
        args = dict(cu_seqlens=ints(cu), state=None if self.state is None else self.state.cuda())
        args.update(kw)
        out, state = w.linear_attention(args.pop("q", self.q.cuda()), args.pop("k", self.k.cuda()),
                                        args.pop("v", self.v.cuda()), args.pop("g", self.g.cuda()), **args)
        torch.cuda.synchronize()
        return out, state

    def check(self, out, state):
        at = self.lead
        for s, n in enumerate(self.lens):
            g = self.g[at:at + n] if self.g.dim() == 2 else self.g.expand(n, self.H)
            S0 = torch.zeros(state.shape[1:]).double() if self.state is None else self.state[s].double()
            o, S, mag, M = mo.linear(self.q[at:at + n].double(), self.k[at:at + n].double(),
                                     self.v[at:at + n].double(), g.double(), S0, self.scale)
            tol, tol_s = mo.linear_bounds(self.dtype, o, mag, M, n)
            err = (out[at:at + n].cpu().double() - o).abs()
            bad = ~(err <= tol)
            assert not bool(bad.any()), (f"sequence {s} of {n}: out off by {float((err / tol).max()):.3g} bounds, "
                                         f"first at {torch.nonzero(bad)[0].tolist()}")
            err = (state[s].cpu().double() - S).abs()
            assert bool((err <= tol_s).all()), f"sequence {s} of {n}: state off by {float((err / tol_s).max()):.3g} bounds"
            at += n


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 257, 400])
def test_single_sequence_lengths(n):
    x = Linear([n], 2, 2, 128, 128, seed=n)
    x.check(*x.run())


@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("dtype,decay,initial,H,Hk", [
    (torch.bfloat16, "token", True, 4, 2), (torch.float16, "head", False, 3, 3), (torch.float16, "token", True, 3, 1),
    (torch.bfloat16, "head", True, 2, 2),
])
def test_dims_types_and_decays(Dk, Dv, dtype, decay, initial, H, Hk):
    x = Linear([70, 0, 1, 130, 64, 3], H, Hk, Dk, Dv, dtype, decay, initial, seed=Dk + Dv, lead=0)
    out, state = x.run()
    x.check(out, state)
    again, state2 = x.run()
    assert torch.equal(out, again) and torch.equal(state, state2)


@pytest.mark.parametrize("n,rate", [(1500, 0.02), (2500, 0.5), (4099, 0.002)])
def test_long_sequences(n, rate):
    """Long enough to be cut into segments whose states are carried on."""
    x = Linear([n, 70], 2, 1, 64, 64, seed=n, rate=rate)
    x.check(*x.run())
    x = Linear([n], 1, 1, 128, 128, torch.float16, "head", False, seed=n, rate=rate)
    x.check(*x.run())


def test_no_decay_strong_decay_and_resets():
    x = Linear([150], 2, 2, 64, 64, seed=1, rate=0.0)
    x.check(*x.run())
    x = Linear([200], 2, 2, 64, 128, seed=2, rate=300.0)         # most weights vanish
    x.check(*x.run())
    x = Linear([260, 90], 2, 2, 128, 64, seed=3)
    x.g[[0, 5, 63, 64, 100, 128, 190, 261, 349]] = -math.inf      # the state is cleared there
    x.check(*x.run())
    x = Linear([140], 1, 1, 64, 64, torch.float16, seed=4)
    x.g[:, 0] = 0.01 * torch.randn(140)                           # growth as well
    x.check(*x.run())


def test_small_and_large_magnitudes():
    x = Linear([100], 2, 2, 64, 64, torch.bfloat16, seed=5, amp=1e-6)
    x.check(*x.run())
    x = Linear([100], 2, 2, 64, 64, torch.bfloat16, seed=6, amp=1e6)
    x.check(*x.run())
    x = Linear([300], 2, 2, 64, 64, torch.float16, "head", seed=7, amp=60.0, rate=1e-4)   # states past 65504
    x.q *= 2.0 ** -13
    x.check(*x.run())


@pytest.mark.parametrize("dtype,Dk,Dv", [(torch.bfloat16, 128, 128), (torch.float16, 64, 128), (torch.bfloat16, 128, 64)])
def test_infinities_and_nan_reach_later_tokens_only(dtype, Dk, Dv):
    """A value that is not finite makes outputs of its own and later tokens not finite, and the parts of
    the state that it enters; all that comes before it, other columns of v and other heads keep their values."""
    n, H = 200, 2
    clean = Linear([n, 70], H, H, Dk, Dv, dtype, seed=30)
    want, state = clean.run()
    for name, t, h, d, value in (("v", 100, 0, 5, math.inf), ("v", 63, 1, Dv - 1, math.nan), ("v", 0, 0, 0, -math.inf),
                                 ("k", 77, 0, 9, math.nan), ("k", 128, 1, Dk - 1, math.inf), ("q", 90, 0, 3, math.nan)):
        x = Linear([n, 70], H, H, Dk, Dv, dtype, seed=30)
        getattr(x, name)[t, h, d] = value
        out, got = x.run()
        bad = torch.zeros(want.shape, dtype=torch.bool)
        bad_state = torch.zeros(state.shape, dtype=torch.bool)
        if name == "v":
            bad[t:n, h, d] = True
            bad_state[0, h, :, d] = True
        elif name == "k":
            bad[t:n, h] = True
            bad_state[0, h, d] = True
        else:
            bad[t, h] = True
        assert torch.equal(~out.cpu().isfinite(), bad), (name, t)
        assert torch.equal(~got.cpu().isfinite(), bad_state), (name, t)
        # the others: the same sums but for what stood in the value's place, so within two bounds
        x2 = Linear([n, 70], H, H, Dk, Dv, dtype, seed=30)
        getattr(x2, name)[t, h, d] = 0.0
        ref, ref_state = x2.run()
        scale = float(want.float().abs().max())
        off = (out.float() - ref.float()).cpu()[~bad].abs().max()
        assert float(off) <= 4 * mo.half_step(dtype) * scale, (name, t)
        off = (got - ref_state).cpu()[~bad_state].abs().max()
        assert float(off) <= 2.0 ** -15 * float(ref_state.abs().max()), (name, t)


def test_step_keeps_infinities_to_their_columns():
    x = Linear([1] * 3, 2, 2, 64, 64, seed=31)
    x.v[1, 0, 7] = math.inf
    q, k, v, g, s = (t.cuda() for t in (x.q, x.k, x.v, x.g, x.state))
    out = w.linear_attention_step(q, k, v, g, s)
    bad = torch.zeros(3, 2, 64, dtype=torch.bool)
    bad[1, 0, 7] = True
    assert torch.equal(~out.cpu().isfinite(), bad)


def test_tokens_outside_sequences_are_left_alone():
    x = Linear([40, 60], 2, 2, 64, 64, seed=8, lead=5)
    extra = torch.full((105, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out, state = x.run(cu_seqlens=ints([5, 45, 85]), out=extra)
    assert bool((out[:5] == 7).all() and (out[85:] == 7).all())
    x.lens = [40, 40]
    x.check(out, state)
    # decreasing and out-of-range values are clamped: sequences of 30, 0 and 75 tokens
    x = Linear([30, 0, 75], 2, 2, 64, 64, seed=9)
    x.check(*x.run(cu_seqlens=ints([-4, 30, 10, 2 ** 31 - 1])))


def test_many_and_long_sequences_share_segments():
    """More sequences than a wave holds, some of them cut into segments."""
    gen = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 4, (80,), generator=gen).tolist()
    lens[3], lens[40], lens[79] = 1300, 700, 513
    x = Linear(lens, 1, 1, 64, 64, seed=32, rate=0.02)
    out, state = x.run()
    x.check(out, state)
    few = Linear([0, 1300, 2, 700, 0, 513, 512, 1], 2, 1, 64, 128, torch.float16, seed=33, rate=0.02)
    few.check(*few.run())


def test_in_place_state_of_several_segments():
    x = Linear([1400], 2, 2, 64, 64, seed=34, rate=0.01)
    state = x.state.cuda()
    out, got = x.run(state=state, state_out=state)
    x.check(out, got)
    again, _ = x.run()
    assert torch.equal(out, again)


def test_many_sequences():
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 5, (700,), generator=gen).tolist()
    lens[300] = 150
    x = Linear(lens, 1, 1, 64, 64, seed=10)
    x.check(*x.run())


def test_strides_stream_in_place_state_and_no_cu():
    H, Hk, D, T = 4, 2, 128, 333
    x = Linear([T], H, Hk, D, D, seed=11)
    fused = torch.zeros(T, 2 * Hk + H + 3, D, dtype=torch.bfloat16, device="cuda")
    fused[:, :Hk], fused[:, Hk:2 * Hk], fused[:, 2 * Hk:2 * Hk + H] = x.q.cuda(), x.k.cuda(), x.v.cuda()
    g = torch.zeros(H, T, device="cuda")
    g.copy_(x.g.T)
    room = torch.full((T, 2 * H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    state = x.state.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, got = x.run(q=fused[:, :Hk], k=fused[:, Hk:2 * Hk], v=fused[:, 2 * Hk:2 * Hk + H], g=g.T, cu_seqlens=None,
                     state=state, state_out=state, out=room[:, ::2], stream=side)
    assert got.data_ptr() == state.data_ptr()
    x.check(out, got)
    assert bool((room[:, 1::2] == 3).all())
    alone, _ = x.run()
    assert torch.equal(alone, out)


def test_graph_replays_match_eager_calls():
    x = Linear([500, 0, 77], 2, 2, 128, 128, seed=12)
    q, k, v, g, s = (t.cuda() for t in (x.q, x.k, x.v, x.g, x.state))
    cu = ints([0, 500, 500, 577])
    out, end, work = torch.empty_like(v), torch.empty_like(s), w.linear_attention_workspace(q, v, 3)
    row, after = torch.empty_like(v[:3]), torch.empty_like(s)

    def call():
        w.linear_attention(q, k, v, g, cu_seqlens=cu, state=s, state_out=end, out=out, workspace=work)
        w.linear_attention_step(q[:3], k[:3], v[:3], g[:3], end, state_out=after, out=row)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rep in range(4):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape).to(t.dtype))
        cu.copy_(ints([0, 500 - 100 * rep, 510 - 100 * rep, 577 - rep]))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in (out, end, row, after)]
        out.zero_()
        call()
        torch.cuda.synchronize()
        for a, b in zip(kept, (out, end, row, after)):
            assert torch.equal(a, b)


def test_empty_and_refusals():
    x = Linear([0, 0], 2, 2, 64, 64, seed=13)
    out, state = x.run()
    assert out.shape == (0, 2, 64) and torch.equal(state.cpu(), x.state)
    x = Linear([8], 2, 2, 64, 64, seed=14)
    with pytest.raises(ValueError, match="log_decay"):
        x.run(g=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError, match="state must be"):
        x.run(state=torch.zeros(2, 2, 64, 64, device="cuda"))
    with pytest.raises(w.W4A16Error, match="shape"):
        x.run(cu_seqlens=ints([0]), state=None)
    with pytest.raises(ValueError, match="shape mismatch"):
        x.run(k=x.k[1:].cuda())


# ---- one token per request -----------------------------------------------------------------------

@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("B,H,Hk,dtype,decay", [
    (1, 1, 1, torch.bfloat16, "token"), (1, 32, 32, torch.float16, "head"), (37, 6, 3, torch.float16, "token"),
    (130, 8, 1, torch.bfloat16, "head"),
])
def test_step(B, H, Hk, dtype, decay, Dk, Dv):
    x = Linear([1] * B, H, Hk, Dk, Dv, dtype, decay, seed=B + Dk)
    q, k, v, g, s = (t.cuda() for t in (x.q, x.k, x.v, x.g, x.state))
    new = torch.full_like(s, 9.0)
    out = w.linear_attention_step(q, k, v, g, s, state_out=new)
    assert torch.equal(s.cpu(), x.state)
    inplace = s.clone()
    again = w.linear_attention_step(q, k, v, g, inplace)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(new, inplace)
    for b in range(B):
        gb = (x.g[b] if decay == "token" else x.g).double()[None]
        o, S, mag, M = mo.linear(x.q[b:b + 1].double(), x.k[b:b + 1].double(), x.v[b:b + 1].double(), gb,
                                 x.state[b].double(), x.scale)
        tol, tol_s = mo.step_bounds(dtype, o[0], mag[0], M, Dk)
        assert bool(((out[b].cpu().double() - o[0]).abs() <= tol).all()), b
        assert bool(((new[b].cpu().double() - S).abs() <= tol_s).all()), b


def test_step_slots():
    x = Linear([1] * 6, 2, 2, 64, 64, seed=20)
    pool = torch.randn(9, 2, 64, 64, device="cuda")
    slots = [4, -1, 8, 0, 9, 2 ** 31 - 1]
    q, k, v, g = (t.cuda() for t in (x.q, x.k, x.v, x.g))
    got = pool.clone()
    out = w.linear_attention_step(q, k, v, g, got, slots=ints(slots))
    dense = torch.zeros(6, 2, 64, 64, device="cuda")
    for b, s in enumerate(slots):
        if 0 <= s < 9:
            dense[b] = pool[s]
    want = w.linear_attention_step(q, k, v, g, dense)
    torch.cuda.synchronize()
    for b, s in enumerate(slots):
        if 0 <= s < 9:
            assert torch.equal(got[s], dense[b]) and torch.equal(out[b], want[b])
        else:
            assert bool((out[b] == 0).all())
    for s in (1, 2, 3, 5, 6, 7):
        assert torch.equal(got[s], pool[s])


def test_step_continues_a_prompt_on_another_stream_with_strides():
    x = Linear([60], 2, 2, 128, 64, torch.float16, seed=21)
    q, k, v, g, s = (t.cuda() for t in (x.q, x.k, x.v, x.g, x.state))
    _, state = w.linear_attention(q[:57], k[:57], v[:57], g[:57], state=s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    room = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda")
    for t in range(57, 60):
        out = w.linear_attention_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], state, out=room[:, ::2],
                                      stream=side)
    torch.cuda.synchronize()
    o, S, mag, M = mo.linear(x.q.double(), x.k.double(), x.v.double(), x.g.double(), x.state[0].double(), x.scale)
    tol, tol_s = mo.linear_bounds(torch.float16, o[-1], mag[-1], M, 60)
    assert bool(((out[0].cpu().double() - o[-1]).abs() <= tol).all())
    assert bool(((state[0].cpu().double() - S).abs() <= tol_s).all())


def test_step_resets_and_empty():
    x = Linear([1] * 3, 2, 2, 64, 64, seed=22)
    x.g[1] = -math.inf
    q, k, v, g, s = (t.cuda() for t in (x.q, x.k, x.v, x.g, x.state))
    w.linear_attention_step(q, k, v, g, s)
    want = x.k[1].double()[:, :, None] * x.v[1].double()[:, None, :]
    assert float((s[1].cpu().double() - want).abs().max()) <= 2.0 ** -23 * float(want.abs().max())
    none = w.linear_attention_step(q[:0], k[:0], v[:0], g[:0], s[:0])
    assert none.shape == (0, 2, 64)


@pytest.mark.parametrize("n", [1, 70, 130])
def test_rows_that_share_memory(n):
    x = Linear([n], 4, 2, 128, 64, seed=n + 900)
    x.q, x.k, x.v = (t[:1].expand(n, -1, -1) for t in (x.q, x.k, x.v))
    kw = {name: getattr(x, name)[:1].cuda().expand(n, -1, -1) for name in "qkv"}
    assert n == 1 or kw["k"].stride(0) == 0
    x.check(*x.run(**kw))


@pytest.mark.parametrize("stride", [0, 8, 64])
def test_one_token_of_any_stride(stride):
    x = Linear([1], 3, 3, 64, 128, dtype=torch.float16, seed=stride + 950)
    kw = {name: getattr(x, name).cuda() for name in "qkv"}
    kw = {name: t.as_strided(t.shape, (stride,) + t.stride()[1:]) for name, t in kw.items()}
    buf = torch.full((4, 3, 128), 7.0, dtype=torch.float16, device="cuda")
    out = buf[:1].as_strided((1, 3, 128), (stride, 128, 1))
    o, state = x.run(out=out, **kw)
    x.check(o, state)
    assert bool((buf[1:] == 7.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_infinite_state_entry_beside_large_ones(dtype):
    x = Linear([100], 2, 2, 128, 128, dtype=dtype, seed=77)
    x.state *= 3e5   # past float16's range
    state = x.state.clone()
    state[0, :, 3, 5] = math.inf
    out, end = x.run(state=state.cuda())
    assert not bool(torch.isfinite(out[:, :, 5]).any())
    assert not bool(torch.isfinite(end[0, :, 3, 5]).any())
    out[:, :, 5] = 0
    x.v[:, :, 5] = 0   # the column apart, all as without it
    x.state[0, :, :, 5] = 0
    end[0, :, :, 5] = 0
    # what rounds past the type's largest value is an infinity of its sign
    want = mo.linear(x.q.double(), x.k.double(), x.v.double(), x.g.double(), x.state[0].double(), x.scale)[0]
    top = torch.finfo(dtype).max
    out = out.cpu().double()
    over = out.isinf() & (want.abs() * (1 + 2 * mo.half_step(dtype)) > top) & (out.sign() == want.sign())
    assert not bool((~over & (want.abs() * (1 - 2 * mo.half_step(dtype)) > top)).any())
    x.check(torch.where(over, want, out), end)


def test_offsets_past_32_bits():
    n, ld = 130, 2 ** 24 - 8   # the longest strides: a chunk's rows lie up to 2^31 bytes apart
    x = Linear([n], 2, 1, 128, 64, seed=990)

    def far(t, dtype):
        big = torch.empty((n - 1) * ld + t[0].numel(), dtype=dtype, device="cuda")
        return big.as_strided(t.shape, (ld,) + t.stride()[1:])

    kw = {}
    for name in "qkvg":
        t = getattr(x, name)
        kw[name] = far(t, t.dtype)
        kw[name].copy_(t)
    out = far(x.v, x.dtype)
    x.check(*x.run(out=out, **kw))
