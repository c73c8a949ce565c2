"""Values that are not finite in the delta rule: NaN in what they reach, in both forms alike."""
import math

import pytest
import torch

import weight_only_int4_w4a16_amd as w
from test_gpu_delta_rule import BF, DIMS, FP, Delta, ints

pytestmark = pytest.mark.gpu

BAD = [math.nan, math.inf, -math.inf]


def put(x, what, token, bad):
    """Head 1's operand of a token; False where that is a value the operand may have."""
    if what == "v":
        x.v[token, 1, 5] = bad
    elif what == "k":
        x.k[token, 1, 3] = bad
    elif what == "beta":
        x.beta[token, 1] = bad
    else:
        x.g[token, 1] = bad
        return bad != -math.inf
    return True


def reached(what, width):
    """Columns of head 1 that become NaN, and those that do not."""
    columns = [5] if what == "v" else list(range(width))
    return columns, [i for i in range(width) if i not in columns]


@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B", [7, 70])                       # slices of a state, whole ones
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("what", ["v", "k", "beta", "decay"])
def test_step(Dk, Dv, dtype, B, bad, what):
    x = Delta([B], 2, 2, Dk, Dv, dtype, seed=3, rate=1.0)
    x.k[4, 1, 7:20] = 0                                      # an infinity times these is no infinity
    state = torch.randn(B, 2, Dk, Dv, generator=torch.Generator().manual_seed(4))
    state[4, 1, :, 9] = 0

    def run():
        s = state.cuda()
        return w.delta_rule_step(*[t.cuda() for t in (x.q, x.k, x.v, x.g, x.beta)], s), s

    out, after = run()
    is_bad = put(x, what, 4, bad)
    out2, after2 = run()
    columns, rest = reached(what, Dv)
    if is_bad:
        assert bool(out2[4, 1, columns].isnan().all()) and bool(after2[4, 1][:, columns].isnan().all())
    else:                                                    # a decay of -inf clears the state
        state[4, 1], x.g[4, 1] = 0, 0
        want, states = run()
        assert torch.equal(out2[4, 1], want[4, 1]) and torch.equal(after2[4, 1], states[4, 1])
    assert torch.equal(out2[4, 1, rest], out[4, 1, rest]) and torch.equal(after2[4, 1][:, rest], after[4, 1][:, rest])
    others = [b for b in range(B) if b != 4]
    assert torch.equal(out2[others], out[others]) and torch.equal(after2[others], after[others])
    assert torch.equal(out2[4, 0], out[4, 0]) and torch.equal(after2[4, 0], after[4, 0])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("what", ["v", "k", "beta", "decay"])
@pytest.mark.parametrize("at", [0, 63, 64, 99])
def test_packed_and_tokens_in_turn(dtype, bad, what, at):
    """The packed form and the single-token form, token after token, have NaN in the same places."""
    x = Delta([100], 2, 2, 64, 64, dtype, seed=5)
    is_bad = put(x, what, at, bad)
    out, state = x.run()
    s, rows = x.state.cuda(), []
    dev = [t.cuda() for t in (x.q, x.k, x.v, x.g, x.beta)]
    for t in range(x.T):
        rows.append(w.delta_rule_step(*[d[t:t + 1] for d in dev], s))
    turn = torch.cat(rows)
    assert torch.equal(out.isnan(), turn.isnan()) and torch.equal(state.isnan(), s.isnan())
    assert bool(torch.isfinite(out[~out.isnan()]).all()) and bool(torch.isfinite(turn[~turn.isnan()]).all())
    columns, rest = reached(what, 64)
    assert bool(out[at:, 1, columns].isnan().all()) == is_bad and bool(state[0, 1][:, columns].isnan().all()) == is_bad
    assert not bool(out[:at].isnan().any()) and not bool(out[:, 0].isnan().any()) and not bool(out[:, 1][:, rest].isnan().any() and is_bad)


def test_slots_keep_what_is_not_finite_to_themselves():
    x = Delta([3], 2, 2, 64, 64, seed=6)
    x.v[1] = math.inf
    pool = torch.randn(5, 2, 64, 64, generator=torch.Generator().manual_seed(7)).cuda()
    before = pool.clone()
    out = w.delta_rule_step(*[t.cuda() for t in (x.q, x.k, x.v, x.g, x.beta)], pool, slots=ints([4, 1, 9]))
    assert bool(pool[1].isnan().all()) and bool(out[1].isnan().all())
    assert bool(torch.isfinite(pool[4]).all()) and bool(torch.isfinite(out[0]).all()) and not bool(out[2].any())
    assert torch.equal(pool[[0, 2, 3]], before[[0, 2, 3]])
