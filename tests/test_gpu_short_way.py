"""The C++ way into the library against the Python one: the same results, the same refusals."""
import pytest
import torch

import weight_only_int4_w4a16_amd as w
from weight_only_int4_w4a16_amd import mixers

pytestmark = pytest.mark.gpu


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def rand(*shape, dtype=torch.bfloat16):
    return torch.randn(shape, device="cuda").to(dtype)


class Declined:
    """A binding that declines everything."""

    def __getattr__(self, name):
        return lambda *a: -1


def both_ways(call, *written):
    """call() by both ways: its outcome (an exception's type and text) and what it wrote are the same."""
    mixers._library()
    kept, found = mixers._binding, []
    start = [t.clone() for t in written]
    for binding in (kept, Declined()):
        for t, s in zip(written, start):
            t.copy_(s)
        mixers._binding = binding
        try:
            call()
            outcome = None
        except Exception as e:
            outcome = (type(e), str(e))
        finally:
            mixers._binding = kept
        torch.cuda.synchronize()
        found.append((outcome, [t.clone() for t in written]))
    assert found[0][0] == found[1][0]
    for a, b in zip(found[0][1], found[1][1]):
        assert torch.equal(a, b)
    return found[0][0]


def changed(base, kw):
    args = dict(base)
    args.update(kw)
    return args


def check(function, base, written, cases):
    assert both_ways(lambda: function(**base), *written) is None
    for kw, kind in cases:
        got = both_ways(lambda: function(**changed(base, kw)), *written)
        assert (got is None) if kind is None else (got is not None and issubclass(got[0], kind)), (kw.keys(), got)


def test_page_tables_both_ways():
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    out = w.page_tables_buffers(3, 20)
    base = dict(ctx_lens=ints([0, 0, 0]), new_lens=ints([5, 7, 2]), page_table=table, free_pages=ints([3, 1, 2, 0]),
                page_size=4, out=out)
    check(w.page_tables, base, (table, *out), [
        (dict(page_size=0), w.W4A16Error), (dict(page_size=-1), w.W4A16Error), (dict(ctx_lens=ints([0, 0])), ValueError),
        (dict(new_lens=torch.zeros(3, device="cuda")), TypeError), (dict(free_pages=ints([1, 2, 3, 4])[::2]), ValueError),
        (dict(page_table=table.t().contiguous().t()), ValueError), (dict(out=out._replace(counts=ints([1]))), ValueError),
        (dict(out=out._replace(positions=ints([1]))), ValueError), (dict(free_pages=ints([])), None),
        (dict(page_size=None), TypeError), (dict(page_table=table.cpu()), ValueError), (dict(max_tokens=19), ValueError),
        (dict(page_table=table[:, :3]), None),
    ])


@pytest.mark.parametrize("fp8", [False, True])
def test_kv_write_both_ways(fp8):
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kc, vc = (torch.zeros(4, 16, 2, 64, device="cuda").to(kind) for _ in range(2))
    raw = [t.view(torch.uint8) for t in (kc, vc)]
    scales = dict(k_scale=torch.ones(2, device="cuda"), v_scale=torch.full((2,), 0.5, device="cuda")) if fp8 else {}
    base = dict(k=rand(5, 2, 64), v=rand(5, 2, 64), k_cache=kc, v_cache=vc, slot_map=ints([0, 17, -1, 63, 64]), **scales)
    check(w.paged_kv_write, base, raw, [
        (dict(k=rand(4, 2, 64)), ValueError), (dict(v=rand(5, 2, 64, dtype=torch.float16)), TypeError),
        (dict(k=rand(5, 64, 2).transpose(1, 2)), ValueError), (dict(slot_map=ints([1, 2])), ValueError),
        (dict(slot_map=torch.zeros(5, device="cuda")), TypeError), (dict(v_cache=vc[1:]), ValueError),
        (dict(k_scale=torch.ones(3, device="cuda")), ValueError), (dict(k=rand(5, 3, 64)[:, 1:]), None),
        (dict(k=rand(5, 2, 68)[..., :64]), w.W4A16Error), (dict(k_scale=None), None),
        (dict(k=base["k"].cpu()), ValueError),
    ])


def test_linear_attention_both_ways():
    T, H, D = 200, 2, 64
    q, k, v = rand(T, 1, D), rand(T, 1, D), rand(T, H, D)
    out, state, end = torch.empty_like(v), torch.randn(2, H, D, D, device="cuda"), torch.zeros(2, H, D, D, device="cuda")
    base = dict(q=q, k=k, v=v, log_decay=-torch.rand(T, H, device="cuda"), cu_seqlens=ints([0, 150, 200]), state=state,
                state_out=end, out=out, workspace=w.linear_attention_workspace(q, v, 2))
    check(w.linear_attention, base, (out, end), [
        (dict(log_decay=-torch.rand(H, device="cuda")), None), (dict(state=None), None), (dict(scale=2.0), None),
        (dict(scale=2), None), (dict(scale=float("nan")), w.W4A16Error), (dict(scale="1"), Exception),
        (dict(log_decay=torch.zeros(T, device="cuda")), ValueError), (dict(cu_seqlens=ints([0, 200])), ValueError),
        (dict(cu_seqlens=None), ValueError), (dict(state=state[:, :1]), ValueError), (dict(k=rand(T, 2, D)), ValueError),
        (dict(state_out=end.double()), TypeError), (dict(out=out[:5]), ValueError), (dict(v=rand(T, 3, D)), ValueError),
        (dict(q=rand(T, 1, 32), k=rand(T, 1, 32)), ValueError), (dict(cu_seqlens=ints([])), Exception),
        (dict(q=rand(T, 1, D, dtype=torch.float16)), TypeError), (dict(q=None), TypeError),
    ])


def test_linear_attention_step_both_ways():
    B, H, D = 3, 2, 64
    q, k, v = rand(B, 1, D), rand(B, 1, D), rand(B, H, D)
    state, out = torch.randn(5, H, D, D, device="cuda"), rand(B, H, D)
    base = dict(q=q, k=k, v=v, log_decay=-torch.rand(B, H, device="cuda"), state=state, slots=ints([4, 0, -1]), out=out)
    check(w.linear_attention_step, base, (out, state), [
        (dict(slots=None), None), (dict(slots=ints([1])), ValueError), (dict(state=state[:2], slots=None), w.W4A16Error),
        (dict(state_out=state[:3]), ValueError), (dict(state=state.half()), TypeError), (dict(out=out[:, :1]), ValueError),
        (dict(slots=torch.zeros(3, device="cuda")), TypeError), (dict(state=state[0]), ValueError),
        (dict(log_decay=torch.zeros(B, 3, device="cuda")), ValueError), (dict(v=rand(B, 3, D)), ValueError),
        (dict(k=rand(B, 2, D)), ValueError), (dict(scale=float("inf")), w.W4A16Error),
    ])
