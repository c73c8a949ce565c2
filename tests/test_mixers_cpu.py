"""The token mixers without a GPU: the oracle on cases worked out by hand or by another route, the
refusals of the C entries (nothing is enqueued) and of the Python binding."""
import ctypes
import math

import pytest
import torch

import mixer_oracle as mo
import weight_only_int4_w4a16_amd as w
from weight_only_int4_w4a16_amd import mixers

OK, NULLP, SHAPE, GROUP, ALIGN, DEVICE, LAUNCH, TYPE, WORK = range(9)
A = 0x10000          # a fake, 16-byte aligned address: validation never dereferences it


# ---- the oracle ----------------------------------------------------------------------------------

def test_page_tables_by_hand():
    table = [[7, -1, -1], [3, 4, -1], [-1, -1, -1]]
    seq, cu, slots, pos, counts, got = mo.page_tables([3, 8, 0], [2, 1, 0], table, [9, 5, 6], 4, 5)
    assert seq == [5, 9, 0] and cu == [0, 2, 3, 3] and counts == [3, 2]
    assert got == [[7, 9, -1], [3, 4, 5], [-1, -1, -1]]
    assert pos == [3, 4, 8, -1, -1] and slots == [7 * 4 + 3, 9 * 4, 5 * 4, -1, -1]


def test_page_tables_short_list_and_full_row():
    # two pages wanted and one left; a row of one page cannot hold position 4
    seq, cu, slots, pos, counts, got = mo.page_tables([0, 4], [5, 1], [[-1, -1], [2, 0]], [8], 4, 6)
    assert got == [[8, -1], [2, -1]] and counts == [6, 3]
    assert slots == [32, 33, 34, 35, -1, -1] and pos == [0, 1, 2, 3, 4, 4]


def test_attention_oracle_against_uniform_and_one_hot():
    v = torch.arange(12, dtype=torch.float64).reshape(3, 1, 4)
    out, lse, _, _, _ = mo.attention(torch.zeros(2, 4).double(), torch.randn(3, 1, 4).double(), v, 1.0)
    assert torch.allclose(out, v.mean(0).expand(2, 4)) and torch.allclose(lse, torch.full((2,), math.log(3.0)).double())
    k = torch.zeros(3, 1, 4).double()
    k[1, 0, 0] = 100.0
    out, _, _, _, _ = mo.attention(torch.ones(2, 4).double(), k, v, 1.0)
    assert torch.allclose(out, v[1].expand(2, 4))


def test_linear_oracle_against_the_quadratic_form():
    torch.manual_seed(0)
    T, H, Dk, Dv = 9, 2, 3, 5
    q, k = torch.randn(2, T, 1, Dk, dtype=torch.float64)
    v, g = torch.randn(T, H, Dv, dtype=torch.float64), -torch.rand(T, H, dtype=torch.float64)
    S0 = torch.randn(H, Dk, Dv, dtype=torch.float64)
    out, S, mag, M = mo.linear(q, k, v, g, S0, 0.5)
    b = g.cumsum(0)
    for h in range(H):
        wgt = torch.exp(b[:, None, h] - b[None, :, h]).tril()
        want = (0.5 * (q[:, 0] @ k[:, 0].T) * wgt) @ v[:, h] + 0.5 * b[:, h].exp()[:, None] * (q[:, 0] @ S0[h])
        assert torch.allclose(out[:, h], want)
    assert (mag >= out.abs() - 1e-12).all() and (M >= S.abs() - 1e-12).all()


# ---- refusals of the C entries -------------------------------------------------------------------

def lib():
    return mixers._library()


def tables(ctx=A, new=A, B=4, table=A, stride=8, pages=8, free=A, nfree=4, page=16, T=32, seq=A, cu=A, slots=A,
           pos=A, counts=A):
    return lib().w4a16_page_tables(ctx, new, B, table, stride, pages, free, nfree, page, T, seq, cu, slots, pos,
                                   counts, None)


@pytest.mark.parametrize("kw,status", [
    (dict(ctx=None), NULLP), (dict(new=None), NULLP), (dict(table=None), NULLP), (dict(free=None), NULLP),
    (dict(seq=None), NULLP), (dict(cu=None), NULLP), (dict(slots=None), NULLP), (dict(pos=None), NULLP),
    (dict(counts=None), NULLP), (dict(B=0), SHAPE), (dict(B=16385), SHAPE), (dict(stride=7), SHAPE),
    (dict(pages=0), SHAPE), (dict(nfree=-1), SHAPE), (dict(page=0), SHAPE), (dict(page=65537), SHAPE),
    (dict(T=-1), SHAPE), (dict(ctx=A + 2), ALIGN), (dict(slots=A + 1), ALIGN), (dict(), DEVICE),
    (dict(free=None, nfree=0), DEVICE), (dict(slots=None, pos=None, T=0), DEVICE),
])
def test_page_tables_validation(kw, status):
    assert tables(**kw) == status


def cache(k=A, v=A, ks=(8192, 128, 2048), vs=(8192, 128, 2048), kscale=None, vscale=None, pages=10, page=16, heads=4,
          dim=128, type=0):
    return mixers._Cache(k, v, mixers._Strides(*ks), mixers._Strides(*vs), kscale, vscale, pages, page, heads, dim,
                         type)


BAD_CACHES = [
    (dict(k=None), NULLP), (dict(v=None), NULLP), (dict(type=1), TYPE), (dict(type=3), TYPE), (dict(pages=0), SHAPE),
    (dict(page=0), SHAPE), (dict(heads=0), SHAPE), (dict(pages=1 << 20, page=4096), SHAPE),
    (dict(ks=(8192, 132, 2048)), ALIGN), (dict(vs=(8192, 128, 2044)), ALIGN), (dict(k=A + 8), ALIGN),
    (dict(type=2, ks=(8200, 128, 2048)), ALIGN), (dict(type=2, kscale=A + 2), ALIGN),
]


def write(c=None, k=A, ldk=512, hsk=128, v=A, ldv=512, hsv=128, T=5, type=0, slots=A):
    c = cache() if c is None else c
    return lib().w4a16_paged_kv_write(k, ldk, hsk, v, ldv, hsv, T, type, slots, ctypes.addressof(c), None)


@pytest.mark.parametrize("kw,status", BAD_CACHES + [(dict(dim=8), SHAPE), (dict(dim=1040), SHAPE), (dict(dim=72), SHAPE)])
def test_kv_write_refuses_caches(kw, status):
    assert write(cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), NULLP), (dict(v=None), NULLP), (dict(slots=None), NULLP), (dict(type=2), TYPE), (dict(type=-1), TYPE),
    (dict(T=-1), SHAPE), (dict(k=A + 2), ALIGN), (dict(ldk=516), ALIGN), (dict(hsv=12), ALIGN), (dict(slots=A + 2), ALIGN),
    (dict(), DEVICE),
])
def test_kv_write_validation(kw, status):
    assert write(**kw) == status


def attend(c=None, q=A, ldq=1024, hsq=128, type=0, table=A, stride=8, pages=8, lens=A, B=3, Hq=8, scale=0.1, window=0,
           out=A, ldo=1024, hso=128, lse=None, work=A, room=1 << 40):
    c = cache() if c is None else c
    return lib().w4a16_paged_attention(q, ldq, hsq, type, ctypes.addressof(c), table, stride, pages, lens, B, Hq, scale,
                                       window, out, ldo, hso, lse, work, room, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES + [(dict(dim=80), SHAPE), (dict(heads=3), SHAPE)])
def test_attention_refuses_caches(kw, status):
    assert attend(cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), NULLP), (dict(table=None), NULLP), (dict(lens=None), NULLP), (dict(out=None), NULLP),
    (dict(work=None), NULLP), (dict(type=2), TYPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(Hq=0), SHAPE),
    (dict(pages=0), SHAPE), (dict(stride=7), SHAPE), (dict(pages=1 << 28, stride=1 << 28), SHAPE), (dict(window=-1), SHAPE),
    (dict(scale=math.inf), SHAPE), (dict(scale=math.nan), SHAPE), (dict(q=A + 8), ALIGN), (dict(out=A + 4), ALIGN),
    (dict(ldq=1028), ALIGN), (dict(hso=4), ALIGN), (dict(lse=A + 2), ALIGN), (dict(work=A + 8), ALIGN),
    (dict(lens=A + 2), ALIGN), (dict(room=0), WORK), (dict(), DEVICE),
])
def test_attention_validation(kw, status):
    assert attend(**kw) == status


def test_attention_workspace_does_not_depend_on_the_batch():
    f = lib().w4a16_paged_attention_workspace
    assert f(32, 8, 128) > 0 and f(33, 8, 128) == 0 and f(32, 8, 100) == 0 and f(0, 1, 64) == 0


def linear(q=A, ldq=256, hsq=128, k=A, ldk=256, hsk=128, v=A, ldv=256, hsv=128, g=A, ldg=2, hsg=1, cu=A, seqs=3, T=50,
           Hk=2, H=2, Dk=128, Dv=128, type=0, scale=1.0, s0=A, s1=A, out=A, ldo=256, hso=128, work=A, room=1 << 40):
    return lib().w4a16_linear_attention(q, ldq, hsq, k, ldk, hsk, v, ldv, hsv, g, ldg, hsg, cu, seqs, T, Hk, H, Dk, Dv,
                                        type, scale, s0, s1, out, ldo, hso, work, room, None)


def step(q=A, ldq=256, hsq=128, k=A, ldk=256, hsk=128, v=A, ldv=256, hsv=128, g=A, ldg=2, hsg=1, slots=A, states=9, B=5,
         Hk=2, H=2, Dk=128, Dv=128, type=0, scale=1.0, s0=A, s1=A, out=A, ldo=256, hso=128):
    return lib().w4a16_linear_attention_step(q, ldq, hsq, k, ldk, hsk, v, ldv, hsv, g, ldg, hsg, slots, states, B, Hk, H,
                                             Dk, Dv, type, scale, s0, s1, out, ldo, hso, None)


SHARED = [
    (dict(q=None), NULLP), (dict(k=None), NULLP), (dict(v=None), NULLP), (dict(g=None), NULLP), (dict(out=None), NULLP),
    (dict(s1=None), NULLP), (dict(type=2), TYPE), (dict(type=5), TYPE), (dict(Hk=0), SHAPE), (dict(Hk=2, H=3), SHAPE),
    (dict(H=0), SHAPE), (dict(Dk=96), SHAPE), (dict(Dv=32), SHAPE), (dict(scale=math.nan), SHAPE), (dict(q=A + 8), ALIGN),
    (dict(ldk=260), ALIGN), (dict(hsv=4), ALIGN), (dict(g=A + 2), ALIGN), (dict(s0=A + 4), ALIGN), (dict(s1=A + 8), ALIGN),
    (dict(ldo=258), ALIGN), (dict(), DEVICE),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(seqs=0), SHAPE), (dict(seqs=16385), SHAPE), (dict(T=-1), SHAPE), (dict(cu=None), SHAPE),
    (dict(cu=None, seqs=1), DEVICE), (dict(s0=None), DEVICE), (dict(cu=A + 2), ALIGN), (dict(work=A + 8), ALIGN),
])
def test_linear_validation(kw, status):
    assert linear(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(s0=None), NULLP), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(states=-1), SHAPE),
    (dict(slots=None, states=4), SHAPE), (dict(slots=None), DEVICE), (dict(slots=A + 2), ALIGN),
])
def test_step_validation(kw, status):
    assert step(**kw) == status


def test_new_status_strings():
    assert w.status_string(TYPE) != w.status_string(99) != w.status_string(WORK)


# ---- refusals of the binding ---------------------------------------------------------------------

def test_binding_refuses_cpu_tensors_and_wrong_types():
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16)
    ints = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        w.paged_attention(q, c, c, ints[None], ints)
    with pytest.raises(TypeError, match="q must be"):
        w.paged_attention(q.float(), c, c, ints[None], ints)
    with pytest.raises(ValueError, match="3 dimensions"):
        w.paged_kv_write(q[0], q, c, c, ints)
    with pytest.raises(TypeError, match="torch.Tensor"):
        w.linear_attention(None, q, q, ints.float())
    with pytest.raises(TypeError, match="ctx_lens"):
        w.page_tables(ints.long(), ints, ints[None], ints, 16, max_tokens=4)


def test_short_way_declines_what_it_does_not_take():
    """The C++ part of the binding leaves everything but plain GPU calls to the Python code."""
    mixers._library()
    b = mixers._binding
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    work = torch.zeros(16, dtype=torch.uint8)
    assert b.page_tables(i, i, i[None], i, 16, i, i, i, i, i) == -1
    assert b.page_tables(i, i, i[None], i, "16", i, i, i, i, i) == -1
    assert b.paged_kv_write(x, x, c, c, None, None, i) == -1
    assert b.paged_attention(x, c, c, None, None, i[None], i, 1.0, 0, x, None, work) == -1
    assert b.paged_attention(None, c, c, None, None, i[None], i, None, 0, x, None, work) == -1
    assert b.linear_attention(x, x, x, i.float(), None, None, x, 1.0, x, work) == -1
    assert b.linear_attention_step(x, x, x, i.float(), x, None, x, 1.0, x) == -1
    assert b.paged_kv_write(x) == -1 and b.linear_attention_step() == -1
    with pytest.raises(TypeError):
        b.bind(1, 2)
    with pytest.raises(ValueError):
        b.bind(0, 1, 2, 3, 4)
