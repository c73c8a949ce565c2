"""The delta rule and the 8-bit cache without a GPU: oracles on cases worked out by hand or by another route, the
refusals of the C entries (nothing is enqueued) and of the Python binding."""
import ctypes
import math

import pytest
import torch

import delta_oracle as do
import quantized_oracle as qo
import weight_only_int4_w4a16_amd as w
from weight_only_int4_w4a16_amd import mixers, quantized

OK, NULLP, SHAPE, GROUP, ALIGN, DEVICE, LAUNCH, TYPE, WORK = range(9)
A = 0x10000          # a fake, 16-byte aligned address: validation never dereferences it


# ---- the oracles ---------------------------------------------------------------------------------

def test_delta_overwrites_what_a_key_held():
    # one orthonormal key per token and beta 1: the state holds each key's last value
    k = torch.eye(3, dtype=torch.float64)[[0, 1, 0]][:, None]
    v = torch.arange(6, dtype=torch.float64).reshape(3, 1, 2)
    z, one = torch.zeros(3, 1, dtype=torch.float64), torch.ones(3, 1, dtype=torch.float64)
    out, S, u, _ = do.delta(k, k, v, z, one, torch.zeros(1, 3, 2, dtype=torch.float64), 1.0)
    assert torch.equal(out, v)
    assert torch.equal(S[0], torch.tensor([[4.0, 5.0], [2.0, 3.0], [0.0, 0.0]], dtype=torch.float64))
    assert torch.equal(u[2, 0], v[2, 0] - v[0, 0])


def test_delta_without_overlap_is_linear_attention():
    import mixer_oracle as mo
    torch.manual_seed(1)
    q = torch.randn(4, 1, 8, dtype=torch.float64)
    k = torch.linalg.qr(torch.randn(8, 8, dtype=torch.float64))[0][:4, None]
    v, g = torch.randn(4, 2, 5, dtype=torch.float64), -torch.rand(4, 2, dtype=torch.float64)
    z = torch.zeros(2, 8, 5, dtype=torch.float64)
    out, S, _, _ = do.delta(q, k, v, g, torch.ones(4, 2, dtype=torch.float64), z, 0.3)
    want, S2, _, _ = mo.linear(q, k, v, g, z, 0.3)
    assert torch.allclose(out, want) and torch.allclose(S, S2)


def test_codes_by_hand():
    assert qo.to_codes(torch.tensor([0.5, 1.5, -2.5, 126.6, 300.0]).double(), torch.int8).tolist() == [0, 2, -2, 127, 127]
    x = torch.tensor([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 460.0]).double()   # ties between e4m3 values
    assert qo.to_codes(x, torch.float8_e4m3fn).float().tolist() == [16.0, 20.0, 0.0, 2.0 ** -8, 448.0]


@pytest.mark.parametrize("kind", [torch.int8, torch.float8_e4m3fn])
def test_write_oracle_grows_a_scale(kind):
    codes, scale = torch.zeros(1, 16, 1, 4).to(kind), torch.full((1, 1, 1), 9.0)
    x = torch.tensor([[[1.0, -0.5, 0.25, 0.0]], [[4.0, 0.0, 0.0, 2.0]]])
    qo.write(x[:1], codes, scale, [0])
    assert float(scale) == float(torch.tensor(1.0 / qo.LARGEST[kind])) and codes[0, 0, 0, 0].float() == qo.LARGEST[kind]
    qo.write(x[1:], codes, scale, [1])
    assert codes[0, 0, 0].float().tolist()[:2] == ([32.0, -16.0] if kind == torch.int8 else [112.0, -56.0])
    got = qo.read(codes, scale, [0, 1, -1, 16], torch.bfloat16)
    assert (got[:2] - x).abs().max() <= 4.0 / 127 and not got[2:].any()


# ---- refusals of the C entries -------------------------------------------------------------------

def lib():
    return mixers._library()


def cache(k=A, v=A, ks=(8192, 128, 2048), vs=(8192, 128, 2048), kscale=A, vscale=A, kss=(4, 4, 1), vss=(4, 4, 1), pages=10,
          page=32, heads=4, dim=128, block=16, type=3):
    s = mixers._Strides
    return quantized._Cache(k, v, s(*ks), s(*vs), kscale, vscale, s(*kss), s(*vss), pages, page, heads, dim, block, type)


BAD_CACHES = [
    (dict(k=None), NULLP), (dict(v=None), NULLP), (dict(kscale=None), NULLP), (dict(vscale=None), NULLP),
    (dict(type=0), TYPE), (dict(type=1), TYPE), (dict(type=4), TYPE), (dict(pages=0), SHAPE), (dict(page=0), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=65536), SHAPE), (dict(pages=1 << 20, page=4096), SHAPE), (dict(block=0), SHAPE),
    (dict(block=8), SHAPE), (dict(block=24), SHAPE), (dict(block=80, page=160), SHAPE), (dict(block=48), SHAPE),
    (dict(dim=80), SHAPE), (dict(dim=0), SHAPE), (dict(ks=(8192, 1 << 24, 2048)), SHAPE),
    (dict(vs=(8192, -128, 2048)), SHAPE), (dict(ks=(8200, 128, 2048)), ALIGN), (dict(vs=(8192, 128, 2056)), ALIGN),
    (dict(k=A + 8), ALIGN), (dict(vscale=A + 2), ALIGN),
]


def write(c=None, k=A, ldk=512, hsk=128, v=A, ldv=512, hsv=128, T=5, type=0, slots=A):
    c = cache() if c is None else c
    return lib().w4a16_quantized_kv_write(k, ldk, hsk, v, ldv, hsv, T, type, slots, ctypes.addressof(c), None)


def read(c=None, k=A, ldk=512, hsk=128, v=A, ldv=512, hsv=128, T=5, type=0, slots=A):
    c = cache() if c is None else c
    return lib().w4a16_quantized_kv_read(ctypes.addressof(c), slots, T, type, k, ldk, hsk, v, ldv, hsv, None)


def attend(c=None, q=A, ldq=1024, hsq=128, type=0, table=A, stride=8, pages=8, lens=A, B=3, Hq=8, scale=0.1, window=0,
           out=A, ldo=1024, hso=128, lse=None, work=A, room=1 << 40):
    c = cache() if c is None else c
    return lib().w4a16_quantized_attention(q, ldq, hsq, type, ctypes.addressof(c), table, stride, pages, lens, B, Hq, scale,
                                           window, out, ldo, hso, lse, work, room, None)


@pytest.mark.parametrize("call", [write, read, attend])
@pytest.mark.parametrize("kw,status", BAD_CACHES + [(dict(), DEVICE), (dict(type=2), DEVICE), (dict(block=32), DEVICE),
                                                    (dict(block=48, page=144), DEVICE)])
def test_caches(call, kw, status):
    assert call(cache(**kw)) == status


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), NULLP), (dict(v=None), NULLP), (dict(slots=None), NULLP), (dict(type=2), TYPE), (dict(type=3), TYPE),
    (dict(T=-1), SHAPE), (dict(k=A + 2), ALIGN), (dict(ldk=516), ALIGN), (dict(hsv=12), ALIGN), (dict(slots=A + 2), ALIGN),
    (dict(T=0, k=None, v=None, slots=None), DEVICE), (dict(T=2 ** 31 - 1), DEVICE),
    (dict(c=cache(heads=17), T=2 ** 31 - 1), SHAPE),
])
def test_rows(call, kw, status):
    assert call(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), NULLP), (dict(table=None), NULLP), (dict(lens=None), NULLP), (dict(out=None), NULLP),
    (dict(work=None), NULLP), (dict(type=3), TYPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(Hq=0), SHAPE),
    (dict(Hq=6), SHAPE), (dict(pages=0), SHAPE), (dict(stride=7), SHAPE), (dict(pages=1 << 28, stride=1 << 28), SHAPE),
    (dict(window=-1), SHAPE), (dict(scale=math.inf), SHAPE), (dict(q=A + 8), ALIGN), (dict(out=A + 4), ALIGN),
    (dict(ldq=1028), ALIGN), (dict(hso=4), ALIGN), (dict(lse=A + 2), ALIGN), (dict(work=A + 8), ALIGN),
    (dict(lens=A + 2), ALIGN), (dict(room=0), WORK),
])
def test_attention(kw, status):
    assert attend(**kw) == status


def delta(q=A, ldq=256, hsq=128, k=A, ldk=256, hsk=128, v=A, ldv=256, hsv=128, g=A, ldg=2, hsg=1, beta=A, ldb=2, hsb=1,
          cu=A, seqs=3, T=50, Hk=2, H=2, Dk=128, Dv=128, type=0, scale=1.0, s0=A, s1=A, out=A, ldo=256, hso=128, work=A,
          room=1 << 40):
    return lib().w4a16_delta_rule(q, ldq, hsq, k, ldk, hsk, v, ldv, hsv, g, ldg, hsg, beta, ldb, hsb, cu, seqs, T, Hk, H,
                                  Dk, Dv, type, scale, s0, s1, out, ldo, hso, work, room, None)


def step(q=A, ldq=256, hsq=128, k=A, ldk=256, hsk=128, v=A, ldv=256, hsv=128, g=A, ldg=2, hsg=1, beta=A, ldb=2, hsb=1,
         slots=A, states=9, B=5, Hk=2, H=2, Dk=128, Dv=128, type=0, scale=1.0, s0=A, s1=A, out=A, ldo=256, hso=128):
    return lib().w4a16_delta_rule_step(q, ldq, hsq, k, ldk, hsk, v, ldv, hsv, g, ldg, hsg, beta, ldb, hsb, slots, states, B,
                                       Hk, H, Dk, Dv, type, scale, s0, s1, out, ldo, hso, None)


SHARED = [
    (dict(q=None), NULLP), (dict(k=None), NULLP), (dict(v=None), NULLP), (dict(g=None), NULLP), (dict(beta=None), NULLP),
    (dict(out=None), NULLP), (dict(s1=None), NULLP), (dict(type=2), TYPE), (dict(type=5), TYPE), (dict(Hk=0), SHAPE),
    (dict(Hk=2, H=3), SHAPE), (dict(H=0), SHAPE), (dict(Dk=96), SHAPE), (dict(Dv=32), SHAPE), (dict(scale=math.nan), SHAPE),
    (dict(ldq=1 << 24), SHAPE), (dict(ldb=1 << 24), SHAPE), (dict(ldb=-2), SHAPE), (dict(ldv=-256), SHAPE),
    (dict(q=A + 8), ALIGN), (dict(ldk=260), ALIGN), (dict(hsv=4), ALIGN), (dict(g=A + 2), ALIGN), (dict(beta=A + 2), ALIGN),
    (dict(s0=A + 4), ALIGN), (dict(s1=A + 8), ALIGN), (dict(ldo=258), ALIGN), (dict(), DEVICE),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(seqs=0), SHAPE), (dict(seqs=16385), SHAPE), (dict(T=-1), SHAPE), (dict(cu=None), SHAPE),
    (dict(seqs=16384, H=8192, Hk=1), SHAPE), (dict(cu=None, seqs=1), DEVICE), (dict(s0=None), DEVICE),
    (dict(cu=A + 2), ALIGN), (dict(work=A + 8), ALIGN), (dict(room=0), WORK), (dict(work=None), NULLP),
])
def test_delta(kw, status):
    assert delta(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(s0=None), NULLP), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(states=-1), SHAPE),
    (dict(slots=None, states=4), SHAPE), (dict(slots=None), DEVICE), (dict(slots=A + 2), ALIGN),
])
def test_step(kw, status):
    assert step(**kw) == status


def test_workspaces():
    f = lib().w4a16_delta_rule_workspace
    sizes = [f(T, 3, 4, 128, 64, 0) for T in (0, 1, 63, 64, 65, 100, 1000, 100000)]
    assert sizes == sorted(sizes) and sizes[0] >= 0
    assert f(100, 4, 4, 128, 64, 0) >= f(100, 3, 4, 128, 64, 0)
    assert f(-1, 1, 4, 128, 64, 0) == f(5, 1, 4, 96, 64, 0) == f(5, 0, 4, 128, 64, 0) == f(5, 1, 4, 128, 64, 2) == -1
    g = lib().w4a16_quantized_attention_workspace
    assert g(32, 8, 128) > 0 and g(33, 8, 128) == 0 and g(32, 8, 100) == 0


# ---- refusals of the binding ---------------------------------------------------------------------

def test_binding_refuses():
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(1, 16, 2, 64, dtype=torch.int8)
    s = torch.ones(1, 1, 2)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        w.quantized_kv_write(x, x, c, c, s, s, i)
    with pytest.raises(ValueError, match="GPU"):
        w.quantized_kv_read(c, c, s, s, i)
    with pytest.raises(TypeError, match="slot_map"):
        w.quantized_kv_read(c, c, s, s, i.long())
    with pytest.raises(TypeError, match="q must be"):
        w.quantized_attention(x.float(), c, c, s, s, i[None], i)
    with pytest.raises(TypeError, match="torch.Tensor"):
        w.delta_rule(None, x, x, i.float(), i.float())
    with pytest.raises(ValueError, match="GPU"):
        w.delta_rule_step(x, x, x, i.float(), i.float(), torch.zeros(2, 2, 64, 64))
    with pytest.raises(ValueError, match="fit 32 bits"):
        w.quantized_attention(x, c, c, s, s, i[None], i, window=2 ** 33)


def test_short_way_declines():
    mixers._library()
    b = mixers._binding
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(1, 16, 2, 64, dtype=torch.int8)
    s, f = torch.ones(1, 1, 2), torch.zeros(2)
    i, work = torch.zeros(2, dtype=torch.int32), torch.zeros(16, dtype=torch.uint8)
    assert b.quantized_kv_write(x, x, c, c, s, s, i) == -1
    assert b.quantized_kv_read(c, c, s, s, i, x, x) == -1
    assert b.quantized_attention(x, c, c, s, s, i[None], i, 1.0, 0, x, None, work) == -1
    assert b.quantized_attention(x, c, c, None, None, i[None], i, 1.0, 0, x, None, work) == -1
    assert b.delta_rule(x, x, x, f, f, None, None, x, 1.0, x, work) == -1
    assert b.delta_rule(x, x, x, f, None, None, None, x, 1.0, x, work) == -1
    assert b.delta_rule_step(x, x, x, f, f, x, None, x, 1.0, x) == -1
    assert b.delta_rule_step() == -1 and b.quantized_kv_read(c) == -1
    with pytest.raises(TypeError):
        b.bind_more(1, 2)
    with pytest.raises(ValueError):
        b.bind_more(0, 1, 2, 3, 4)


def test_workspace_is_as_large_as_said():
    f = lib().w4a16_delta_rule_workspace
    for dtype in (0, 1):
        assert f(64, 1, 1, 128, 128, dtype) == f(1, 1, 1, 64, 64, dtype) == 31360
        assert f(131072, 1, 32, 128, 128, dtype) == 2048 * 32 * 31360
        assert f(1000, 7, 4, 128, 64, dtype) <= (-(-1000 // 64) + 7) * 4 * 31360
