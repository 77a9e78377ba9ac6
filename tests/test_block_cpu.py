"""The norm, the choice of experts and rows in 8 bits without a GPU: sizes, and bad arguments refused before any HIP
call (pointer values are never dereferenced on these paths)."""
import ctypes
import math

import pytest
import torch

mvq = pytest.importorskip("bit_vector_quantised_amd")
import block_ref as ref  # noqa: E402
from bit_vector_quantised_amd import _lib  # noqa: E402
from bit_vector_quantised_amd.block import ExpertChoice, RmsNorm  # noqa: E402
from bit_vector_quantised_amd.dense import Rows8  # noqa: E402

A, B, C, D, F, G = (0x100000000 * i for i in range(1, 7))  # aligned addresses far apart
RAW = _lib.raw()


def r8(q=B, e=C):
    return ctypes.byref(_lib.Rows8Desc(q, e))


def test_pitch():
    assert [_lib.rows8_pitch(c) for c in (1, 31, 32, 33, 7168, 32768)] == [32, 32, 32, 64, 7168, 32768]
    assert [_lib.rows8_pitch(c) for c in (0, -1, 32769)] == [0, 0, 0]


BAD_ROWS = (dict(M=-1), dict(C=0), dict(C=32769), dict(dt=2), dict(x=None), dict(x=A + 8), dict(r=None), dict(r=r8(q=None)), dict(r=r8(e=None)),
            dict(r=r8(q=B + 8)), dict(M=2097152, C=8193), dict(gs=D + 2, n=4), dict(gs=D, n=0), dict(gs=D, n=1025),
            dict(x=B), dict(r=r8(q=A)), dict(x=C))


def test_rows8_refusals():
    def pack(x=A, dt=_lib.BF16, M=4, C=64, gs=None, n=0, r=r8()):
        return RAW.moe_vq_rows8_pack(x, dt, M, C, gs, n, r, None)

    def unpack(x=A, dt=_lib.BF16, M=4, C=64, gs=None, n=0, r=r8()):
        return RAW.moe_vq_rows8_unpack(r, M, C, gs, n, x, dt, None)

    for kw in BAD_ROWS:
        assert pack(**kw) == unpack(**kw) == _lib.EINVAL, kw
    assert pack(M=0, x=None) == unpack(M=0, r=None) == _lib.OK
    assert unpack(x=D, gs=D + 16, n=4) == pack(r=r8(q=D), gs=D + 16, n=4) == _lib.EINVAL  # the table is read meanwhile
    assert pack(r=r8(e=B + 16)) == _lib.EINVAL  # the scales inside the values

    def gather(r=r8(), T=4, k=2, C=64, pair=D, xs=A, dt=_lib.BF16):
        return RAW.moe_vq_gather_rows8(r, T, k, C, pair, xs, dt, None)

    for kw in (dict(T=-1), dict(T=65537), dict(k=0), dict(k=33), dict(C=0), dict(C=32769), dict(dt=5), dict(r=None), dict(r=r8(q=B + 4)),
               dict(pair=None), dict(pair=D + 2), dict(xs=None), dict(xs=A + 8), dict(xs=B), dict(xs=D)):
        assert gather(**kw) == _lib.EINVAL, kw
    assert gather(T=0, r=None) == _lib.OK


def test_act_backward_refusals():
    def call(z=r8(), act=_lib.ACT_SWIGLU, lim=0.0, T=4, k=2, N=64, pair=D, w=F, dy=A, ddt=_lib.BF16, dz=G, y=G + (1 << 20),
             dt=_lib.BF16, dw=G + (1 << 21)):
        return RAW.moe_vq_act_backward8(z, act, lim, T, k, N, pair, w, dy, ddt, dz, y, dt, dw, None)

    for kw in (dict(z=None), dict(z=r8(e=None)), dict(act=-1), dict(act=4), dict(lim=-1.0), dict(lim=math.inf), dict(lim=math.nan),
               dict(T=-1), dict(T=65537), dict(k=0), dict(k=33), dict(N=0), dict(N=16385), dict(pair=None), dict(pair=D + 1), dict(w=F + 2),
               dict(dy=None), dict(dy=A + 8), dict(ddt=3), dict(dz=G + 8), dict(y=G + 8), dict(dt=-1), dict(dw=G + 1),
               dict(dz=A), dict(y=G), dict(dw=D), dict(dz=B), dict(dw=F + 4), dict(y=F)):
        assert call(**kw) == _lib.EINVAL, kw
    assert call(T=0, z=None) == call(dz=None, y=None, dw=None) == _lib.OK


def test_linear_backward8_refusals():
    def lin(act=_lib.ACT_SWIGLU, **kw):
        return _lib.LinearDesc(kw.get("n_in", 64), kw.get("n_out", 32), 1, act, _lib.BF16, 0.0, D, None)

    assert _lib.linear_bytes8(lin(), 16) >= _lib.linear_bytes(lin(), 16, True) and _lib.linear_bytes8(lin(n_in=0), 16) == 0
    assert _lib.linear_bytes8(lin(), -1) == 0
    need = [_lib.linear_bytes8(lin(n_in=4096, n_out=512), m) for m in (1, 16, 17, 300, 2000, 5000, 40000)]
    assert need == sorted(need)

    def call(x=None, x8=r8(), z=None, z8=r8(B + (1 << 20), C + (1 << 20)), M=8, act=_lib.ACT_SWIGLU, dy=A, dx=F, dw=F + (1 << 20), db=None, ws=G, n=1 << 24):
        return RAW.moe_vq_linear_backward8(ctypes.byref(lin(act)), x, x8, M, None, z, z8, dy, _lib.BF16, dx, dw, db, ws, n, None)

    for kw in (dict(x=A), dict(z=A), dict(x8=None), dict(z8=None), dict(x8=r8(q=None)), dict(z8=r8(q=B + 8)), dict(dy=None), dict(dx=B), dict(dw=C),
               dict(ws=B), dict(dx=B + (1 << 20)), dict(ws=G + 16), dict(dw=F)):
        assert call(**kw) == _lib.EINVAL, kw
    assert call(n=255) == _lib.ENOSPACE
    assert call(dx=None, dw=None) == _lib.OK


def test_norm_refusals():
    def fwd(x=A, dt=_lib.BF16, res=B, s=C, sdt=_lib.F32, M=4, n=64, gain=D, eps=1e-6, y=F, ydt=_lib.BF16, y8=None):
        return RAW.moe_vq_norm_forward(x, dt, res, s, sdt, M, n, gain, eps, y, ydt, y8, None)

    for kw in (dict(x=None), dict(x=A + 8), dict(dt=2), dict(sdt=-1), dict(ydt=9), dict(res=B + 8), dict(s=C + 4), dict(M=-1), dict(n=0), dict(n=16385),
               dict(gain=None), dict(gain=D + 2), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(y=F + 8), dict(y8=r8(q=None)),
               dict(s=A), dict(y=B), dict(y=C), dict(y=D), dict(s=B + 16), dict(y=A + 16), dict(y=A, ydt=_lib.F32), dict(y8=r8(q=A)), dict(y8=r8(q=F)), dict(y8=r8(q=G, e=G))):
        assert fwd(**kw) == _lib.EINVAL, kw
    assert fwd(M=0, x=None) == fwd(s=None, y=None) == _lib.OK

    assert _lib.norm_bytes(4, 64) > 0 and _lib.norm_bytes(0, 64) > 0
    assert [_lib.norm_bytes(*a) for a in ((-1, 64), (4, 0), (4, 16385))] == [0, 0, 0]
    for n in (16, 300, 7168, 16384):
        need = [_lib.norm_bytes(m, n) for m in (1, 3, 100, 511, 512, 5000, 100000)]
        assert need == sorted(need)

    def back(s=A, sdt=_lib.BF16, M=4, n=64, gain=D, eps=1e-6, dy=B, dy2=None, ddt=_lib.BF16, ds=None, dx=C, xdt=_lib.BF16, dg=F, ws=G, nb=1 << 20):
        return RAW.moe_vq_norm_backward(s, sdt, M, n, gain, eps, dy, dy2, ddt, ds, dx, xdt, dg, ws, nb, None)

    for kw in (dict(s=None), dict(s=A + 8), dict(sdt=2), dict(M=-1), dict(n=0), dict(gain=None), dict(gain=D + 1), dict(eps=0.0), dict(dy=None), dict(dy=B + 8),
               dict(dy2=B + 8), dict(ddt=5), dict(ds=C + 8), dict(dx=C + 8), dict(xdt=5), dict(dg=F + 2), dict(ws=None), dict(ws=G + 16),
               dict(dx=A), dict(dx=B), dict(ds=C + 16), dict(dg=D), dict(ws=A), dict(dg=G)):
        assert back(**kw) == _lib.EINVAL, kw
    assert back(nb=255) == _lib.ENOSPACE
    assert back(dx=None, dg=None) == _lib.OK
    assert back(M=0, s=None, dx=C, dg=None, ws=None) == _lib.OK  # nothing to do, no workspace needed


def choice(E=64, k=4, score=0, G=8, top=4, best=2, renorm=1, scale=1.0, bias=None):
    return ctypes.byref(_lib.Choice(E, k, score, G, top, best, renorm, scale, bias))


def test_choose_refusals():
    bad = (dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(score=2), dict(score=-1), dict(G=0), dict(G=65), dict(G=7), dict(top=0), dict(top=9), dict(best=0),
           dict(best=3), dict(renorm=2), dict(scale=math.nan), dict(scale=math.inf), dict(bias=D + 1), dict(k=9, top=1))
    for kw in bad:
        assert RAW.moe_vq_choose(choice(**kw), A, 4, B, C, None) == _lib.EINVAL, kw
        assert RAW.moe_vq_choose_backward(choice(**kw), A, 4, B, C, F, None) == _lib.EINVAL, kw
    for args in ((None, 4, B, C), (A + 2, 4, B, C), (A, -1, B, C), (A, 65537, B, C), (A, 4, None, C), (A, 4, B + 1, C), (A, 4, B, None), (A, 4, B, B), (A, 4, A, C)):
        assert RAW.moe_vq_choose(choice(), *args, None) == _lib.EINVAL, args
        assert RAW.moe_vq_choose_backward(choice(), args[0], args[1], args[2], args[3], args[2], None) == _lib.EINVAL, args
    assert RAW.moe_vq_choose(None, A, 4, B, C, None) == _lib.EINVAL
    assert RAW.moe_vq_choose(choice(bias=D), A, 4, D, C, None) == _lib.EINVAL
    assert RAW.moe_vq_choose_backward(choice(), A, 4, B, C, A + 4, None) == _lib.EINVAL
    assert RAW.moe_vq_choose(choice(), None, 0, None, None, None) == _lib.OK


def test_objects_need_a_gpu():
    for make in (lambda: Rows8(4, 64, device="cpu"), lambda: RmsNorm(torch.ones(8)), lambda: ExpertChoice(8, 2, device="cpu")):
        with pytest.raises(ValueError):
            make()


def test_8_bits_by_definition_round_as_torch_does():
    """The definition that the kernels are held to: within half a step of x, and to the bit torch's conversion."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(40, 100, generator=g) * torch.exp2(torch.randint(-120, 100, (40, 1), generator=g).float())
    x[7] = 0
    q, e = ref.to8(x)
    v = ref.from8(q, e, 100)
    scale = torch.exp2(e.double() - 127).repeat_interleave(32, 1)[:, :100]
    assert ((v - x.double()).abs() <= torch.maximum(x.double().abs() / 16, scale * 2.0 ** -10)).all()
    assert (e[7] == 17).all() and (q[:, 100:] == 0).all()
    assert torch.equal(v.to(torch.bfloat16).double(), v)  # bf16 holds every value
