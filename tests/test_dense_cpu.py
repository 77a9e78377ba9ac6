"""The row operators and the dense product without a GPU: sizes, and bad arguments refused
before any HIP call (pointer values are never dereferenced on these paths)."""
import ctypes

import pytest

mvq = pytest.importorskip("bit_vector_quantised_amd")
from bit_vector_quantised_amd import _lib  # noqa: E402

A = 0x100000  # an aligned address
RAW = _lib.raw()


def lin(n_in=256, n_out=128, groups=1, act=_lib.ACT_NONE, dtype=_lib.BF16, lim=0.0, w=A, bias=None):
    return _lib.LinearDesc(n_in, n_out, groups, act, dtype, lim, w, bias)


def test_sort_bytes():
    assert _lib.sort_bytes(1, 8, 256) > 0 and _lib.sort_bytes(0, 1, 1) > 0
    for bad in ((-1, 8, 256), (65537, 8, 256), (1, 0, 256), (1, 33, 256), (1, 8, 0), (1, 8, 1025)):
        assert _lib.sort_bytes(*bad) == 0, bad
    # a workspace made for more tokens serves any smaller call
    for k, E in ((1, 1), (8, 256), (32, 1024)):
        need = [_lib.sort_bytes(t, k, E) for t in (1, 100, 2048, 4096, 4097, 16384, 16385, 40000, 65536)]
        assert need == sorted(need)


def test_sort_refusals():
    ok = dict(ids=A, T=4, k=2, E=8, start=A, pair=A, row=A, ws=A, n=1 << 20)

    def call(**kw):
        a = {**ok, **kw}
        return RAW.moe_vq_sort_pairs(a["ids"], a["T"], a["k"], a["E"], a["start"], a["pair"], a["row"], a["ws"], a["n"], None)

    for kw in (dict(ids=None), dict(start=None), dict(pair=None), dict(row=None), dict(ws=None), dict(ws=A + 16),
               dict(T=-1), dict(T=65537), dict(k=0), dict(k=33), dict(E=0), dict(E=1025), dict(ids=A + 2),
               dict(start=A + 1), dict(pair=A + 2), dict(row=A + 2)):
        assert call(**kw) == _lib.EINVAL, kw
    assert call(n=31) == _lib.ENOSPACE


def test_rows_refusals():
    def gather(x=A, dt=_lib.BF16, T=4, k=2, C=64, pair=A, xs=A):
        return RAW.moe_vq_gather_rows(x, dt, T, k, C, pair, xs, None)

    def combine(rows=A, dt=_lib.BF16, T=4, k=2, C=64, pair=A, w=None, res=None, y=A, ydt=_lib.F32):
        return RAW.moe_vq_combine_rows(rows, dt, T, k, C, pair, w, res, y, ydt, None)

    def back(dy=A, ddt=_lib.F32, T=4, k=2, C=64, pair=A, w=None, rows=A, dt=_lib.BF16, drows=A, dw=A):
        return RAW.moe_vq_combine_rows_backward(dy, ddt, T, k, C, pair, w, rows, dt, drows, dw, None)

    dims = (dict(T=-1), dict(T=65537), dict(k=0), dict(k=33), dict(C=0), dict(C=65537), dict(dt=2), dict(dt=-1),
            dict(pair=None), dict(pair=A + 2))
    for kw in dims + (dict(x=None), dict(x=A + 8), dict(xs=None), dict(xs=A + 4)):
        assert gather(**kw) == _lib.EINVAL, kw
    for kw in dims + (dict(rows=None), dict(rows=A + 8), dict(y=None), dict(y=A + 8), dict(res=A + 8), dict(ydt=7),
                      dict(w=A + 1)):
        assert combine(**kw) == _lib.EINVAL, kw
    for kw in dims + (dict(dy=None), dict(dy=A + 8), dict(rows=None), dict(rows=A + 4), dict(drows=A + 8), dict(ddt=7),
                      dict(w=A + 2), dict(dw=A + 2)):
        assert back(**kw) == _lib.EINVAL, kw
    assert gather(T=0) == combine(T=0) == back(T=0) == _lib.OK
    assert back(drows=None, dw=None) == _lib.OK


BAD_LINEAR = (dict(n_in=0), dict(n_in=16385), dict(n_out=0), dict(n_out=16385), dict(groups=0), dict(groups=1025),
              dict(act=-1), dict(act=4), dict(dtype=2), dict(act=_lib.ACT_SWIGLU, lim=-1.0),
              dict(act=_lib.ACT_SWIGLU, lim=float("nan")), dict(act=_lib.ACT_SWIGLU, lim=float("inf")))


def test_linear_bytes():
    assert _lib.linear_bytes(lin(), 1) > 0 and _lib.linear_bytes(lin(), 0, True) > 0
    for kw in BAD_LINEAR:
        assert _lib.linear_bytes(lin(**kw), 16) == 0, kw
    assert _lib.linear_bytes(lin(), -1) == 0 and _lib.linear_bytes(lin(), 65536 * 32 + 1) == 0
    assert RAW.moe_vq_linear_bytes(None, 4, 0) == 0 and RAW.moe_vq_linear_bytes(ctypes.byref(lin()), 4, 2) == 0
    # a workspace made for more rows serves any smaller call, whose contraction may be split further
    for kw in (dict(), dict(n_in=8192, n_out=64), dict(n_in=333, n_out=4097, act=_lib.ACT_SWIGLU),
               dict(groups=16, dtype=_lib.F32), dict(n_in=64, n_out=64)):
        for backward in (False, True):
            need = [_lib.linear_bytes(lin(**kw), m, backward) for m in (0, 1, 16, 17, 64, 65, 128, 500, 4096, 100000)]
            assert need == sorted(need), (kw, backward, need)


@pytest.mark.parametrize("backward", [False, True])
def test_linear_refusals(backward):
    big = 1 << 40

    def call(desc=None, x=A, M=4, start=None, res=None, y=A, dt=_lib.F32, z=A, dx=A, dw=A, db=A, ws=A, n=big):
        d = ctypes.byref(desc if desc is not None else lin(act=_lib.ACT_SILU))
        if backward:
            return RAW.moe_vq_linear_backward(d, x, M, start, z, y, dt, dx, dw, db, ws, n, None)
        return RAW.moe_vq_linear_forward(d, x, M, start, res, y, dt, z, ws, n, None)

    for kw in BAD_LINEAR + (dict(w=None), dict(w=A + 8), dict(bias=A + 2), dict(groups=4)):
        assert call(lin(**kw)) == _lib.EINVAL, kw
    bad = [dict(x=None), dict(x=A + 4), dict(M=-1), dict(M=65536 * 32 + 1), dict(y=None), dict(y=A + 8), dict(dt=5),
           dict(z=A + 8), dict(ws=None), dict(ws=A + 128), dict(start=A + 2)]
    bad += [dict(z=None), dict(dx=A + 8), dict(dw=A + 8), dict(db=A + 2)] if backward else [dict(res=A + 8)]
    for kw in bad:
        assert call(**kw) == _lib.EINVAL, kw
    assert call(n=0) == _lib.ENOSPACE
    if backward:
        assert call(dx=None, dw=None, db=None) == _lib.OK
    else:
        assert call(M=0) == _lib.OK


def test_overlapping_buffers_are_refused():
    """A workgroup would read what another has overwritten.  (Buffers far apart are let through to the launch,
    so only refusals are tried here: one byte of overlap from either side.)"""
    far = [A + (i << 30) for i in range(1, 8)]

    def fwd(x=far[0], res=None, y=far[1], z=far[2]):
        d = lin(n_in=64, n_out=32, act=_lib.ACT_SWIGLU)  # 4 rows: x 512 bytes, y 512, z 512
        return RAW.moe_vq_linear_forward(ctypes.byref(d), x, 4, None, res, y, _lib.F32, z, far[6], 1 << 40, None)

    def bwd(x=far[0], z=far[1], dy=far[2], dx=far[3], dw=far[4], act=_lib.ACT_NONE):
        d = lin(n_in=64, n_out=32, act=act)  # dw 32 x 64: 4096 bytes, or 8192
        return RAW.moe_vq_linear_backward(ctypes.byref(d), x, 4, None, z, dy, _lib.F32, dx, dw, None, far[6], 1 << 40, None)

    for off in (-496, 0, 496):
        assert fwd(y=far[0] + off) == fwd(z=far[0] + off) == fwd(z=far[1] + off) == _lib.EINVAL
        assert fwd(res=far[2] + off) == _lib.EINVAL  # z over the residual
        for act in (_lib.ACT_NONE, _lib.ACT_SWIGLU):
            assert bwd(dx=far[0] + off, act=act) == bwd(dw=far[0] + off, act=act) == _lib.EINVAL
            assert bwd(dx=far[4] + off, act=act) == _lib.EINVAL
        assert bwd(dx=far[2] + off) == bwd(dw=far[2] + off) == _lib.EINVAL
    for off in (-496, 496):
        assert fwd(res=far[1] + off) == _lib.EINVAL  # y may be residual, but not part of it

    def gather(x, xs):  # x 512 bytes, xs 1024
        return RAW.moe_vq_gather_rows(x, _lib.BF16, 4, 2, 64, far[4], xs, None)

    def combine(rows, res, y):  # rows 1024, y 1024
        return RAW.moe_vq_combine_rows(rows, _lib.BF16, 4, 2, 64, far[4], None, res, y, _lib.F32, None)

    def back(dy, rows, drows):
        return RAW.moe_vq_combine_rows_backward(dy, _lib.F32, 4, 2, 64, far[4], None, rows, _lib.BF16, drows, far[5], None)

    for off in (-1008, 0, 496):
        assert gather(far[0], far[0] + off) == _lib.EINVAL
        assert combine(far[0], None, far[0] + off) == _lib.EINVAL
        assert back(far[0], far[1], far[0] + off) == back(far[0], far[1], far[1] + off) == _lib.EINVAL
    for off in (-1008, 1008):
        assert combine(far[0], far[1] + off, far[1]) == _lib.EINVAL


def test_a_refused_experts_call_keeps_nothing():
    """After a call that failed on the way, backward must not mix two passes' buffers."""
    import torch

    from bit_vector_quantised_amd.dense import DenseExperts

    class Refusing:
        top_k = 1
        expert_start = None

        def sort(self, ids):
            raise ValueError("refused")

        def combine_backward(self, *a):
            raise ValueError("refused")

    step = DenseExperts.__new__(DenseExperts)
    step.rows, step.z, x = Refusing(), torch.zeros(2, 4), torch.zeros(2, 4)
    step.o = step.do = x
    for call in (lambda: step.forward(x, x, x, keep=True), lambda: step.backward(x, x, x, x, x)):
        step._kept = (x, x)
        with pytest.raises(ValueError, match="refused"):
            call()
        with pytest.raises(ValueError, match="kept nothing"):
            step.backward(x, x, x, x, x)


def test_python_refuses_what_the_library_cannot_see():
    import torch

    from bit_vector_quantised_amd.dense import DenseExperts, ExpertRows, Linear, _need
    with pytest.raises(ValueError):
        ExpertRows(8, 2, 4, device="cpu")
    with pytest.raises(ValueError):
        Linear(torch.zeros(4, 8))  # weights in host memory
    with pytest.raises(ValueError):
        Linear(torch.zeros(4, 8), act="relu")
    with pytest.raises(ValueError):
        DenseExperts(torch.zeros(2, 8, 16), torch.zeros(2, 16, 5), 1, 4)
    cpu = torch.device("cpu")
    t = torch.zeros(4, 6)
    assert _need(t, "t", (4, 6), torch.float32, cpu) == t.data_ptr()
    for bad in (t.t(), t[:, :3], t.bfloat16(), t[:3]):
        with pytest.raises(ValueError):
            _need(bad, "t", (4, 6), torch.float32, cpu)


class Buffers:
    """Named buffers far apart: their sizes, the alignment each needs, and calls with one of them moved onto another."""

    def __init__(self, **sizes):
        self.size = {n: v[0] for n, v in sizes.items()}
        self.align = {n: v[1] for n, v in sizes.items()}
        self.at = {n: A + ((i + 1) << 32) for i, n in enumerate(sizes)}

    def refused(self, call, a, b, same=True):
        """a's last bytes on b's first, both at one address (unless `same` allows that), a's first on b's last."""
        step = self.align[a]
        spots = {-self.size[a] + step, 0, (self.size[b] - 1) // step * step}
        for off in spots if same else spots - {0}:
            assert call({**self.at, a: self.at[b] + off}) == _lib.EINVAL, (a, "at", b, off)


def test_every_written_buffer_is_kept_apart():
    """Each buffer that a call writes against each other one that it reads or writes (only refusals, which return
    before any launch)."""
    big = 1 << 40
    b = Buffers(ids=(16, 4), start=(16, 4), pair=(16, 4), row=(16, 4), ws=(256, 256))

    def sort(p):
        return RAW.moe_vq_sort_pairs(p["ids"], 4, 1, 3, p["start"], p["pair"], p["row"], p["ws"], big, None)

    for a, c in (("start", "ids"), ("pair", "ids"), ("row", "ids"), ("start", "pair"), ("start", "row"), ("pair", "row"),
                 ("ws", "ids"), ("ws", "start"), ("ws", "pair"), ("ws", "row")):
        b.refused(sort, a, c)

    # 4 tokens, top-2, 64 columns
    b = Buffers(x=(512, 16), rows=(1024, 16), res=(1024, 16), y=(1024, 16), pair=(32, 4), w=(32, 4), dy=(1024, 16),
                drows=(1024, 16), dw=(32, 4))

    def gather(p):
        return RAW.moe_vq_gather_rows(p["x"], _lib.BF16, 4, 2, 64, p["pair"], p["rows"], None)

    def combine(p):
        return RAW.moe_vq_combine_rows(p["rows"], _lib.BF16, 4, 2, 64, p["pair"], p["w"], p["res"], p["y"], _lib.F32, None)

    def back(p):
        return RAW.moe_vq_combine_rows_backward(p["dy"], _lib.F32, 4, 2, 64, p["pair"], p["w"], p["rows"], _lib.BF16,
                                                p["drows"], p["dw"], None)

    for a, c in (("rows", "x"), ("rows", "pair")):
        b.refused(gather, a, c)
    for a in ("rows", "pair", "w"):
        b.refused(combine, a, "y")
    b.refused(combine, "res", "y", same=False)
    for a in ("dy", "rows", "pair", "w", "dw"):
        b.refused(back, a, "drows")
    for a in ("dy", "rows", "pair"):
        b.refused(back, "dw", a)
    b.refused(back, "dw", "w", same=False)

    # 4 rows, 64 -> 32, bf16 with fp32 outputs; dx and dw of x's and w's sizes
    for act, R in ((_lib.ACT_NONE, 32), (_lib.ACT_SILU, 32), (_lib.ACT_SWIGLU, 64)):
        sizes = dict(x=(512, 16), w=(R * 128, 16), bias=(R * 4, 4), table=(8, 4), res=(512, 16), y=(512, 16), z=(R * 8, 16),
                     dy=(512, 16), dx=(512, 16), dw=(R * 128, 16), db=(R * 4, 4))

        def fwd(p):
            d = lin(n_in=64, n_out=32, act=act, w=p["w"], bias=p["bias"])
            return RAW.moe_vq_linear_forward(ctypes.byref(d), p["x"], 4, p["table"], p["res"], p["y"], _lib.F32, p["z"], p["ws"],
                                             big, None)

        def bwd(p):
            d = lin(n_in=64, n_out=32, act=act, w=p["w"], bias=p["bias"])
            return RAW.moe_vq_linear_backward(ctypes.byref(d), p["x"], 4, p["table"], p["z"], p["dy"], _lib.F32, p["dx"], p["dw"],
                                              p["db"], p["ws"], big, None)

        b = Buffers(**sizes, ws=(256, 256))
        for a in ("x", "w", "bias", "table"):
            b.refused(fwd, a, "y")
            b.refused(fwd, a, "z")
            b.refused(fwd, "ws", a)
        b.refused(fwd, "y", "z")
        b.refused(fwd, "res", "z")
        b.refused(fwd, "res", "y", same=False)
        for a in ("res", "y", "z"):
            b.refused(fwd, "ws", a)
        read = ["x", "table", "dy"] + (["z"] if act != _lib.ACT_NONE else [])
        for a in ["w", "dx", "dw"] + read:
            b.refused(bwd, "db", a)
            b.refused(bwd, "ws", a)
        for a in ("w", "x", "table", "dw"):
            b.refused(bwd, "dx", a)
        for a in ("x", "table"):
            b.refused(bwd, "dw", a)
        if act == _lib.ACT_NONE:
            b.refused(bwd, "dx", "dy")
            b.refused(bwd, "dw", "dy")


def test_a_workspace_serves_every_smaller_call():
    """What a call needs itself, not only its bound: with the bytes for the largest number of rows no smaller call is
    told that its workspace is too small.  (The calls' buffers overlap, which is looked at last: nothing is launched.)"""
    shapes = [dict(n_in=k, n_out=n, groups=g, act=a, dtype=t)
              for k, n in ((256, 128), (8192, 64), (64, 8192), (333, 4097), (7168, 2048), (16384, 40), (24, 24))
              for g in (1, 3, 64, 1024) for a in (_lib.ACT_NONE, _lib.ACT_SWIGLU) for t in (_lib.BF16, _lib.F32)]
    rows = (1, 2, 15, 16, 17, 63, 64, 65, 100, 128, 129, 300, 511, 512, 513, 1000, 2048, 5000, 20000, 100000)
    for kw in shapes:
        d = lin(**kw)
        for i, most in enumerate(rows):
            need = [_lib.linear_bytes(d, most, b) for b in (False, True)]
            for m in rows[:i + 1]:
                p = ctypes.byref(d)
                start = A if kw["groups"] > 1 else None
                assert RAW.moe_vq_linear_forward(p, A, m, start, None, A, _lib.F32, A, A, need[0], None) == _lib.EINVAL, (kw, most, m)
                assert RAW.moe_vq_linear_backward(p, A, m, start, A, A, _lib.F32, A, A, A, A, need[1], None) == _lib.EINVAL, (kw, most, m)
        assert RAW.moe_vq_linear_forward(p, A, m, start, None, A, _lib.F32, A, A, 255, None) == _lib.ENOSPACE
