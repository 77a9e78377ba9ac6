"""The norm, the choice of experts and rows in 8 bits on the GPU against 64-bit plain forms (block_ref.py: each
bound counts the roundings of the computation)."""
import math

import pytest
import torch

import block_ref as ref
import dense_ref
from bit_vector_quantised_amd import _lib
from bit_vector_quantised_amd.block import ExpertChoice, RmsNorm
from bit_vector_quantised_amd.dense import ExpertRows, Linear, Rows8

from gpu_util import say
from test_gpu_dense import BF16, F32, gen, outside, randn, routing

pytestmark = pytest.mark.gpu


def stream(g, M, C, dtype):
    """Rows of several sizes, a few columns far larger than the others."""
    x = randn(g, M, C) * torch.where(torch.rand(C, generator=g) < 0.02, 20.0, 1.0)
    return (x * torch.exp(torch.randn(M, 1, generator=g))).to(dtype)


# ---------------------------------------------------------------------------------
# rows in 8 bits
# ---------------------------------------------------------------------------------

def test_every_e4m3_value():
    """Each of the 256 bytes stands for its value, and the value goes back to it."""
    say("e4m3 values")
    r = Rows8(8, 32)
    r.q.copy_(torch.arange(256, dtype=torch.uint8).view(8, 32))
    r.e.fill_(127 + 3)
    want = ref.from8(r.q, r.e, 32)
    for dtype in (BF16, F32):
        got = r.unpack(out=torch.empty(8, 32, dtype=dtype, device="cuda")).double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(), want.nan_to_num())
        back = Rows8(8, 32).pack(torch.where(torch.isnan(got), 448.0 * 8, got).to(dtype).cuda())
        assert torch.equal(ref.from8(back.q, back.e, 32), torch.where(torch.isnan(want), 448.0 * 8, want))


def test_ties_and_borders():
    """Values half way between two e4m3 values go to the even one, also below the smallest normal one; the scale changes
    where the largest magnitude passes 448 of them."""
    say("8 bits: ties and borders")
    step = torch.arange(0, 129).float() / 2  # halves of the steps of [8, 16): 8 + i / 2 steps
    tie = 256.0 + step * 2
    small = torch.arange(0, 33).float() * 2.0 ** -10  # halves of 2^-9, the smallest step
    x = torch.zeros(12, 160)
    x[0, :129], x[1, :33], x[2, :33] = tie, small, -small
    x[0, 128::32], x[1, 31], x[2, 31] = 448.0, 448.0, 448.0
    up = torch.nextafter(torch.tensor(448.0), torch.tensor(1e9)).item()
    for i, v in enumerate((448.0, up, 2.0 ** -126, 2.0 ** -149, 448 * 2.0 ** -110, up * 2.0 ** -110, 3.4e38, 448 * 2.0 ** 119)):
        x[3 + i, 40] = v
    r = Rows8(12, 160).pack(x.cuda())
    q, e = ref.to8(x)
    assert torch.equal(r.e.cpu(), e) and torch.equal(r.q.cpu(), q)


@pytest.mark.parametrize("M,C,dtype", [(1, 1, BF16), (1, 31, F32), (3, 32, BF16), (7, 33, BF16), (5, 7168, BF16), (129, 1000, F32),
                                       (64, 2047, BF16), (2, 32768, BF16), (1000, 64, F32)])
def test_pack_and_unpack(M, C, dtype):
    say(f"8 bits M={M} C={C} {dtype}")
    x = stream(gen(M * 7 + C), M, C, dtype)
    r = Rows8(M + 2, C)
    r.q.fill_(77)
    r.e.fill_(99)
    r.pack(x.cuda())
    q, e = ref.to8(x.float())
    assert torch.equal(r.q.cpu()[:M], q) and torch.equal(r.e.cpu()[:M], e)
    assert (r.q[M:] == 77).all() and (r.e[M:] == 99).all()  # rows behind: as they were
    want = ref.from8(q, e, C)
    for out in (BF16, F32):
        got = r.unpack(M, torch.empty(M, C, dtype=out, device="cuda"))
        assert torch.equal(got.double().cpu(), want)  # exact in either type


def test_values_that_are_not_finite():
    """A block with an infinity or NaN stands for NaNs; its neighbours do not know of it."""
    say("8 bits: not finite")
    for dtype in (BF16, F32):
        x = randn(gen(1), 4, 100, dtype=dtype)
        x[0, 3], x[1, 40], x[2, 99] = math.inf, -math.inf, math.nan
        r = Rows8(4, 100).pack(x.cuda())
        got = r.unpack(out=torch.empty(4, 100, dtype=dtype, device="cuda")).cpu()
        bad = torch.zeros(4, 100, dtype=torch.bool)
        bad[0, :32] = bad[1, 32:64] = bad[2, 96:] = True
        assert torch.equal(torch.isnan(got), bad)
        clean = torch.where(bad, 0.0, x.float())
        assert torch.equal(got[~bad].double(), ref.from8(*ref.to8(clean), 100)[~bad])


def test_rows_in_no_group_stay():
    say("8 bits: groups")
    x = randn(gen(2), 20, 70, dtype=BF16).cuda()
    start = torch.tensor([3, 9, 9, 14], dtype=torch.int32, device="cuda")
    r = Rows8(20, 70)
    r.q.fill_(7)
    r.e.fill_(9)
    r.pack(x, start)
    q, e = ref.to8(x.float().cpu())
    assert torch.equal(r.q.cpu()[3:14], q[3:14]) and torch.equal(r.e.cpu()[3:14], e[3:14])
    for rows in (slice(0, 3), slice(14, 20)):
        assert (r.q[rows] == 7).all() and (r.e[rows] == 9).all()
    out = torch.full((20, 70), -5.0, dtype=BF16, device="cuda")
    r.unpack(out=out, group_start=start)
    assert torch.equal(out.double().cpu()[3:14], ref.from8(q, e, 70)[3:14])
    assert (out[:3] == -5).all() and (out[14:] == -5).all()


@pytest.mark.parametrize("T,k,E,C,dropped,dtype", [(1, 8, 16, 7168, 0.0, BF16), (65, 3, 5, 333, 0.3, F32), (40, 6, 9, 4097, 0.1, BF16),
                                                   (33, 1, 4, 16, 1.0, BF16), (200, 8, 64, 96, 0.0, F32)])
def test_gather_from_8_bits(T, k, E, C, dropped, dtype):
    """To the bit what gathering the values gives, and nothing else is written."""
    say(f"gather from 8 bits T={T} k={k} C={C}")
    g = gen(T + C)
    rows = ExpertRows(E, k, T)
    rows.sort(routing(g, T, k, E, dropped).cuda())
    x8 = Rows8(T, C).pack(stream(g, T, C, F32).cuda())
    out = torch.full((T * k, C), -3.0, dtype=dtype, device="cuda")
    want = out.clone()
    rows.gather(x8, out)
    rows.gather(x8.unpack(out=torch.empty(T, C, dtype=dtype, device="cuda")), want)
    assert torch.equal(out, want)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("T,k,N,dtype,dy_dtype,dropped,weighted", [
    (1, 8, 2048, BF16, BF16, 0.0, True), (37, 3, 130, F32, F32, 0.2, True), (30, 2, 1, BF16, F32, 0.0, True),
    (21, 4, 1025, BF16, F32, 0.1, False), (9, 2, 4097, F32, BF16, 0.0, True), (50, 1, 64, BF16, BF16, 1.0, True),
    (64, 6, 40, F32, F32, 0.3, True)])
def test_act_backward(act, T, k, N, dtype, dy_dtype, dropped, weighted):
    say(f"act backward {act} T={T} k={k} N={N}")
    g = gen(T * 5 + N)
    P, R, lim = T * k, 2 * N if act == "swiglu" else N, 2.5
    rows = ExpertRows(8, k, T)
    rows.sort(routing(g, T, k, 8, dropped).cuda())
    z8 = Rows8(P, R).pack(randn(g, P, R, scale=1.7).cuda())
    dy, w = randn(g, P, N, dtype=dy_dtype), torch.rand(T, k, generator=g)
    dy[-1] = math.nan if dropped else dy[-1]  # (behind the last expert's rows nothing is looked at)
    dz, y, dw = (torch.full((P, n), -3.0, dtype=dtype, device="cuda") for n in (R, N, 1))
    dw = torch.full((T, k), -3.0, device="cuda")
    rows.act_backward(z8, dy.cuda(), w.cuda() if weighted else None, act, lim, dz, y, dw)
    want, named = ref.act_backward64(ref.from8(z8.q, z8.e, R), dy, rows.pair_row.cpu(), w if weighted else None, act, lim, dtype)
    rest = [r for r in range(P) if r not in set(named)]
    for name, got in (("dz", dz), ("y", y)):
        v, b = want[name]
        dense_ref.check(got[named], v[named], b[named], name)
        assert (got[rest] == -3).all()
    dense_ref.check(dw.reshape(-1), *want["dw"], "dw")
    # each output alone is the same
    for name, whole in (("dz", dz), ("y", y), ("dw", dw)):
        one = torch.full_like(whole, -3.0)
        rows.act_backward(z8, dy.cuda(), w.cuda() if weighted else None, act, lim, **{name: one})
        if name == "dw" or dtype == dy_dtype or one.dtype == dtype:
            assert torch.equal(one, whole), name


def test_outputs_larger_than_the_cache():
    """Streamed rows: gathered from 8 bits, unpacked, and those of the way back through swiglu, looked at where they begin, end
    and in between."""
    say("streamed rows")
    g = gen(77)
    T, k, E, N = 9000, 8, 16, 1032
    rows = ExpertRows(E, k, T)
    ids = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
    rows.sort(ids.cuda())
    pair_row, P = rows.pair_row.cpu(), T * k
    some = torch.cat((torch.arange(4), torch.randint(0, T, (60,), generator=g), torch.arange(T - 4, T)))
    x8 = Rows8(T, 2 * N).pack(torch.randn(T, 2 * N, device="cuda"))
    for dtype in (BF16, F32):
        out = torch.full((P, 2 * N), -3.0, dtype=dtype, device="cuda")
        rows.gather(x8, out)
        for t in some.tolist():
            want = ref.from8(x8.q[t:t + 1], x8.e[t:t + 1], 2 * N)[0]
            for i in range(k):
                r = int(pair_row[t * k + i])
                if r >= 0:
                    assert torch.equal(out[r].double().cpu(), want)
        n = int(rows.expert_start[-1])
        assert (out[n:] == -3).all()
    z8 = Rows8(P, 2 * N).pack(out)
    assert torch.equal(z8.unpack()[:n], out[:n].to(BF16))  # (they are values of 8 bits already)
    del out
    dy, w = torch.randn(P, N, device="cuda").bfloat16(), torch.rand(T, k, generator=g)
    dz, y, dw = torch.empty(P, 2 * N, dtype=BF16, device="cuda"), torch.empty(P, N, dtype=BF16, device="cuda"), torch.empty(T, k, device="cuda")
    rows.act_backward(z8, dy, w.cuda(), "swiglu", 2.0, dz, y, dw)
    pairs = torch.cat([torch.arange(t * k, t * k + k) for t in some.tolist()])
    pairs = pairs[pair_row[pairs] >= 0]
    at = pair_row[pairs].long()
    want, _ = ref.act_backward64(ref.from8(z8.q[at.cuda()], z8.e[at.cuda()], 2 * N), dy[at.cuda()].cpu(), torch.arange(len(at)),
                                 w.view(-1)[pairs], "swiglu", 2.0, BF16)
    dense_ref.check(dz[at.cuda()], *want["dz"], "dz")
    dense_ref.check(y[at.cuda()], *want["y"], "y")
    dense_ref.check(dw.view(-1)[pairs.cuda()], *want["dw"], "dw")
    assert not dw[ids.cuda() < 0].any()


@pytest.mark.parametrize("x8,z8", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("M,K,N,act,start,dtype,dy_dtype,bias", [
    (40, 64, 48, "swiglu", None, BF16, BF16, True), (33, 100, 37, "gelu", None, F32, F32, True),
    (130, 72, 33, "swiglu", [0, 50, 50, 125], BF16, F32, True), (65, 200, 96, "silu", [2, 30, 65], F32, BF16, False),
    (50, 31, 20, "none", None, BF16, BF16, True), (1, 256, 130, "swiglu", None, BF16, BF16, True),
    (300, 520, 264, "silu", None, BF16, BF16, True)])
def test_linear_gradients_from_8_bits(x8, z8, M, K, N, act, start, dtype, dy_dtype, bias):
    """The gradients of the values that the bytes stand for, whichever of x and z are in 8 bits."""
    say(f"linear gradients from 8 bits M={M} K={K} N={N} {act} {dtype}")
    g = gen(M + K + N)
    R = 2 * N if act == "swiglu" else N
    G = None if start is None else len(start) - 1
    lead = () if G is None else (G,)
    w = randn(g, *lead, R, K, dtype=dtype, scale=K ** -0.5)
    b = randn(g, *lead, R) if bias else None
    dy = randn(g, M, N, dtype=dy_dtype)
    xk, zk = Rows8(M, K).pack(randn(g, M, K).cuda()), Rows8(M, R).pack(randn(g, M, R).cuda())
    x, z = xk.unpack(out=torch.empty(M, K, dtype=dtype, device="cuda")), zk.unpack(out=torch.empty(M, R, dtype=dtype, device="cuda"))
    gs = None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
    lin = Linear(w.cuda(), None if b is None else b.cuda(), act=act, swiglu_limit=1.5, max_rows=M, backward=True, kept8=True)
    dx, dw = torch.full((M, K), -3.0, dtype=dtype, device="cuda"), torch.empty_like(w, device="cuda")
    db = torch.empty(*lead, R, device="cuda") if bias else None
    lin.backward(xk if x8 else x, dy.cuda(), None if act == "none" else (zk if z8 else z), gs, dx, dw, db)
    want = dense_ref.linear_backward64(x.float().cpu(), w, start, act, 1.5, z.float().cpu(), dy, dtype)
    rest = outside(M, start)
    inside = ~rest
    dense_ref.check(dx[inside], want["dx"][0][inside], want["dx"][1][inside], "dx")
    assert (dx[rest] == -3).all()
    dense_ref.check(dw, *want["dw"], "dw")
    if bias:
        dense_ref.check(db, *want["dbias"], "dbias")
    # and to the bit those of the plain tensors
    one = [torch.full_like(dx, -3.0), torch.empty_like(dw), torch.empty_like(db) if bias else None]
    lin.backward(x, dy.cuda(), None if act == "none" else z, gs, *one)
    assert torch.equal(one[0], dx) and torch.equal(one[1], dw) and (not bias or torch.equal(one[2], db))


# ---------------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------------

@pytest.mark.parametrize("M,C,dtype,s_dtype,y_dtype,residual", [
    (1, 7168, BF16, BF16, BF16, True), (1, 1, F32, F32, F32, False), (5, 3, BF16, F32, BF16, True), (17, 100, F32, BF16, F32, True),
    (9, 128, BF16, BF16, BF16, True), (9, 129, BF16, BF16, F32, False), (33, 512, BF16, F32, BF16, True), (6, 513, F32, F32, BF16, True),
    (50, 2047, BF16, F32, F32, True), (3, 8192, BF16, BF16, BF16, True), (3, 8193, F32, F32, F32, True), (2, 16384, BF16, BF16, BF16, True),
    (300, 64, BF16, BF16, BF16, True)])
def test_norm(M, C, dtype, s_dtype, y_dtype, residual):
    say(f"norm M={M} C={C}")
    g = gen(M + C)
    x, r, gain = stream(g, M, C, dtype), stream(g, M, C, s_dtype), 1 + 0.3 * randn(g, C)
    if M > 2:
        x[1] = 0
        r[1] = 0  # a row of zeros stays zeros
    norm = RmsNorm(gain.cuda(), eps=1e-5, max_rows=M + 1)
    s, y = torch.full((M + 1, C), -3.0, dtype=s_dtype, device="cuda"), torch.full((M + 1, C), -3.0, dtype=y_dtype, device="cuda")
    r8 = Rows8(M + 1, C)
    r8.q.fill_(5)
    r8.e.fill_(6)
    res = r.cuda() if residual else None
    norm.forward(x.cuda(), res, s[:M], y[:M], r8)
    want = ref.norm64(x, r if residual else None, gain, 1e-5, s_dtype, y_dtype)
    dense_ref.check(s[:M], want[0], want[1], "s")
    dense_ref.check(y[:M], want[2], want[3], "y")
    ref.check8(r8.q[:M], r8.e[:M], want[2], want[4], "8 bits")
    assert (s[M:] == -3).all() and (y[M:] == -3).all() and (r8.q[M:] == 5).all() and (r8.e[M:] == 6).all()
    # each output alone, and 8 bits alone, to the bit
    only = Rows8(M, C)
    assert norm.forward(x.cuda(), res, rows8=only, dense=False) is None
    assert torch.equal(only.q, r8.q[:M]) and torch.equal(only.e, r8.e[:M])
    assert torch.equal(norm.forward(x.cuda(), res, out=torch.empty_like(y[:M])), y[:M])


def test_norm_in_place():
    say("norm in place")
    g = gen(5)
    for C in (96, 400, 1000):
        x, r, gain = randn(g, 40, C).cuda(), randn(g, 40, C).cuda(), (1 + randn(g, C)).cuda()
        norm = RmsNorm(gain, max_rows=40)
        s = torch.empty_like(r)
        y = norm.forward(x, r, s)
        a, b = x.clone(), r.clone()
        norm.forward(a, b, s=b, out=a)  # the sum over the residual, y over x
        assert torch.equal(a, y) and torch.equal(b, s)
        a = x.clone()
        assert torch.equal(norm.forward(a, r, s=a), y) and torch.equal(a, s)


@pytest.mark.parametrize("M,C,dy_dtype,s_dtype,dx_dtype,two,stream_too", [
    (1, 7168, BF16, BF16, BF16, True, True), (1, 1, F32, F32, F32, False, False), (5, 3, BF16, F32, F32, True, True),
    (17, 100, F32, BF16, F32, False, True), (40, 128, BF16, BF16, BF16, True, False), (9, 129, BF16, BF16, BF16, False, True),
    (1300, 512, BF16, F32, F32, True, True), (600, 2047, BF16, F32, F32, True, True), (3, 8193, F32, F32, F32, True, True),
    (2, 16384, BF16, BF16, BF16, True, True), (70000, 16, BF16, BF16, BF16, False, True)])
def test_norm_backward(M, C, dy_dtype, s_dtype, dx_dtype, two, stream_too):
    say(f"norm backward M={M} C={C}")
    g = gen(M * 3 + C)
    s, gain = stream(g, M, C, s_dtype), 1 + 0.3 * randn(g, C)
    if M > 2:
        s[1] = 0
    dy, dy2 = randn(g, M, C, dtype=dy_dtype), randn(g, M, C, dtype=dy_dtype) if two else None
    ds = randn(g, M, C, dtype=dx_dtype) if stream_too else None
    norm = RmsNorm(gain.cuda(), eps=1e-5, max_rows=M, backward=True)
    dx, dg = torch.empty(M, C, dtype=dx_dtype, device="cuda"), torch.empty(C, device="cuda")
    on = lambda t: None if t is None else t.cuda()  # noqa: E731
    norm.backward(s.cuda(), dy.cuda(), on(dy2), on(ds), dx, dg)
    want = ref.norm_backward64(s, gain, 1e-5, dy, dy2, ds, dx_dtype)
    dense_ref.check(dx, want[0], want[1], "dx")
    dense_ref.check(dg, want[2], want[3], "dgain")
    one, other = torch.empty_like(dx), torch.empty_like(dg)
    norm.backward(s.cuda(), dy.cuda(), on(dy2), on(ds), dx=one)
    norm.backward(s.cuda(), dy.cuda(), on(dy2), on(ds), dgain=other)
    assert torch.equal(one, dx) and torch.equal(other, dg)
    if stream_too:  # dx over ds
        same = ds.cuda()
        norm.backward(s.cuda(), dy.cuda(), on(dy2), same, same, other)
        assert torch.equal(same, dx)


def test_norm_gradient_by_differences():
    """dx and dgain are the slopes of sum(c y) + sum(d s) in 64 bits: central differences of step h are off by h^2 times the third
    derivative and 2^-52 of the value over h."""
    say("norm: differences")
    g = gen(9)
    M, C, h = 3, 40, 1e-4
    x, r, gain, c, d = randn(g, M, C), randn(g, M, C), 1 + 0.3 * randn(g, C), randn(g, M, C), randn(g, M, C)
    norm = RmsNorm(gain.cuda(), max_rows=M, backward=True)
    s = torch.empty(M, C, device="cuda")
    norm.forward(x.cuda(), r.cuda(), s)
    dx, dg = torch.empty_like(s), torch.empty(C, device="cuda")
    norm.backward(s, c.cuda(), None, d.cuda(), dx, dg)

    def value(x, gain):
        s, _, y, _, _ = ref.norm64(x, r, gain, 1e-6, F32, F32)
        return ((c.double() * y).sum(1) + (d.double() * s).sum(1))

    x64, g64 = x.double(), gain.double()
    for i in range(C):
        step = torch.zeros(M, C, dtype=torch.float64)
        step[:, i] = h
        slope = (value(x64 + step, g64) - value(x64 - step, g64)) / (2 * h)
        # (values below 40, third derivatives below 100 here: 1e-6; the gradient itself a few 1e-7 of its terms)
        assert (slope - dx[:, i].double().cpu()).abs().max() < 2e-5
        by = (value(x64, g64 + step[0]) - value(x64, g64 - step[0])).sum() / (2 * h)
        assert abs(by.item() - dg[i].item()) < 2e-5


# ---------------------------------------------------------------------------------
# choice of experts
# ---------------------------------------------------------------------------------

CHOICES = [dict(E=1, k=1), dict(E=5, k=3), dict(E=64, k=8, score="sigmoid"), dict(E=65, k=6, renorm=False), dict(E=256, k=8, scale=2.5),
           dict(E=128, k=4, score="sigmoid", renorm=False, bias=True), dict(E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4, scale=2.5),
           dict(E=160, k=6, groups=8, top_groups=3, best=1, renorm=False, scale=16.0), dict(E=40, k=5, groups=5, top_groups=1, bias=True),
           dict(E=1024, k=32, score="sigmoid", bias=True), dict(E=1000, k=32, groups=10, top_groups=2, best=2),
           dict(E=512, k=9, bias=True), dict(E=64, k=4, groups=64, top_groups=7, score="sigmoid", best=1), dict(E=300, k=2, renorm=False, bias=True)]


def make(E, k, score="softmax", bias=None, groups=1, top_groups=None, best=2, renorm=True, scale=1.0):
    return ExpertChoice(E, k, score, bias, groups, top_groups, best, renorm, scale)


def spec(c):
    c = dict(c)
    E, k, biased = c.pop("E"), c.pop("k"), c.pop("bias", False)
    return E, k, biased, c


@pytest.mark.parametrize("case", CHOICES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
@pytest.mark.parametrize("T", [1, 37])
def test_choose(case, T):
    """Ids equal, weights within their bound: logits spread and close together, rows with some, most and all experts off."""
    E, k, biased, rest = spec(case)
    say(f"choose {case} T={T}")
    g = gen(E + T)
    bias = 0.2 * randn(g, E) if biased else None
    for size in (1.5, 0.01, 8.0):
        logits = size * randn(g, T, E)
        if T > 8:
            logits[2] = -math.inf                                              # nothing left
            logits[3, torch.rand(E, generator=g) < 0.8] = -math.inf            # fewer than k, perhaps
            logits[4, torch.rand(E, generator=g) < 0.3] = math.nan
            logits[5] = 0.25                                                   # all equal
            logits[6] = torch.round(logits[6])                                 # many equal
            logits[7] -= 100                                                   # scores that fp32 loses
        choice = make(E, k, bias=None if bias is None else bias.cuda(), **rest)
        ids, w = choice.forward(logits.cuda())
        want, ww, rel = ref.choose64(logits, bias, k, **{"top_groups": rest.get("groups", 1), **rest})
        assert torch.equal(ids.cpu().long(), want), (ids.cpu().long() != want).nonzero()[:4]
        dense_ref.check(w, ww, rel * ww.abs(), "w")
        dw = randn(g, T, k)
        got = choice.backward(logits.cuda(), ids, dw.cuda())
        v, b = ref.choose_backward64(logits, bias, want, dw, rest.get("score", "softmax"), rest.get("renorm", True), rest.get("scale", 1.0))
        dense_ref.check(got, v, b, "dlogits")
        over = logits.cuda()
        choice.backward(over, ids, dw.cuda(), dlogits=over)
        assert torch.equal(over, got)


def test_choose_tells_close_values_apart():
    """Values v = sigmoid(l) + b that fp32 holds equal are ordered as 64 bits do; equal ones by number."""
    say("choose: close values")
    E, T = 64, 200
    g = gen(11)
    logits = randn(g, T, E)
    # biases that nearly cancel the scores' differences
    base = torch.sigmoid(logits[0].double())
    bias = (1.0 - base).float()
    logits[1:T // 2] = logits[0] + 1e-7 * randn(g, T // 2 - 1, E)
    choice = make(E, 8, "sigmoid", bias.cuda())
    ids, _ = choice.forward(logits.cuda())
    want, _, _ = ref.choose64(logits, bias, 8, "sigmoid")
    assert torch.equal(ids.cpu().long(), want)
    # groups whose two best add up alike
    grouped = make(E, 8, "sigmoid", bias.cuda(), groups=8, top_groups=3)
    ids, _ = grouped.forward(logits.cuda())
    want, _, _ = ref.choose64(logits, bias, 8, "sigmoid", groups=8, top_groups=3)
    assert torch.equal(ids.cpu().long(), want)


def test_choose_scores_below_fp32():
    """Scores and biases that are subnormal in fp32, or less, are ordered by their values all the same."""
    say("choose: scores below fp32")
    E, T = 64, 48
    g = gen(17)
    logits = torch.cat([0.5 * randn(g, T // 3, E) - 89.5, 8 * randn(g, T // 3, E) - 110, 2 * randn(g, T // 3, E) - 62])
    # one score that fp32 may hold against a group whose scores it may not, of which two are more
    for row, (one, many) in enumerate([(-87.2, -87.5), (-88.6, -88.75), (-88.0, -88.5)]):
        logits[row] = -97.0 - torch.arange(E) / 16
        logits[row, 0], logits[row, 8], logits[row, 9] = one, many, many + 0.01
    for bias in (None, 1e-40 * randn(g, E), torch.zeros(E)):
        for kw in (dict(), dict(groups=8, top_groups=1), dict(groups=8, top_groups=3)):
            choice = make(E, 8, "sigmoid", bias=None if bias is None else bias.cuda(), **kw)
            ids, w = choice.forward(logits.cuda())
            want, ww, rel = ref.choose64(logits, bias, 8, "sigmoid", **{"top_groups": kw.get("groups", 1), **kw})
            assert torch.equal(ids.cpu().long(), want)
            dense_ref.check(w, ww, rel * ww.abs(), "w")


def test_choose_infinities():
    say("choose: infinities")
    E = 70
    logits = randn(gen(3), 6, E)
    logits[0, 5] = math.inf
    logits[1, [4, 66]] = math.inf
    bias = torch.zeros(E)
    bias[9], bias[11], bias[13] = -math.inf, math.nan, math.inf
    for renorm in (True, False):
        ids, w = make(E, 3, renorm=renorm).forward(logits.cuda())
        assert ids[0, 0] == 5 and ids[1, :2].tolist() == [4, 66]
        assert w[0].tolist() == [1.0, 0.0, 0.0] and w[1].tolist() == [0.5, 0.5, 0.0]
        ids, w = make(E, 3, "sigmoid", renorm=renorm, bias=bias.cuda()).forward(logits.cuda())
        assert (ids[:, 0] == 13).all() and not ((ids == 9) | (ids == 11)).any() and torch.isfinite(w).all()
        everything = make(E, 32, "softmax", renorm=renorm, bias=bias.cuda())
        ids, w = everything.forward(logits[2:].cuda())
        assert torch.isfinite(w).all()
        d = everything.backward(logits[2:].cuda(), ids, torch.ones(4, 32, device="cuda"))
        assert torch.isfinite(d).all() and (d[:, [9, 11]] == 0).all()


def test_choose_masks_of_the_lowest_value():
    """The type's lowest value is a value, not -inf: such experts come last, in order, with weights of 0."""
    say("choose: lowest values")
    E, T, k = 96, 12, 16
    low = torch.finfo(F32).min
    g = gen(31)
    logits = randn(g, T, E)
    logits[:, 5:] = torch.where(torch.rand(T, E - 5, generator=g) < 0.9, low, logits[:, 5:])
    logits[1] = low
    bias = 0.1 * randn(g, E)
    bias[[2, 40, 41]] = low
    for b in (None, bias):
        for kw in (dict(), dict(score="sigmoid"), dict(score="softmax", renorm=False), dict(score="sigmoid", groups=8, top_groups=5)):
            choice = make(E, k, bias=None if b is None else b.cuda(), **kw)
            ids, w = choice.forward(logits.cuda())
            want, ww, rel = ref.choose64(logits, b, k, **{"top_groups": kw.get("groups", 1), **kw})
            assert torch.equal(ids.cpu().long(), want) and (ids >= 0).all()
            dense_ref.check(w, ww, rel * ww.abs(), "w")
            d = choice.backward(logits.cuda(), ids, torch.ones(T, k, device="cuda"))
            assert torch.isfinite(d).all()


def test_choose_backward_of_other_ids():
    """The same expert twice gets both parts; ids that are none get nothing."""
    say("choose backward: other ids")
    g = gen(8)
    logits, dw = randn(g, 12, 100), randn(g, 12, 5)
    ids = torch.randint(0, 100, (12, 5), generator=g)
    ids[:, 3] = ids[:, 1]
    ids[0, 0], ids[1, 2], ids[2, 4] = -1, 100, 2 ** 31 - 1
    ids[5] = -1
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = make(100, 5, score, renorm=renorm).backward(logits.cuda(), ids.int().cuda(), dw.cuda())
            v, b = ref.choose_backward64(logits, None, ids, dw, score, renorm)
            dense_ref.check(got, v, 2 * b, "dlogits")  # (two parts of one expert are two roundings more)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_choose_gradient_by_differences(score, renorm):
    """dlogits are the slopes of sum(c w) at fixed ids, in 64 bits."""
    say(f"choose: differences {score} {renorm}")
    g = gen(21)
    T, E, k, h = 4, 20, 5, 1e-5
    logits, c = randn(g, T, E), randn(g, T, k)
    choice = make(E, k, score, renorm=renorm, scale=2.5)
    ids, _ = choice.forward(logits.cuda())
    got = choice.backward(logits.cuda(), ids, c.cuda()).double().cpu()
    at = ids.cpu().long()

    def value(l):
        s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
        p = s.gather(1, at)
        return (c.double() * 2.5 * (p / p.sum(1, keepdim=True) if renorm else p)).sum(1)

    for e in range(E):
        step = torch.zeros(T, E, dtype=torch.float64)
        step[:, e] = h
        slope = (value(logits.double() + step) - value(logits.double() - step)) / (2 * h)
        assert (slope - got[:, e]).abs().max() < 5e-6  # (values below 10: 1e-10 / 1e-5, and a few 1e-7 of the fp32 gradient)
