"""The row operators and the dense product on the GPU against 64-bit plain forms
(dense_ref.py: each bound counts the roundings of the computation)."""
import pytest
import torch

import dense_ref as ref
from bit_vector_quantised_amd import _lib
from bit_vector_quantised_amd.dense import DenseExperts, ExpertRows, Linear

from gpu_util import say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def routing(g, T, k, E, dropped=0.0, repeat=False):
    if repeat:
        ids = torch.randint(0, E, (T, k), generator=g)
    else:
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    ids = torch.where(torch.rand(T, k, generator=g) < dropped, -1, ids)
    return ids.to(torch.int32)


# ---------------------------------------------------------------------------------
# sort
# ---------------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E,dropped,repeat", [
    (1, 1, 1, 0.0, False), (1, 8, 256, 0.0, False), (7, 3, 5, 0.3, False), (5, 4, 3, 0.0, True), (33, 8, 40, 1.0, False),
    (512, 8, 1024, 0.1, False),     # 4096 pairs: the most of the four-step sort in one workgroup
    (2049, 2, 16, 0.0, False),      # one more: sixteen steps
    (2048, 8, 256, 0.05, False),    # 16384 pairs: the most in one workgroup
    (2049, 8, 256, 0.05, False),    # two launches
    (16384, 8, 1, 0.0, True),       # 131072 pairs of one expert
    (16385, 8, 1000, 0.2, True),    # the longer workgroups of two launches
    (65536, 32, 3, 0.01, True),     # the most pairs there can be
])
def test_sort(T, k, E, dropped, repeat):
    say(f"sort T={T} k={k} E={E}")
    g = gen(T * 31 + k)
    ids = torch.randint(-1 if dropped else 0, E, (T, k), generator=g, dtype=torch.int32) if T > 4096 else routing(g, T, k, E, dropped, repeat)
    if T == 7:
        ids[0, 0], ids[1, 1] = E, 2 ** 31 - 1  # ids behind the last expert are dropped too
    rows = ExpertRows(E, k, T)
    rows.sort(ids.cuda())
    torch.cuda.synchronize()
    if T <= 4096 and E <= 256:
        start, pair_row, row_pair = (torch.tensor(v) for v in ref.sort64(ids.reshape(-1), E))
    else:
        flat = ids.reshape(-1).long()
        key = torch.where((flat < 0) | (flat >= E), E, flat)
        order = torch.argsort(key, stable=True)
        start = torch.zeros(E + 1, dtype=torch.int64)
        start[1:] = torch.cumsum(torch.bincount(key, minlength=E + 1)[:E], 0)
        n = int(start[E])
        row_pair = torch.where(torch.arange(T * k) < n, order, -1)
        pair_row = torch.full((T * k,), -1)
        pair_row[order[:n]] = torch.arange(n)
    assert torch.equal(rows.expert_start.cpu().long(), start)
    assert torch.equal(rows.pair_row.cpu().long(), pair_row)
    assert torch.equal(rows.row_pair.cpu().long(), row_pair)


def test_sort_of_fewer_and_of_no_tokens():
    say("sort: fewer tokens than made for, then none")
    rows = ExpertRows(6, 2, 40)
    ids = routing(gen(3), 9, 2, 6).cuda()
    rows.pair_row.fill_(-7)
    rows.sort(ids)
    start, pair_row, _ = ref.sort64(ids.cpu().reshape(-1), 6)
    assert rows.expert_start.tolist() == start and rows.pair_row[:18].tolist() == pair_row
    assert rows.pair_row[18:].tolist() == [-7] * 62  # behind this call's pairs: as it was
    rows.sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    assert rows.expert_start.tolist() == [0] * 7
    assert rows.combine(torch.empty((0, 16), dtype=BF16, device="cuda")).shape == (0, 16)


# ---------------------------------------------------------------------------------
# rows out and back
# ---------------------------------------------------------------------------------

ROW_CASES = [  # T, k, E, C, dropped
    (1, 1, 1, 1, 0.0), (1, 8, 256, 7168, 0.0), (3, 9, 16, 40, 0.3), (5, 32, 40, 2047, 0.2), (33, 6, 8, 128, 0.0),
    (70, 2, 4, 1002, 1.0), (600, 8, 32, 24, 0.1), (517, 1, 3, 6, 0.1)]


@pytest.mark.parametrize("dtype,y_dtype", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("T,k,E,C,dropped", ROW_CASES)
def test_rows(T, k, E, C, dropped, dtype, y_dtype):
    say(f"rows T={T} k={k} C={C} {dtype} {y_dtype}")
    g = gen(T + 7 * k + C)
    ids = routing(g, T, k, E, dropped)
    rows = ExpertRows(E, k, T)
    rows.sort(ids.cuda())
    pair_row = rows.pair_row.cpu()
    named = pair_row[pair_row >= 0].long()
    x = randn(g, T, C, dtype=dtype)
    xs = torch.full((T * k, C), -3.0, dtype=dtype, device="cuda")
    rows.gather(x.cuda(), xs)
    want = torch.full((T * k, C), -3.0, dtype=dtype)
    want[named] = x[torch.nonzero(pair_row >= 0).view(-1) // k]
    assert torch.equal(xs.cpu(), want)

    # what dropped pairs and unnamed rows hold must not matter
    o = torch.full((T * k, C), float("nan"), dtype=dtype)
    o[named] = randn(g, len(named), C, dtype=dtype)
    w = torch.rand(T, k, generator=g)
    w[ids < 0] = float("nan")
    res = randn(g, T, C, dtype=y_dtype)
    for wt in (w, None):
        for r in (res, None):
            out = torch.empty((T, C), dtype=y_dtype, device="cuda")
            rows.combine(o.cuda(), None if wt is None else wt.cuda(), None if r is None else r.cuda(), out)
            y, b = ref.combine64(o, pair_row, wt, r, T, k, y_dtype)
            ref.check(out, y, b, "combine")
    inplace = res.cuda()
    rows.combine(o.cuda(), w.cuda(), inplace, inplace)
    y, b = ref.combine64(o, pair_row, w, res, T, k, y_dtype)
    ref.check(inplace, y, b, "combine in place")

    dy = randn(g, T, C, dtype=y_dtype)
    for wt in (w, None):
        drows = torch.full((T * k, C), -3.0, dtype=dtype, device="cuda")
        _, dw = rows.combine_backward(dy.cuda(), None if wt is None else wt.cuda(), o.cuda(), drows)
        d, bd, nm, v, bv = ref.combine_backward64(dy, pair_row, wt, o, T, k)
        untouched = torch.ones(T * k, dtype=torch.bool)
        untouched[nm] = False
        d[untouched] = -3.0
        ref.check(drows, d, bd, "drows")
        ref.check(dw, v, bv, "dw")
    dx = rows.gather_backward(o.cuda())
    y, b = ref.combine64(o, pair_row, None, None, T, k, dtype)
    ref.check(dx, y, b, "dx")


def test_combine_backward_of_one_output_alone():
    say("combine backward: drows alone, dw alone")
    T, k, C = 6, 3, 72
    rows = ExpertRows(4, k, T)
    rows.sort(routing(gen(1), T, k, 4).cuda())
    g = gen(2)
    o, dy, w = randn(g, T * k, C).cuda(), randn(g, T, C).cuda(), torch.rand(T, k, generator=g).cuda()
    both, dw = rows.combine_backward(dy, w, o)
    only, alone = torch.zeros_like(both), torch.zeros_like(dw)
    st = torch.cuda.current_stream().cuda_stream
    _lib.combine_rows_backward(dy.data_ptr(), _lib.F32, T, k, C, rows.pair_row.data_ptr(), w.data_ptr(), 0, _lib.F32,
                               only.data_ptr(), 0, st)
    _lib.combine_rows_backward(dy.data_ptr(), _lib.F32, T, k, C, rows.pair_row.data_ptr(), w.data_ptr(), o.data_ptr(),
                               _lib.F32, 0, alone.data_ptr(), st)
    assert torch.equal(both, only) and torch.equal(dw, alone)


# ---------------------------------------------------------------------------------
# the dense product
# ---------------------------------------------------------------------------------

LINEAR_CASES = [  # M, K, N, start (None: one matrix), act, dtype, y_dtype, bias, residual
    (1, 1, 1, None, "none", BF16, F32, False, False),
    (1, 256, 128, None, "swiglu", BF16, BF16, True, True),
    (1, 7168, 48, None, "swiglu", BF16, F32, False, False),
    (3, 40, 17, None, "gelu", BF16, BF16, True, False),
    (16, 512, 64, None, "silu", BF16, F32, True, True),
    (17, 72, 33, None, "swiglu", BF16, BF16, True, True),
    (64, 1000, 130, None, "none", BF16, BF16, False, True),
    (65, 333, 100, None, "silu", BF16, F32, True, True),
    (129, 200, 257, None, "swiglu", BF16, F32, True, False),
    (200, 1024, 64, None, "gelu", BF16, BF16, True, True),   # few tiles
    (300, 2056, 31, None, "swiglu", BF16, BF16, True, True),  # few tiles: the contraction is split forward
    (300, 136, 520, None, "none", BF16, BF16, True, True),
    (1, 100, 40, None, "swiglu", F32, F32, True, True),
    (77, 130, 67, None, "gelu", F32, F32, True, True),
    (200, 513, 96, None, "swiglu", F32, BF16, False, True),
    (140, 1024, 40, None, "silu", F32, F32, True, False),
    (9, 64, 48, [0, 0, 4, 4, 9], "swiglu", BF16, BF16, True, True),
    (70, 128, 40, [0, 1, 1, 30, 64], "silu", BF16, F32, True, True),      # six rows in no group
    (300, 96, 136, [0, 150, 150, 299], "none", BF16, BF16, True, False),
    (500, 264, 72, [3, 130, 259, 259, 400, 490], "swiglu", BF16, F32, True, True),  # rows before the first, too
    (40, 33, 21, [0, 7, 7, 40], "gelu", F32, F32, True, True),
    (130, 64, 24, [0, 130], "swiglu", BF16, BF16, True, False),
    (20, 64, 24, [0] * 71, "none", BF16, BF16, False, False),             # every group empty
    (260, 64, 40, list(range(0, 261, 2)), "silu", BF16, F32, True, False),  # 130 groups of two rows
    (130, 2000, 70, [0, 3, 40, 40, 121], "swiglu", BF16, BF16, True, True),  # a split contraction of grouped rows
    (300, 2048, 40, [2, 150, 299], "swiglu", F32, F32, True, True),          # the same in fp32
    (700, 1001, 333, [0, 100, 357, 613, 700], "gelu", BF16, BF16, True, True),
    # large enough for the large tiles, in each product, with short last tiles and odd widths
    (4500, 264, 1100, [7, 1500, 1501, 4490], "swiglu", BF16, BF16, True, True),
    (4099, 2056, 2050, None, "none", BF16, F32, True, True),
    (300, 4100, 4104, None, "silu", BF16, BF16, True, False),
    (2060, 4104, 300, None, "gelu", BF16, BF16, True, True),
    (4099, 200, 2053, None, "swiglu", BF16, F32, False, True),
    (2500, 1000, 1200, None, "none", F32, F32, True, True),
]


def linear_inputs(M, K, N, start, act, dtype, y_dtype, bias, residual, seed=0):
    g = gen(seed + M + K + N)
    R = 2 * N if act == "swiglu" else N
    lead = () if start is None else (len(start) - 1,)
    x = randn(g, M, K, dtype=dtype)
    w = randn(g, *lead, R, K, dtype=dtype, scale=1.5 / K ** 0.5)
    b = randn(g, *lead, R, scale=0.5) if bias else None
    r = randn(g, M, N, dtype=y_dtype) if residual else None
    return g, R, x, w, b, r


def outside(M, start):
    """Which rows belong to no group."""
    out = torch.zeros(M, dtype=torch.bool)
    if start is not None:
        out[:start[0]] = True
        out[start[-1]:] = True
    return out


def cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("M,K,N,start,act,dtype,y_dtype,bias,residual", LINEAR_CASES)
def test_linear_forward(M, K, N, start, act, dtype, y_dtype, bias, residual):
    say(f"linear M={M} K={K} N={N} {act} {dtype}")
    lim = 1.25 if act == "swiglu" and M % 2 else 0.0
    g, R, x, w, b, r = linear_inputs(M, K, N, start, act, dtype, y_dtype, bias, residual)
    none = outside(M, start)
    x[none] = float("nan")  # rows in no group are not looked at
    lin = Linear(w.cuda(), cuda(b), act=act, swiglu_limit=lim, max_rows=M)
    gs = None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
    out = torch.full((M, N), -3.0, dtype=y_dtype, device="cuda")
    z = torch.full((M, R), -3.0, dtype=dtype, device="cuda")
    lin.forward(x.cuda(), gs, cuda(r), out, z)
    y, by, zz, bz = ref.linear_forward64(x, w, b, start, act, lim, r, y_dtype, dtype)
    y[none], zz[none] = -3.0, -3.0
    ref.check(out, y, by, "y")
    ref.check(z, zz, bz, "z")
    again = torch.full((M, N), -3.0, dtype=y_dtype, device="cuda")
    lin.forward(x.cuda(), gs, cuda(r), again)
    assert torch.equal(out, again)  # (z is not needed for y, and the same call gives the same bits)
    if r is not None:
        same = r.cuda()
        lin.forward(x.cuda(), gs, same, same)
        keep = ~none
        assert torch.equal(same.cpu()[keep], out.cpu()[keep])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", [3, 5, 9, 15, 17, 31, 33, 63, 65, 255, 1001, 2047, 4102])
def test_few_rows_of_odd_widths(K, dtype):
    """Rows whose last 16 bytes overlap the 16 before them: every value counts once, and an infinity in one of the
    last values stays one (the values left out there are not multiplied by zero)."""
    say(f"few rows K={K} {dtype}")
    for M, N, act in ((1, 33, "swiglu"), (16, 21, "none")):
        g, R, x, w, b, r = linear_inputs(M, K, N, None, act, dtype, F32, True, True)
        lin = Linear(w.cuda(), b.cuda(), act=act, max_rows=M)
        out, z = torch.empty((M, N), device="cuda"), torch.empty((M, R), dtype=dtype, device="cuda")
        lin.forward(x.cuda(), None, r.cuda(), out, z)
        y, by, zz, bz = ref.linear_forward64(x, w, b, None, act, 0.0, r, F32, dtype)
        ref.check(out, y, by, "y")
        ref.check(z, zz, bz, "z")
    w[:, max(0, K - 8):] = 0.5
    for m in range(8):
        x[m, max(0, K - 1 - m)] = float("inf")
    y = Linear(w.cuda(), max_rows=M).forward(x.cuda(), out=torch.empty((M, N), device="cuda")).cpu()
    assert (y[:8] == float("inf")).all() and torch.isfinite(y[8:]).all()


@pytest.mark.parametrize("M,K,N,start,act,dtype,y_dtype,bias,residual", LINEAR_CASES)
def test_linear_backward(M, K, N, start, act, dtype, y_dtype, bias, residual):
    say(f"linear backward M={M} K={K} N={N} {act} {dtype}")
    lim = 1.25 if act == "swiglu" and M % 2 else 0.0
    g, R, x, w, b, _ = linear_inputs(M, K, N, start, act, dtype, y_dtype, True, False)
    z = randn(g, M, R, dtype=dtype, scale=1.5)
    dy = randn(g, M, N, dtype=y_dtype)
    none = outside(M, start)
    x[none], dy[none], z[none] = float("nan"), float("nan"), float("nan")
    lin = Linear(w.cuda(), b.cuda(), act=act, swiglu_limit=lim, max_rows=M, backward=True)
    gs = None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
    dx = torch.full((M, K), -3.0, dtype=dtype, device="cuda")
    dw = torch.full(w.shape, -3.0, dtype=dtype, device="cuda")
    db = torch.full(w.shape[:-1], -3.0, device="cuda")
    zc = None if act == "none" else z.cuda()
    lin.backward(x.cuda(), dy.cuda(), zc, gs, dx, dw, db)
    want = ref.linear_backward64(x, w, start, act, lim, z, dy, dtype)
    want["dx"][0][none] = -3.0
    for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
        ref.check(got, *want[name], name)
    for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):  # each alone, the same bits
        alone = torch.full_like(got, -3.0)
        lin.backward(x.cuda(), dy.cuda(), zc, gs, **{name: alone})
        assert torch.equal(alone, got), name


def test_linear_fewer_rows_than_made_for_and_none():
    say("linear: every number of rows up to 70 on one workspace; none")
    K, N, M = 264, 40, 70
    g, R, x, w, b, r = linear_inputs(M, K, N, None, "swiglu", BF16, F32, True, True)
    lin = Linear(w.cuda(), b.cuda(), act="swiglu", max_rows=M, backward=True)
    y, by, _, _ = ref.linear_forward64(x, w, b, None, "swiglu", 0.0, r, F32, BF16)
    for m in range(0, M + 1, 3):
        out = lin.forward(x[:m].cuda(), residual=r[:m].cuda())
        ref.check(out, y[:m], by[:m], f"{m} rows")
    dw, db = torch.full(w.shape, -3.0, dtype=BF16, device="cuda"), torch.full((R,), -3.0, device="cuda")
    none = x[:0].cuda()
    lin.backward(none, torch.empty((0, N), device="cuda"), torch.empty((0, R), dtype=BF16, device="cuda"), dw=dw, dbias=db)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_special_values_stay_in_their_rows(dtype):
    """Infinities and NaN in one row (or one group's weights) reach that row's outputs only."""
    say(f"linear: special values {dtype}")
    M, K, N, start = 150, 200, 72, [0, 60, 61, 140, 150]
    g, R, x, w, b, _ = linear_inputs(M, K, N, start, "silu", dtype, F32, True, False)
    x[60, 3], x[139, 0], x[141, 199] = float("nan"), float("inf"), float("-inf")
    z, dy = randn(g, M, R, dtype=dtype), randn(g, M, N)
    lin = Linear(w.cuda(), b.cuda(), act="silu", max_rows=M, backward=True)
    gs = torch.tensor(start, dtype=torch.int32, device="cuda")
    y = lin.forward(x.cuda(), gs, out=torch.empty((M, N), device="cuda")).cpu()
    clean = torch.ones(M, dtype=torch.bool)
    clean[[60, 139, 141]] = False
    assert torch.isfinite(y[clean]).all() and y[60].isnan().all()
    want, by, _, _ = ref.linear_forward64(x, w, b, start, "silu", 0.0, None, F32, dtype)
    ref.check(y[clean], want[clean], by[clean], "clean rows")
    dw = torch.empty_like(w).cuda()
    lin.backward(x.cuda(), dy.cuda(), z.cuda(), gs, dw=dw)
    dw = dw.cpu()
    assert torch.isfinite(dw[0]).all()                       # the group before the bad rows
    assert dw[1][:, 3].isnan().all() and torch.isfinite(dw[1][:, :3]).all()
    assert torch.isfinite(dw[2][:, 1:]).all() and not torch.isfinite(dw[2][:, 0]).any()
    assert torch.isfinite(dw[3][:, :199]).all() and not torch.isfinite(dw[3][:, 199]).any()


def test_clamp_border_has_the_value_and_the_gradient():
    say("swiglu clamp at its border")
    lim = 2.0
    z = torch.tensor([[2.0, 2.0, 2.0156, -300.0, 300.0, 1.0], [2.0, 2.0156, 1.0, 1.0, -2.0, -2.0156]]).reshape(1, 12)
    w = torch.zeros(12, 8)
    lin = Linear(w.cuda(), act="swiglu", swiglu_limit=lim, max_rows=1, backward=True)
    dy, x, db = torch.ones(1, 6).cuda(), torch.ones(1, 8).cuda(), torch.empty(12).cuda()
    lin.backward(x, dy, z.cuda(), dbias=db)
    f, e = ref.act_grad64(z.double(), "swiglu", lim)
    ref.check(db, f[0], e[0] + 4 * ref.U * f[0].abs(), "gradient")
    assert db[2] == 0 and db[4] == 0 and db[7] == 0 and db[11] == 0 and db[0] != 0 and db[10] != 0


def test_gradients_are_differences():
    """<gradient, d> against differences of the 64-bit forward along d (central: the error is a third
    derivative times step^2, far below the fp32 bound here)."""
    say("linear: gradients against differences")
    M, K, N, start = 30, 24, 20, [0, 11, 11, 30]
    for act in ("none", "silu", "gelu", "swiglu"):
        g, R, x, w, b, _ = linear_inputs(M, K, N, start, act, F32, F32, True, False, seed=5)
        dy = randn(g, M, N)
        lin = Linear(w.cuda(), b.cuda(), act=act, max_rows=M, backward=True)
        gs = torch.tensor(start, dtype=torch.int32, device="cuda")
        z = torch.empty((M, R), device="cuda")
        lin.forward(x.cuda(), gs, z=z)
        dx, dw, db = torch.empty_like(x).cuda(), torch.empty_like(w).cuda(), torch.empty_like(b).cuda()
        lin.backward(x.cuda(), dy.cuda(), z, gs, dx, dw, db)
        h = 2.0 ** -13

        def f(x64, w64, b64):
            return (ref.linear_forward64(x64, w64, b64, start, act, 0.0, None, F32, F32)[0] * dy.double()).sum().item()

        args = [x.double(), w.double(), b.double()]
        for i, grad in enumerate((dx, dw, db)):
            d = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + h * d, args[i] - h * d
            want = (f(*up) - f(*down)) / (2 * h)
            got = (grad.double().cpu() * d).sum().item()
            size = (grad.double().cpu() * d).abs().sum().item()
            # each gradient element is off by < 2^-18 of its terms' size here; h^2 d^3 terms stay below 1e-5 of it
            assert abs(got - want) <= 2e-5 * max(size, 1.0), (act, i, got, want, size)


def test_offsets_beyond_32_bits():
    say("rows and products over more than 4 GiB")
    T, k, C = 40000, 8, 8192  # 5.2 GB of rows
    rows = ExpertRows(16, k, T)
    ids = torch.randint(0, 16, (T, k), dtype=torch.int32, device="cuda")
    rows.sort(ids)
    x = torch.randn(T, C, device="cuda").to(BF16)
    xs = rows.gather(x)
    at = rows.pair_row.view(T, k)[-3:].long()
    assert int(rows.row_pair[-1]) >= 0 and torch.equal(xs[-1], x[rows.row_pair[-1].long() // k])
    assert torch.equal(xs[at[2]], x[-1:].expand(k, C))
    y = rows.combine(xs, out=torch.empty((T, C), device="cuda"))
    assert torch.equal(y[-1], x[-1].float() * k)  # (eight equal bf16 values add up exactly)
    N = 24
    w = torch.randn(16, N, C, device="cuda").to(BF16) / 64
    lin = Linear(w, max_rows=T * k, backward=True)
    z = lin.forward(xs, rows.expert_start, out=torch.empty((T * k, N), device="cuda"))
    for r in (0, T * k // 2, T * k - 1):
        e = int((rows.expert_start[1:] <= r).sum())
        want, by, _, _ = ref.linear_forward64(xs[r:r + 1].cpu(), w[e].cpu(), None, None, "none", 0.0, None, F32, BF16)
        ref.check(z[r:r + 1], want, by, f"row {r}")
    dy = torch.randn(T * k, N, device="cuda").to(BF16)
    lin.backward(xs, dy, group_start=rows.expert_start, dx=xs)  # (x is not read for dx)
    for r in (0, T * k - 1):
        e = int((rows.expert_start[1:] <= r).sum())
        want = ref.linear_backward64(torch.zeros(1, C), w[e].cpu(), None, "none", 0.0, None, dy[r:r + 1].cpu(), BF16)["dx"]
        ref.check(xs[r:r + 1], *want, f"dx row {r}")


# ---------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------

def experts64(x, ids, w, w1, w2, lim):
    """y, and its gradients by torch, in 64 bits, of the routed-expert step."""
    x, w, w1, w2 = (t.double().requires_grad_() for t in (x, w, w1, w2))
    T, k = ids.shape
    inter = w2.shape[2]
    y = []
    for t in range(T):
        acc = torch.zeros(x.shape[1], dtype=torch.float64)
        for i in range(k):
            e = int(ids[t, i])
            if e < 0:
                continue
            z = w1[e] @ x[t]
            gate, up = z[:inter], z[inter:]
            if lim > 0:
                gate, up = gate.clamp(max=lim), up.clamp(-lim, lim)
            acc = acc + w[t, i] * (w2[e] @ (gate * torch.sigmoid(gate) * up))
        y.append(acc)
    return torch.stack(y), (x, w, w1, w2)


@pytest.mark.parametrize("dtype,lim", [(F32, 0.0), (F32, 1.0), (BF16, 0.0)])
def test_experts_step_and_its_gradients(dtype, lim):
    """The whole step and back.  In fp32 the result is held to 1e-5 of the largest value (sums of at
    most 96 terms three deep: 3 * 96 * 2^-23 = 3.4e-5 of the sums of sizes, which exceed the values'
    norm).  In bf16 six tensors between are rounded (xs exactly, z, h, o; do, dh, dz): at most
    2^-8 each, on sums of random signs; 6 * 2^-8 of a tensor's norm bounds what they add."""
    say(f"experts step {dtype} {lim}")
    T, H, I, E, k = 37, 96, 64, 7, 3
    g = gen(11)
    x = randn(g, T, H, dtype=dtype)
    w1, w2 = randn(g, E, 2 * I, H, dtype=dtype, scale=H ** -0.5), randn(g, E, H, I, dtype=dtype, scale=I ** -0.5)
    ids = routing(g, T, k, E, dropped=0.1)
    ids[5] = -1  # a token without experts
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    dy = randn(g, T, H)
    y64, leaves = experts64(x, ids, w, w1, w2, lim)
    y64.backward(dy.double())
    step = DenseExperts(w1.cuda(), w2.cuda(), k, T, swiglu_limit=lim, backward=True)
    xc, idc, wc = x.cuda(), ids.cuda(), w.cuda()
    y = step.forward(xc, idc, wc, keep=True)
    dx, dw = torch.empty_like(xc), torch.empty_like(wc)
    dw1, dw2 = torch.empty_like(w1).cuda(), torch.empty_like(w2).cuda()
    step.backward(dy.cuda(), dx, dw, dw1, dw2)
    tol = 4e-5 if dtype is F32 else 6 * 2.0 ** -8
    for name, got, want in (("y", y, y64.detach()), ("dx", dx, leaves[0].grad), ("dw", dw, leaves[1].grad),
                            ("dw1", dw1, leaves[2].grad), ("dw2", dw2, leaves[3].grad)):
        off = (got.double().cpu() - want).norm() / want.norm()
        say(f"  {name}: {off:.2e}")
        assert off <= tol, (name, off)
    assert not y[5].any() and not dx[5].any() and not dw[5].any()
    base = torch.ones(T, H, device="cuda")
    added = step.forward(xc, idc, wc, base, add=True)
    assert added is base and torch.allclose(base, y + 1, atol=1e-6)


def test_graph_replays_match_eager_runs():
    """The step and its gradients captured into one graph: every replay, on new inputs and with eager work of
    the same objects between, gives the eager results' bits."""
    say("experts step in a graph")
    T, H, I, E, k = 29, 128, 96, 9, 4
    g = gen(5)
    w1, w2 = randn(g, E, 2 * I, H, dtype=BF16, scale=0.1).cuda(), randn(g, E, H, I, dtype=BF16, scale=0.1).cuda()
    step = DenseExperts(w1, w2, k, T, backward=True)
    x, dy = torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(T, H, device="cuda")
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    y, dx, dw = torch.empty(T, H, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    dw1, dw2 = torch.empty_like(w1), torch.empty_like(w2)

    def fill(seed):
        s = gen(seed)
        x.copy_(randn(s, T, H)); dy.copy_(randn(s, T, H)); w.copy_(torch.rand(T, k, generator=s))
        ids.copy_(routing(s, T, k, E, dropped=0.1))

    def run():
        step.forward(x, ids, w, y, keep=True)
        step.backward(dy, dx, dw, dw1, dw2)

    fill(0)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(1, 5):
        fill(seed)
        run()
        want = [t.clone() for t in (y, dx, dw, dw1, dw2)]
        for t in (y, dx, dw, dw1, dw2):
            t.fill_(-3.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((y, dx, dw, dw1, dw2), want):
            assert torch.equal(a, b)


def test_on_another_stream():
    say("experts step on a side stream")
    T, H, I, E, k = 21, 64, 32, 5, 2
    g = gen(8)
    w1, w2 = randn(g, E, 2 * I, H, dtype=BF16, scale=0.1).cuda(), randn(g, E, H, I, dtype=BF16, scale=0.1).cuda()
    step, other = DenseExperts(w1, w2, k, T), DenseExperts(w1, w2, k, T)
    x, ids, w = randn(g, T, H, dtype=BF16).cuda(), routing(g, T, k, E).cuda(), torch.rand(T, k, generator=g).cuda()
    want = step.forward(x, ids, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = other.forward(x, ids, w)
    step.forward(x, ids, w)
    s.synchronize()
    assert torch.equal(got, want)


def test_two_products_at_once():
    """Two objects on two streams, large enough to overlap, with and without a split contraction: each gives
    what it gives alone."""
    say("two products at once")
    g = gen(21)
    cases = []
    for M, K, N, act in ((1500, 512, 1024, "swiglu"), (96, 4096, 256, "gelu")):
        R = 2 * N if act == "swiglu" else N
        w = randn(g, R, K, dtype=BF16, scale=K ** -0.5).cuda()
        x, dy = randn(g, M, K, dtype=BF16).cuda(), randn(g, M, N, dtype=BF16).cuda()
        lin = Linear(w, act=act, max_rows=M, backward=True)
        new = lambda: (torch.empty(M, N, dtype=BF16, device="cuda"), torch.empty(M, R, dtype=BF16, device="cuda"),  # noqa: E731
                       torch.empty_like(x), torch.empty_like(w))
        cases.append((lin, x, dy, new(), new()))

    def run(c, out):
        lin, x, dy = c[:3]
        y, z, dx, dw = out
        lin.forward(x, out=y, z=z)
        lin.backward(x, dy, z, dx=dx, dw=dw)

    for c in cases:
        run(c, c[3])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                run(c, c[4])
    torch.cuda.synchronize()
    for c in cases:
        for a, b in zip(c[3], c[4]):
            assert torch.equal(a, b)


def test_same_routing_as_the_coded_step():
    """The unquantised layer behind Step.route: the experts' own decoded weights give the coded
    step's output (held to the coded step's own tolerance, 1e-2 of the largest value, plus bf16
    roundings of h and o that the coded step does not make: 2 * 2^-8 of the sums' sizes)."""
    import numpy as np

    import oracle
    import synth
    from bit_vector_quantised_amd.layer import DeviceLayer, Step
    from gpu_util import x_tensor
    say("unquantised step behind Step.route")
    syn = synth.SynthLayer(synth.Config("dense", 6, 256, 128, 8, 2, "bf16", "normal", seed=99))
    dev = DeviceLayer.from_synth(syn)
    step = Step(dev, 6)
    x = x_tensor(syn.x(), "bf16")
    y = step.forward(x).clone()
    mats = [oracle.decode_expert(syn.expert(e), syn.codebook) for e in range(8)]
    w1 = torch.from_numpy(np.stack([np.concatenate((m[0], m[1])) for m in mats])).to(BF16).cuda()
    w2 = torch.from_numpy(np.stack([m[2] for m in mats])).to(BF16).cuda()
    dense = DenseExperts(w1.contiguous(), w2.contiguous(), 2, 6)
    got = dense.forward(x, step.ids[:6], step.w[:6])
    off = (got - y).abs().amax(1) / y.abs().amax(1)
    say(f"  off {off.max().item():.2e}")
    # the decoded weights are rounded to bf16 here (2^-8 each, random over sums of 128 and more terms)
    assert off.max() <= 1e-2 + 4 * 2.0 ** -8
