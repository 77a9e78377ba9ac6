"""The dense product where its output is cut into large tiles, or its contraction into parts, over groups of unequal
rows: which cut a product takes goes by its sizes, and is stated for each case as side of the tiles x parts."""
import pytest
import torch

import dense_ref as ref
import test_gpu_dense as base
from bit_vector_quantised_amd.dense import Linear
from gpu_util import say
from test_gpu_dense import BF16, F32, linear_inputs, outside, randn

pytestmark = pytest.mark.gpu

CUTS = [  # as test_gpu_dense.LINEAR_CASES                                       forward, dx, dw
    (1300, 72, 300, [3, 200, 1296], "swiglu", F32, F32, True, True),           # 64 x 1, 64 x 2, 64 x 2
    (1700, 40, 520, [0, 0, 1100, 1690], "gelu", F32, BF16, True, False),       # 64 x 1, 64 x 2, 64 x 2
    (700, 300, 1500, [1, 699, 700], "silu", F32, F32, True, True),             # 64 x 1, 64 x 4, 64 x 1
    (5000, 300, 700, [100, 140, 5000], "none", F32, F32, True, True),          # 128 x 1, 64 x 1, 64 x 4
    (3000, 1500, 1500, [0, 1201, 1201, 2990], "silu", F32, F32, False, False),  # 64 x 1, 64 x 1, 128 x 1
    (2700, 72, 1030, [0, 130, 2600, 2600], "swiglu", BF16, BF16, True, True),  # 128 x 1, 64 x 4, 64 x 1
    (1500, 1000, 2100, [0, 0, 1, 1499], "swiglu", BF16, BF16, True, True),     # 128 x 1, 128 x 4, 256 x 1
    (5000, 520, 520, [7, 9, 4990], "silu", BF16, F32, True, True),             # 128 x 1, 128 x 1, 128 x 4
    (9000, 700, 520, [0, 40, 8000, 9000], "swiglu", BF16, BF16, True, False),  # 256 x 1, 128 x 1, 128 x 2
    (4600, 2100, 1100, [9, 300, 300, 4000, 4600], "swiglu", BF16, BF16, True, True),  # 256 x 1, 256 x 1, 128 x 1
    (4600, 2100, 2100, [4, 1500, 1500, 4590], "none", BF16, BF16, True, True),  # 256 x 1, 256 x 1, 256 x 1
    (300, 2056, 600, [0, 17, 300], "gelu", BF16, BF16, True, True),            # 64 x 4, 64 x 1, 128 x 1
    (900, 8200, 520, [0, 500, 501, 900], "silu", BF16, F32, True, True),       # 128 x 8, 256 x 1, 128 x 1
]


@pytest.mark.parametrize("M,K,N,start,act,dtype,y_dtype,bias,residual", CUTS)
def test_forward(M, K, N, start, act, dtype, y_dtype, bias, residual):
    base.test_linear_forward(M, K, N, start, act, dtype, y_dtype, bias, residual)


@pytest.mark.parametrize("M,K,N,start,act,dtype,y_dtype,bias,residual", CUTS)
def test_backward(M, K, N, start, act, dtype, y_dtype, bias, residual):
    base.test_linear_backward(M, K, N, start, act, dtype, y_dtype, bias, residual)


def test_special_values_on_the_largest_tiles():
    """As test_special_values_stay_in_their_rows, on 256 x 256 tiles of groups: infinities and NaN in a group's rows,
    and in rows of no group, reach that row's outputs and that group's gradient only."""
    say("special values, 256 x 256 tiles")
    M, K, N, start = 4600, 2100, 2100, [4, 1500, 1500, 3001, 4590]
    g, R, x, w, b, _ = linear_inputs(M, K, N, start, "none", BF16, BF16, False, False)
    none = outside(M, start)
    dy = randn(g, M, N, dtype=BF16)
    x[none], dy[none] = float("nan"), float("inf")
    x[3000, 17], dy[3001, 2099] = float("inf"), float("nan")  # the last row of one group, the first of the next
    gs = torch.tensor(start, dtype=torch.int32, device="cuda")
    lin = Linear(w.cuda(), max_rows=M, backward=True)
    y = lin.forward(x.cuda(), gs, out=torch.full((M, N), -3.0, dtype=BF16, device="cuda")).cpu()
    dx, dw = torch.full((M, K), -3.0, dtype=BF16, device="cuda"), torch.empty(w.shape, dtype=BF16, device="cuda")
    lin.backward(x.cuda(), dy.cuda(), group_start=gs, dx=dx, dw=dw)
    dx, dw = dx.cpu(), dw.cpu()
    assert (y[none] == -3.0).all() and (dx[none] == -3.0).all()
    rest = torch.ones(M, dtype=torch.bool)
    rest[3000] = False
    assert torch.isfinite(y[rest]).all() and not torch.isfinite(y[3000]).any()
    rest[3000], rest[3001] = True, False
    assert torch.isfinite(dx[rest]).all() and dx[3001].isnan().all()
    assert torch.isfinite(dw[0]).all() and not dw[1].any()
    assert not torch.isfinite(dw[2][:, 17]).any() and torch.isfinite(dw[2][:, torch.arange(K) != 17]).all()
    assert dw[3][2099].isnan().all() and torch.isfinite(dw[3][:2099]).all()


@pytest.mark.parametrize("dtype,K,N", [(BF16, 2304, 40), (F32, 1280, 36), (BF16, 44, 2304), (F32, 30, 1100)])
def test_fewer_rows_on_one_workspace(dtype, K, N):
    """Every size of call on the workspace of the largest, whose contraction (K forward, N for dx) is split into
    parts at many of these sizes; what lies behind the workspace stays as it was."""
    say(f"fewer rows {dtype} {K} {N}")
    M, act = 1100, "silu"
    g, R, x, w, b, r = linear_inputs(M, K, N, None, act, dtype, F32, True, True)
    z, dy = randn(g, M, R, dtype=dtype), randn(g, M, N)
    lin = Linear(w.cuda(), b.cuda(), act=act, max_rows=M, backward=True)
    big = torch.full((lin.ws_bytes + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    lin.ws = big[:lin.ws_bytes]
    y, by, _, _ = ref.linear_forward64(x, w, b, None, act, 0.0, r, F32, dtype)
    for m in (0, 1, 15, 16, 17, 63, 64, 65, 130, 300, 700, M):
        xm, zm, dm = x[:m].cuda(), z[:m].cuda(), dy[:m].cuda()
        ref.check(lin.forward(xm, residual=r[:m].cuda()), y[:m], by[:m], f"{m} rows")
        dx, dw, db = torch.empty_like(xm), torch.empty(w.shape, dtype=dtype, device="cuda"), torch.empty(R, device="cuda")
        lin.backward(xm, dm, zm, dx=dx, dw=dw, dbias=db)
        want = ref.linear_backward64(x[:m], w, None, act, 0.0, z[:m], dy[:m], dtype)
        for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
            ref.check(got, *want[name], f"{name} of {m} rows")
        assert (big[lin.ws_bytes:] == 0xA5).all(), m
