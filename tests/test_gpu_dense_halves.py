"""The dense product where the tiles of an XCD's last round run as two halves of their rows: products of 256 x 256 tiles whose
last round holds at most 16 tiles for an XCD.  Which tiles those are goes by the sizes; for each case it is stated how many
are halved, how many of them have all 256 rows, 129 to 255 (the second half is short) and 128 or fewer (it is empty)."""
import pytest

import test_gpu_dense as base
from test_gpu_dense import BF16, F32

SIDE = 256


def halved(start, cols, per_n):
    """Rows of each tile that is halved: rows in groups start, cols output columns of per_n to a tile."""
    count = [(b - a + SIDE - 1) // SIDE for a, b in zip(start, start[1:])]
    nt = -(-cols // per_n)
    tiles, out = sum(count) * nt, []
    for x in range(8):
        mine = tiles // 8 + (x < tiles % 8)
        last = mine % 32 if mine % 32 <= 16 else 0
        for q in range(mine - last, mine):
            at = x * (tiles // 8) + min(x, tiles % 8) + q
            g, before = 0, 0
            while at // nt >= before + count[g]:
                before, g = before + count[g], g + 1
            band, rest = divmod(at - before * nt, 8 * nt)
            row = band * 8 + rest % min(8, count[g] - band * 8)
            out.append(min(SIDE, start[g + 1] - start[g] - row * SIDE))
    return len(out), sum(r == SIDE for r in out), sum(128 < r < SIDE for r in out), sum(r <= 128 for r in out)


# as test_gpu_dense.LINEAR_CASES; (halved tiles forward, of dx), None where the product takes other tiles
CASES = [
    ((1567, 264, 2056, [2, 762, 762, 1441, 1549], "swiglu", BF16, BF16, True, True), (119, 68, 34, 17), None),
    ((2588, 200, 2570, [2, 276, 276, 701, 1341, 2570], "none", BF16, F32, True, True), (64, 50, 11, 3), None),
    ((2658, 2570, 200, [1, 867, 867, 1872, 1925, 2639], "silu", BF16, BF16, True, False), None, (64, 37, 16, 11)),
    ((4496, 1544, 1544, [1, 953, 3725, 3969, 4273, 4489], "none", BF16, BF16, False, True), (48, 20, 21, 7), (48, 20, 21, 7)),
    ((4624, 1544, 776, [2, 212, 212, 3601, 4606], "swiglu", BF16, BF16, True, True), (48, 37, 7, 4), (48, 37, 7, 4)),
    ((3602, 2100, 2100, [3, 1771, 1771, 3529, 3592], "none", BF16, BF16, False, False), (16, 6, 1, 9), (16, 6, 1, 9)),
    # behind a whole round of the XCD's 32 CUs
    ((7100, 200, 2570, [5, 900, 900, 4000, 7090], "silu", BF16, BF16, False, True), (74, 68, 0, 6), None),
    ((6800, 264, 1290, [2, 1500, 1733, 1733, 6790], "swiglu", BF16, F32, True, False), (41, 32, 9, 0), None),
    ((7000, 2570, 264, [5, 2900, 2900, 4000, 6990], "none", BF16, BF16, True, True), None, (63, 57, 3, 3)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case,forward,dx", CASES)
def test_halves(case, forward, dx):
    base.test_linear_forward(*case)
    base.test_linear_backward(*case)


@pytest.mark.parametrize("case,forward,dx", CASES)
def test_cases_are_what_they_are_meant_for(tmp_path, case, forward, dx):
    """Without a GPU: the products take 256 x 256 tiles where the case says so, and so many of them are halved."""
    import launches
    M, K, N, start, act, _, y_dtype, _, _ = case
    if forward:
        assert forward == halved(start, N, SIDE // 2 if act == "swiglu" else SIDE)
    if dx:
        assert dx == halved(start, K, SIDE)
    (status, fwd), (status2, back) = launches.run(tmp_path, f"""
A, B, C, D, E, F, G, H, I, J = (i << 38 for i in range(1, 11))
act = {{"none": _lib.ACT_NONE, "silu": _lib.ACT_SILU, "swiglu": _lib.ACT_SWIGLU}}[{act!r}]
lin = ctypes.byref(_lib.LinearDesc({K}, {N}, {len(start) - 1}, act, _lib.BF16, 0.0, A, B))
call(raw.moe_vq_linear_forward, lin, C, {M}, D, None, E, _lib.BF16, F, G, 1 << 36, None)
call(raw.moe_vq_linear_backward, lin, C, {M}, D, F, E, _lib.BF16, H, None, None, G, 1 << 36, None)
""")
    large = [any("gemm_kernel" in name and "Li256ELi256E" in name for name, _, _ in kernels) for kernels in (fwd, back)]
    assert (status, status2) == (0, 0) and large == [forward is not None, dx is not None]
