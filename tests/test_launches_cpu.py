"""A launch that fails is reported by its call, whichever of the call's launches it is (without a GPU: launches.py)."""
import pytest

import launches

pytest.importorskip("bit_vector_quantised_amd")

# Addresses far apart, which nothing looks at; a table of groups, x and z in 8 bits or as they are.
CALLS = r"""
A, B, C, D, E, F, G, H, I, J = (i << 38 for i in range(1, 11))
r8 = lambda q: ctypes.byref(_lib.Rows8Desc(q, q + (1 << 36)))
def linear(n_in, n_out, act, dtype, groups=1, bias=True):
    return ctypes.byref(_lib.LinearDesc(n_in, n_out, groups, act, dtype, 0.0, A, B if bias else None))
def back8(lin, M, gs, x8, z8, dx=F, db=H):
    return (raw.moe_vq_linear_backward8, lin, None if x8 else C, r8(C) if x8 else None, M, gs, None if z8 else D, r8(D) if z8 else None,
            E, _lib.BF16, dx, G, db, I, 1 << 34, None)
def back(lin, M, gs):
    return (raw.moe_vq_linear_backward, lin, C, M, gs, D, E, _lib.BF16, F, G, H, I, 1 << 34, None)
def forward(lin, M, gs):
    return (raw.moe_vq_linear_forward, lin, C, M, gs, None, E, _lib.F32, D, I, 1 << 34, None)
S, N = _lib.ACT_SWIGLU, _lib.ACT_NONE
choice = ctypes.byref(_lib.Choice(256, 8, 1, 8, 4, 2, 1, 1.0, B))
SETS = {
    "rows in 8 bits": [(raw.moe_vq_rows8_pack, A, _lib.BF16, 100, 64, None, 0, r8(B), None),
                       (raw.moe_vq_rows8_unpack, r8(B), 100, 64, None, 0, A, _lib.BF16, None),
                       (raw.moe_vq_rows8_unpack, r8(B), 2000000, 8000, None, 0, A, _lib.F32, None),  # (several launches)
                       (raw.moe_vq_gather_rows8, r8(B), 10, 4, 64, A, C, _lib.F32, None),
                       (raw.moe_vq_act_backward8, r8(B), S, 0.0, 10, 4, 64, A, C, D, _lib.BF16, E, F, _lib.BF16, G, None)],
    "norm": [(raw.moe_vq_norm_forward, A, _lib.BF16, None, None, _lib.BF16, 9, 100, B, 1e-6, C, _lib.BF16, None, None),
             (raw.moe_vq_norm_backward, A, _lib.BF16, 9, 100, B, 1e-6, C, None, _lib.BF16, None, D, _lib.BF16, E, F, 1 << 20, None)],
    "choice": [(raw.moe_vq_choose, choice, A, 9, C, D, None), (raw.moe_vq_choose_backward, choice, A, 9, C, D, E, None)],
    "product": [forward(linear(64, 48, S, _lib.BF16), 300, None), forward(linear(2304, 40, N, _lib.BF16), 300, None),
                back(linear(64, 48, S, _lib.BF16), 300, None), back(linear(2304, 40, N, _lib.F32), 300, None),
                back(linear(4096, 4096, S, _lib.BF16, 4), 8192, J)],
    "gradients from 8 bits": [back8(linear(64, 48, S, _lib.BF16), 300, None, x, z) for x, z in ((True, True), (True, False), (False, True))]
        + [back8(linear(1000, 333, _lib.ACT_GELU, _lib.F32), 515, None, True, True), back8(linear(4096, 4096, S, _lib.BF16, 4), 8192, J, True, True),
           back8(linear(64, 48, N, _lib.BF16), 300, None, True, False), back8(linear(63, 48, S, _lib.BF16), 300, None, True, True, None, None)],
}
for one in SETS[SET]:
    status, kernels = call(*one)
    for i in range(len(kernels)):
        call(*one, fails_at=i + 1)
"""


@pytest.mark.parametrize("calls", ["rows in 8 bits", "norm", "choice", "product", "gradients from 8 bits"])
def test_a_launch_that_fails_is_reported(tmp_path, calls):
    from bit_vector_quantised_amd import _lib
    results = launches.run(tmp_path, f"SET = {calls!r}\n" + CALLS)
    i = 0
    while i < len(results):
        status, kernels = results[i]
        assert status == _lib.OK and kernels
        for n in range(len(kernels)):
            assert results[i + 1 + n][0] == _lib.EHIP, (n, [k[0] for k in kernels])
        i += 1 + len(kernels)


def test_no_rows_in_8_bits(tmp_path):
    """Gradients of no rows, whose buffers in 8 bits are empty (null): zeros, as those of plain tensors without rows."""
    from bit_vector_quantised_amd import _lib
    results = launches.run(tmp_path, r"""
A, D, E, F, G = (i << 38 for i in range(1, 6))
lin = ctypes.byref(_lib.LinearDesc(64, 48, 1, _lib.ACT_SWIGLU, _lib.BF16, 0.0, A, D))
none = ctypes.byref(_lib.Rows8Desc(None, None))
call(raw.moe_vq_linear_backward, lin, None, 0, None, None, None, _lib.BF16, None, E, F, G, 1 << 34, None)
call(raw.moe_vq_linear_backward8, lin, None, none, 0, None, None, none, None, _lib.BF16, None, E, F, G, 1 << 34, None)
call(raw.moe_vq_linear_backward8, lin, None, none, 1, None, None, none, A, _lib.BF16, None, E, F, G, 1 << 34, None)
""")
    (plain, kernels), (status, same), (refused, nothing) = results
    assert plain == status == _lib.OK and kernels and same == kernels
    assert refused == _lib.EINVAL and not nothing
