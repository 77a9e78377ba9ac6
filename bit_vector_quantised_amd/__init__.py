"""MI355X-native MoE-VQ routed-expert step: a C-ABI HIP library (libmoe_vq.so,
include/moe_vq.h) and its thin Python binding.

Importing this package loads the library; it raises if the library is not built.
"""
from . import _lib  # noqa: F401  (loads libmoe_vq.so, fails loudly if missing)
from ._lib import (ACT_GELU, ACT_NONE, ACT_SILU, ACT_SWIGLU, BF16, EHIP, EINVAL, ENOSPACE, ENOTRESIDENT, EUNSUPPORTED, F32, FMT_ABSENT,  # noqa: F401
                   FMT_MXFP4, FMT_VQ2, MAT_DOWN, MAT_GATE, MAT_UP, OK, SCORE_SIGMOID, SCORE_SOFTMAX, MoeVqError, act_backward8, check,
                   choose, choose_backward,
                   combine_rows, combine_rows_backward, decode_expert, gather_rows, gather_rows8, linear_backward,
                   linear_backward8, linear_bytes, linear_bytes8, linear_forward, norm_backward, norm_bytes, norm_forward,
                   rows8_pack, rows8_pitch, rows8_unpack, sort_bytes, sort_pairs,
                   expert_bytes, fc1_silu, fc2_combine, forward, prefill_gemm, route_topk, slot_layout, step_info, strerror,
                   workspace_bytes)
