"""Calls of the operators around the experts at their edges, each against a 64-bit plain form or against a call that it must
equal to the bit."""
import math

import pytest
import torch

import block_ref as ref
import dense_ref
from bit_vector_quantised_amd.block import ExpertChoice

from gpu_util import say
from test_gpu_dense import gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(16, 6), (200, 8), (256, 20), (700, 8)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_at_experts_that_the_bias_turns_off(score, renorm, E, k):
    """An id that names an expert whose bias (or logit) is -inf or NaN has no part: its place is as one of id -1."""
    say(f"choice gradient, experts off by the bias E={E} k={k} {score} renorm={renorm}")
    g = gen(E + k)
    T = 23
    logits, bias, dw = randn(g, T, E, scale=2.0), 0.1 * randn(g, E), randn(g, T, k)
    off = torch.randperm(E, generator=g)[:E // 4]
    bias[off[::2]], bias[off[1::2]] = -math.inf, math.nan
    logits[:, off[0]] = 30.0  # (far above the others that are on)
    logits[3, 1], logits[4, 2] = -math.inf, math.nan
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    ids[:, 0] = off[0]
    ids[5] = off[:k] if len(off) >= k else off[0]  # nothing but experts that are off
    on = (bias[ids.long()] > -math.inf)
    assert (~on).sum() > T and on.any()
    choice = ExpertChoice(E, k, score, bias.cuda(), renorm=renorm, scale=1.7)
    got = choice.backward(logits.cuda(), ids.cuda(), dw.cuda())
    named = torch.where(on, ids, -1)
    assert torch.equal(got, choice.backward(logits.cuda(), named.cuda(), dw.cuda()))
    assert not got[:, off.cuda()].any()
    dense_ref.check(got, *ref.choose_backward64(logits, bias, named, dw, score, renorm, 1.7), "dlogits")
