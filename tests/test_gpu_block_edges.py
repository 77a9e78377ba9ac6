"""Calls of the operators around the experts at their edges, each against a 64-bit plain form or against a call that it must
equal to the bit."""
import gc
import math
import weakref

import pytest
import torch

import block_ref as ref
import dense_ref
from bit_vector_quantised_amd.block import ExpertChoice, MoeBlock, RmsNorm, Router
from bit_vector_quantised_amd.dense import DenseExperts, Rows8

from gpu_util import say
from test_gpu_dense import BF16, F32, gen, randn

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


@pytest.mark.parametrize("E,groups", [(4, 2), (60, 5), (320, 5)])
@pytest.mark.parametrize("steps", [(12740, 12740, 624, 624), (15990, 4635, 976, 13613), (522, 522, 12214, 12214)])
def test_groups_whose_roundings_add_up(E, groups, steps):
    """Two groups whose sums of two values differ by less than the roundings of fp32 move them: 64 bits order them.  With
    biases of some 512 values are rounded to h = 2^-14 and sums to 2 h.  The scores lie half way between two steps
    of h, up to a few steps of fp32 logits; where rounding moves one group's two up and the other's two down, their sums
    become 3 h and 1 h (mod 4 h), which rounding to even moves to 4 h and 0: fp32 sees 4 h where hardly
    anything is, and its scores' own errors decide which group that favours."""
    say(f"groups whose roundings add up E={E} {steps}")
    g = gen(E + steps[0])
    T, h, size = 65536, 2.0 ** -14, E // groups
    steps = torch.tensor(steps, dtype=torch.float64)
    score = (steps + 0.5) * h
    l = torch.log(score / (1 - score)).float().repeat(T, 1)
    l = (l.view(torch.int32) + torch.randint(-5, 6, l.shape, generator=g, dtype=torch.int32)).view(F32)  # up to 5 steps away
    b = (512 + (16384 + torch.tensor([0, 4001, 0, 4001]) - steps) * h).float()  # the values: 513 + (0 or 4001, and a half) h
    at = torch.tensor([0, 1, size, size + 1])  # two experts in each of the first two groups
    logits, bias = torch.full((T, E), -8.0), torch.zeros(E)
    logits[:, at], bias[at] = l, b
    value = torch.sigmoid(l.double()) + b.double()
    one, two = value[:, 0] + value[:, 1], value[:, 2] + value[:, 3]
    ids, _ = ExpertChoice(E, 2, "sigmoid", bias.cuda(), groups=groups, top_groups=1).forward(logits.cuda())
    want = torch.where((two > one)[:, None], at[[3, 2]], at[[1, 0]])  # (the one of 4001 steps more comes first)
    told = (one - two).abs() > 1e-11  # 64 bits: values of 513 are off by 2^-44 each, sums by 2^-43
    assert told.sum() > 0.99 * T and torch.equal(ids.cpu().long()[told], want[told])


@pytest.mark.parametrize("C", [64, 500, 1024, 9000])
@pytest.mark.parametrize("eps", [1e-6, 2.0 ** -126, 2.0 ** -129, 2.0 ** -140])
def test_norm_of_rows_of_zeros_by_any_eps(C, eps):
    """Rows of zeros (padding) have s^3 mean(t s) = 0, whatever eps: dx = t / sqrt(eps), dgain nothing."""
    say(f"norm of zeros C={C} eps={eps}")
    g = gen(C)
    M = 5
    s, gain, dy = torch.zeros(M, C), 1 + 0.3 * randn(g, C), randn(g, M, C) * 2.0 ** -20
    s[1], s[3] = randn(g, C), 2.0 ** -64 * randn(g, C)
    norm = RmsNorm(gain.cuda(), eps=eps, max_rows=M, backward=True)
    assert not norm.forward(s.cuda())[[0, 2, 4]].any()
    dx, dg = torch.empty(M, C, device="cuda"), torch.empty(C, device="cuda")
    norm.backward(s.cuda(), dy.cuda(), dx=dx, dgain=dg)
    want = ref.norm_backward64(s, gain, eps, dy, None, None, F32)
    for row in (0, 1, 2, 4):
        dense_ref.check(dx[row], want[0][row], want[1][row], f"dx of row {row}")
    assert torch.isfinite(dx).all() and torch.isfinite(dg).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_columns_behind_the_last_are_zeros(dtype):
    """Also where the row's last block holds an infinity or NaN, which makes its values NaN by the exponent alone; as pack
    and norm write it."""
    say(f"8 bits: columns behind the last, {dtype}")
    g = gen(11)
    for C in (1, 35, 100, 127):
        x = randn(g, 5, C, dtype=dtype)
        x[1, -1], x[2, -1], x[3, -1] = math.inf, -math.inf, math.nan
        r, by_norm = Rows8(5, C), Rows8(5, C)
        r.q.fill_(77)
        by_norm.q.fill_(77)
        r.pack(x.cuda())
        RmsNorm(torch.ones(C, device="cuda"), max_rows=5).forward(x.cuda(), rows8=by_norm, dense=False)
        for rows in (r, by_norm):
            assert (rows.e[1:4, -1] == 255).all() and (rows.q[:, C:] == 0).all()
            got = rows.unpack(out=torch.empty(5, C, dtype=dtype, device="cuda"))
            last = (C - 1) // 32 * 32
            assert got[1:4, last:].isnan().all() and torch.isfinite(got[[0, 4]]).all()


def small_experts(g, T, k, H=64, I=48, E=4, kept8=True, **more):
    w1, w2 = randn(g, E, 2 * I, H, dtype=BF16, scale=H ** -0.5).cuda(), randn(g, E, H, I, dtype=BF16, scale=I ** -0.5).cuda()
    return DenseExperts(w1, w2, k, T, backward=True, kept8=kept8, **more)


@pytest.mark.parametrize("kept8", [False, True])
def test_a_kept_pass_holds_no_tensor_of_its_caller(kept8):
    """What backward needs is kept in the step's own buffers: the caller's x, ids and w may be freed before it."""
    say(f"kept pass, the caller's tensors kept8={kept8}")
    g = gen(21)
    T, k, H, E = 30, 2, 64, 4
    step = small_experts(g, T, k, kept8=kept8)
    inputs = [randn(g, T, H, dtype=BF16).cuda(), torch.randint(0, E, (T, k), generator=g).int().cuda(), torch.rand(T, k, generator=g).cuda()]
    refs = [weakref.ref(t) for t in inputs]
    step.forward(*inputs, keep=True)
    del inputs
    gc.collect()
    assert [r() for r in refs] == [None] * 3
    dy = randn(g, T, H, dtype=BF16).cuda()
    dx, dw = torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(T, k, device="cuda")
    step.backward(dy, dx, dw, torch.empty_like(step.fc1.w), torch.empty_like(step.fc2.w))
    assert dx.any() and dw.any()


def test_a_kept_pass_records_no_graph():
    """Weights that require a gradient leave none in the step's buffers, pass after pass."""
    say("kept pass, weights that require a gradient")
    g = gen(22)
    T, k, H, E = 9, 2, 64, 4
    step = small_experts(g, T, k)
    x, ids = randn(g, T, H, dtype=BF16).cuda(), torch.randint(0, E, (T, k), generator=g).int().cuda()
    results = []
    for leaf in (False, True, True):
        w = torch.full((T, k), 0.5, device="cuda", requires_grad=leaf)
        y = step.forward(x, ids, w, keep=True)
        assert not step.w_kept.requires_grad and step.w_kept.grad_fn is None and not y.requires_grad
        dx, dw = torch.empty_like(x), torch.empty(T, k, device="cuda")
        step.backward(x, dx, dw, torch.empty_like(step.fc1.w), torch.empty_like(step.fc2.w))
        results.append((y, dx, dw))
    for got in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got, results[0]))


@pytest.mark.parametrize("kept8", [False, True])
def test_weights_replaced_between_passes(kept8):
    """A step whose weight tensors are replaced computes with the new ones, forward and back, as one made from them."""
    say(f"weights replaced kept8={kept8}")
    g = gen(23)
    T, k, H, E = 20, 2, 64, 4
    step, other = small_experts(g, T, k, kept8=kept8), small_experts(g, T, k, kept8=kept8)
    x, ids, w = randn(g, T, H, dtype=BF16).cuda(), torch.randint(0, E, (T, k), generator=g).int().cuda(), torch.rand(T, k, generator=g).cuda()
    dy = randn(g, T, H, dtype=BF16).cuda()
    results = []
    step.forward(x, ids, w, keep=True)
    step.fc1.w, step.fc2.w = other.fc1.w.clone(), other.fc2.w.clone()
    for one in (step, other):
        y = one.forward(x, ids, w, keep=True)
        grads = [torch.empty_like(t) for t in (x, w, one.fc1.w, one.fc2.w)]
        one.backward(dy, *grads)
        results.append([y, *grads])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def small_block(g, T, k, H=64, E=4, kept8=True, router=None, step=None):
    step = small_experts(g, T, k, H=H, E=E, kept8=kept8) if step is None else step
    router = Router(randn(g, E, H, dtype=BF16).cuda(), k, T, backward=True) if router is None else router
    return MoeBlock(RmsNorm((1 + 0.2 * randn(g, H)).cuda(), max_rows=T, backward=True), router, step)


def block_gradients(b, s, dy):
    out = [torch.empty_like(s), torch.empty_like(b.norm.gain), torch.empty_like(b.router.linear.w), torch.empty_like(b.experts.fc1.w),
           torch.empty_like(b.experts.fc2.w)]
    b.backward(s, dy, None, *out)
    return out


@pytest.mark.parametrize("kept8", [False, True])
def test_a_block_whose_parts_went_on_refuses(kept8):
    """A kept block goes back through its own pass only: not after its router or its experts have made another one, alone or
    as parts of another block, of as many tokens."""
    say(f"block whose parts went on kept8={kept8}")
    g = gen(24)
    T, k, H, E = 20, 2, 64, 4
    b = small_block(g, T, k, kept8=kept8)
    x, other, dy = (randn(g, T, H, dtype=BF16).cuda() for _ in range(3))
    ids, w = torch.randint(0, E, (T, k), generator=g).int().cuda(), torch.rand(T, k, generator=g).cuda()
    b.forward(x, keep=True)
    want = block_gradients(b, x, dy)
    same_router = small_block(g, T, k, kept8=kept8, router=b.router)
    same_experts = small_block(g, T, k, kept8=kept8, step=b.experts)
    for went_on in (lambda: b.router.forward(other), lambda: b.experts.forward(other, ids, w), lambda: b.experts.forward(other, ids, w, keep=True),
                    lambda: same_router.forward(other, keep=True), lambda: same_experts.forward(other, keep=True),
                    lambda: same_router.forward(other), lambda: same_experts.forward(other)):
        b.forward(x, keep=True)
        went_on()
        for _ in range(2):  # (nor later)
            with pytest.raises(ValueError, match="another pass|kept nothing"):
                block_gradients(b, x, dy)
    b.forward(x, keep=True)
    for a, c in zip(block_gradients(b, x, dy), want):
        assert torch.equal(a, c)


def test_a_refused_block_leaves_no_mixed_pass():
    """The norm writes the experts' rows in 8 bits first: if the router then refuses, a pass that the experts kept before is
    gone."""
    say("refused block")
    g = gen(25)
    T, k, H, E = 20, 2, 64, 4
    b = small_block(g, T, k)
    x, other, dy = (randn(g, T, H, dtype=BF16).cuda() for _ in range(3))
    ids, w = torch.randint(0, E, (T, k), generator=g).int().cuda(), torch.rand(T, k, generator=g).cuda()
    b.experts.forward(x, ids, w, keep=True)
    weights, b.router.linear.w = b.router.linear.w, b.router.linear.w.float()  # (of another type: refused)
    with pytest.raises(ValueError):
        b.forward(other, keep=True)
    b.router.linear.w = weights
    with pytest.raises(ValueError, match="kept nothing"):
        b.experts.backward(dy, torch.empty_like(x), torch.empty_like(w), torch.empty_like(b.experts.fc1.w), torch.empty_like(b.experts.fc2.w))
