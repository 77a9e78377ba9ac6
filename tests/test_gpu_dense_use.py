"""The row operators and the dense product as programs use them: buffers that lie over each
other where that is allowed, weights and routings that change between calls, streams."""
import pytest
import torch

import dense_ref as ref
from bit_vector_quantised_amd.dense import DenseExperts, ExpertRows, Linear  # noqa: F401

from gpu_util import say
from test_gpu_dense import BF16, F32, gen, linear_inputs, outside, randn, routing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
def test_gradients_over_their_inputs(act):
    """The overlaps that are allowed give the gradients of separate buffers, to the bit: dw over w, dx over z, and
    over dy where an activation makes dz another tensor.  Sizes at which every product has many workgroups."""
    say(f"gradients over inputs {act}")
    M, N = 600, 512
    K = 2 * N if act == "swiglu" else N  # (z and dx of one size)
    g, R, x, w, b, _ = linear_inputs(M, K, N, None, act, BF16, BF16, True, False)
    z, dy = randn(g, M, R, dtype=BF16).cuda(), randn(g, M, N, dtype=BF16).cuda()
    x, w = x.cuda(), w.cuda()

    def grads(**over):
        xx, ww, zz, dd = x.clone(), w.clone(), z.clone(), dy.clone()
        at = {"w": ww, "z": zz, "dy": dd}
        dx = at[over["dx"]] if "dx" in over else torch.empty_like(x)
        dw = at[over["dw"]] if "dw" in over else torch.empty_like(w)
        db = torch.empty(R, device="cuda")
        lin = Linear(ww, b.cuda(), act=act, max_rows=M, backward=True)
        lin.backward(xx, dd, None if act == "none" else zz, dx=dx, dw=dw, dbias=db)
        return dx.clone(), dw.clone(), db

    want = grads()
    cases = [dict(dw="w")]
    if act != "none":
        cases += [dict(dx="z"), dict(dx="z", dw="w")]
        if act != "swiglu":
            cases += [dict(dx="dy"), dict(dx="dy", dw="w")]
    for over in cases:
        for a, c in zip(grads(**over), want):
            assert torch.equal(a, c), over


def test_weight_gradients_over_the_weights():
    say("dw of combine over w")
    T, k, C = 700, 8, 264
    rows = ExpertRows(16, k, T)
    g = gen(4)
    rows.sort(routing(g, T, k, 16, dropped=0.1).cuda())
    o, dy, w = randn(g, T * k, C, dtype=BF16).cuda(), randn(g, T, C).cuda(), torch.rand(T, k, generator=g).cuda()
    want = rows.combine_backward(dy, w, o, torch.zeros_like(o))
    same = w.clone()
    got = rows.combine_backward(dy, same, o, torch.zeros_like(o), same)
    assert torch.equal(got[0], want[0]) and torch.equal(same, want[1])


def test_weights_that_move():
    """Weights and a bias whose storage is replaced after the object was made: the next call reads the new one."""
    say("weights moved")
    M, K, N = 5, 64, 24
    g, R, x, w, b, _ = linear_inputs(M, K, N, None, "silu", F32, F32, True, False)
    x, w, b = x.cuda(), w.cuda(), b.cuda()
    lin = Linear(w, b, act="silu", max_rows=M, backward=True)
    first = lin.forward(x).clone()
    old = (w.data, b.data)  # (kept alive: nothing else can be given their memory)
    w.data, b.data = w.data * 2, b.data + 1
    assert w.data_ptr() != old[0].data_ptr() and b.data_ptr() != old[1].data_ptr()
    z = torch.empty(M, R, device="cuda")
    y = lin.forward(x, z=z)
    want = Linear(w.clone(), b.clone(), act="silu", max_rows=M, backward=True)
    assert torch.equal(y, want.forward(x)) and not torch.equal(y, first)
    dx, dwant = torch.empty_like(x), torch.empty_like(x)
    lin.backward(x, y, z, dx=dx)
    want.backward(x, y, z, dx=dwant)
    assert torch.equal(dx, dwant)
    w.data = old[0].double()
    with pytest.raises(ValueError, match="w: need"):
        lin.forward(x)


def test_the_next_routing_before_backward():
    """The routing's buffers are the caller's: the next step may overwrite them before this one's backward."""
    say("routing overwritten before backward")
    T, H, I, E, k = 19, 64, 32, 5, 2
    g = gen(17)
    w1, w2 = randn(g, E, 2 * I, H, scale=0.1).cuda(), randn(g, E, H, I, scale=0.1).cuda()
    step = DenseExperts(w1, w2, k, T + 3, backward=True)
    x, dy = randn(g, T, H).cuda(), randn(g, T, H).cuda()
    ids, w = routing(g, T, k, E).cuda(), torch.rand(T, k, generator=g).cuda()

    def grads(change):
        i, v, xx = ids.clone(), w.clone(), x.clone()
        step.forward(xx, i, v, keep=True)
        if change:
            i.fill_(-1); v.fill_(7.0); xx.fill_(3.0)
        out = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w1), torch.empty_like(w2)
        step.backward(dy, *out)
        return out

    for a, b in zip(grads(False), grads(True)):
        assert torch.equal(a, b)


def test_buffers_outlive_the_calls_of_a_dropped_object():
    """An object used on a side stream and dropped at once: its buffers are not given out again while the side
    stream's work is under way (here a wait of the stream, then nothing: the buffers are only looked at by address)."""
    say("buffers of dropped objects")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    g = gen(31)
    T, H, I, E, k = 64, 64, 32, 4, 2
    w1, w2 = randn(g, E, 2 * I, H, dtype=BF16).cuda(), randn(g, E, H, I, dtype=BF16).cuda()
    x, ids, w = randn(g, T, H, dtype=BF16).cuda(), routing(g, T, k, E).cuda(), torch.rand(T, k, generator=g).cuda()
    wl, y = randn(g, 40, 64, dtype=BF16).cuda(), torch.empty(T, H, device="cuda")

    def buffers(o, seen):
        for v in vars(o).values():
            if isinstance(v, torch.Tensor):
                seen.append(v)
            elif isinstance(v, (Linear, ExpertRows)):
                buffers(v, seen)
        return seen

    def linear():
        return Linear(wl, max_rows=T, backward=True), lambda o: o.forward(x)

    def experts():
        return DenseExperts(w1, w2, k, T, backward=True), lambda o: o.forward(x, ids, w, y)

    def rows():
        return ExpertRows(E, k, T), lambda o: o.sort(ids)

    mine = {t.data_ptr() for t in (w1, w2, wl, x, ids, w, y)}
    for make in (linear, experts, rows):
        o, call = make()
        own = {t.data_ptr(): t.numel() * t.element_size() for t in buffers(o, []) if t.data_ptr() not in mine}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
            call(o)
        del o
        again = [torch.empty(size, dtype=torch.uint8, device="cuda") for size in own.values() for _ in range(3)]
        assert not side.query()  # (the wait is still under way, so the answer means something)
        for t in again:
            assert not any(p <= t.data_ptr() < p + max(size, 1) for p, size in own.items()), make.__name__
        side.synchronize()


def test_experts_outputs_are_not_rounded_before_their_sum():
    """Whole numbers of more than eight bits as the experts' outputs, exact in fp32: y and the weights' gradients,
    sums of multiples of 32 below 2^29, are exact too.  (silu(64) is 64 in fp32; x picks columns of w1, so h = 64 u is exact in bf16.)"""
    say("experts' outputs in fp32")
    T, H, I, E, k = 11, 32, 16, 4, 3
    g = gen(23)
    whole = lambda n, *s: torch.randint(-n, n + 1, s, generator=g).float()  # noqa: E731
    w1, w2 = torch.cat((torch.full((E, I, H), 64.0), whole(100, E, I, H)), 1), whole(3, E, H, I)
    x = torch.zeros(T, H)
    x[torch.arange(T), torch.randint(0, H, (T,), generator=g)] = 1.0
    ids, w, dy = routing(g, T, k, E, dropped=0.1), 2.0 ** torch.randint(-1, 2, (T, k), generator=g), whole(3, T, H)
    h = 64 * torch.einsum("th,eih->tei", x.double(), w1[:, I:].double())
    o = torch.einsum("tei,ehi->teh", h, w2.double())
    assert (o.bfloat16().double() != o).any() and o.abs().max() * 3 * H < 2 ** 29
    at = torch.where(ids < 0, 0, ids).long()
    mine = torch.where((ids < 0)[:, :, None], 0.0, o[torch.arange(T)[:, None], at])
    step = DenseExperts(w1.to(BF16).cuda(), w2.to(BF16).cuda(), k, T, backward=True)
    y = step.forward(x.to(BF16).cuda(), ids.cuda(), w.cuda(), keep=True)
    assert torch.equal(y.cpu().double(), (mine * w[:, :, None].double()).sum(1))
    dx, dw = torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(T, k, device="cuda")
    step.backward(dy.cuda(), dx, dw, torch.empty(w1.shape, dtype=BF16, device="cuda"), torch.empty(w2.shape, dtype=BF16, device="cuda"))
    assert torch.equal(dw.cpu().double(), (mine * dy[:, None].double()).sum(2))


@pytest.mark.parametrize("dtype,other", [(F32, BF16), (BF16, F32)])
def test_combine_backward_into_rows_of_another_type(dtype, other):
    say(f"combine backward {dtype} into {other}")
    T, k, C = 23, 4, 101
    g = gen(6)
    ids = routing(g, T, k, 6, dropped=0.2)
    rows = ExpertRows(6, k, T)
    rows.sort(ids.cuda())
    o, dy, w = randn(g, T * k, C, dtype=dtype), randn(g, T, C), torch.rand(T, k, generator=g)
    drows, wc = torch.full((T * k, C), -3.0, dtype=other, device="cuda"), w.cuda()
    _, dw = rows.combine_backward(dy.cuda(), wc, o.cuda(), drows, wc)
    d, _, named, v, bv = ref.combine_backward64(dy, rows.pair_row.cpu(), w, o, T, k)
    bd = (ref.U + ref.HALF[other]) * d.abs()
    left = torch.ones(T * k, dtype=torch.bool)
    left[named] = False
    d[left] = -3.0
    ref.check(drows, d, bd, "drows")
    ref.check(dw, v, bv, "dw")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gelu_keeps_its_relative_precision(dtype):
    """z Phi(z) and its derivative where Phi(z) is tiny.  Errors, with t = -z / sqrt(2): Phi(z) = erfc(t) / 2 falls as
    exp(-t^2), whose exponent is off by up to 1.5 * 2^-24 of itself twice over (z^2 and the product with the
    base's logarithm, each rounded once, and the constant), that is 3 t^2 * 2^-24 of the value; what multiplies
    it, and the products: 16 * 2^-24, and 2.3 t * 2^-24 of a reciprocal of 1 + a multiple of t.  phi(z): the same
    exponent, and 8 * 2^-23 of the rest."""
    say(f"gelu tail {dtype}")
    z = torch.cat((torch.linspace(-12, 12, 4001), torch.tensor([0.0, -0.0, -1e-20, 1e-20, -5.5, -6.0, -10.5]))).to(dtype).reshape(-1, 1)
    n = z.shape[0]
    lin = Linear(torch.ones(1, 1, dtype=dtype, device="cuda"), act="gelu", max_rows=n, backward=True)
    y = lin.forward(z.cuda(), out=torch.empty(n, 1, device="cuda"))
    v = z.double()
    t = -v / 2.0 ** 0.5
    half = 0.5 * torch.special.erfc(t)
    e = (1.5 * (2 * t * t + 1.5 * t.abs() + 1) + 16) * 2.0 ** -24
    ref.check(y, v * half, e * (v * half).abs(), "gelu")
    dz = torch.empty(1, device="cuda")
    phi = torch.exp(-v * v / 2) / (2 * torch.pi) ** 0.5
    slope = half + v * phi
    be = e * half + (3 * v * v / 2 + 16) * 2.0 ** -24 * (v * phi).abs() + 2 * ref.U * slope.abs()
    # one row at a time (its column sum is its own dz, not rounded to the type)
    one = torch.ones(1, 1, device="cuda")
    for i in list(range(0, n, 97)) + list(range(n - 7, n)):
        lin.backward(z[i:i + 1].cuda(), one, z[i:i + 1].cuda(), dbias=dz)
        ref.check(dz, slope[i], be[i], f"derivative at {v[i].item()}")


@pytest.mark.parametrize("K,dtype", [(201, BF16), (33, F32)])
def test_repacking_leaves_out_what_no_group_uses(K, dtype):
    """Widths that are repacked: neither rows in no group nor the weights of groups without rows are copied, so no
    more of the workspace changes than the others take; and the outputs are those of the groups."""
    say(f"repacking K={K} {dtype}")
    start, M, N = [9, 9, 9, 20, 20, 31, 31, 31, 31], 50, 40
    g, R, x, w, b, _ = linear_inputs(M, K, N, start, "silu", dtype, F32, True, False)
    size = x.element_size()
    row = (K * size + 15) // 16 * 16
    none = outside(M, start)
    lin = Linear(w.cuda(), b.cuda(), act="silu", max_rows=M, backward=True)
    gs = torch.tensor(start, dtype=torch.int32, device="cuda")
    y = torch.full((M, N), -3.0, device="cuda")

    def changed(call):
        lin.ws.fill_(0xA5)
        call()
        return int((lin.ws != 0xA5).sum())

    assert changed(lambda: lin.forward(x.cuda(), gs, out=y)) <= (22 + 2 * R) * row
    want, by, _, _ = ref.linear_forward64(x, w, b, start, "silu", 0.0, None, F32, dtype)
    want[none] = -3.0
    ref.check(y, want, by, "y")
    lin = Linear(w.cuda(), max_rows=M, backward=True)
    dy = randn(g, M, N, dtype=dtype)
    dx, dw = torch.full((M, K), -3.0, dtype=dtype, device="cuda"), torch.full(w.shape, -3.0, dtype=dtype, device="cuda")
    assert changed(lambda: lin.backward(x.cuda(), dy.cuda(), group_start=gs, dx=dx)) <= 2 * R * row
    assert changed(lambda: lin.backward(x.cuda(), dy.cuda(), group_start=gs, dw=dw)) <= 22 * row
    want = ref.linear_backward64(x, w, start, "none", 0.0, None, dy, dtype)
    want["dx"][0][none] = -3.0
    ref.check(dx, *want["dx"], "dx")
    ref.check(dw, *want["dw"], "dw")


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_gradients_that_need_no_x(act):
    """dx and dbias are made without x; dw is not."""
    say(f"gradients without x {act}")
    M, K, N = 21, 48, 24
    g, R, x, w, b, _ = linear_inputs(M, K, N, None, act, BF16, F32, True, False)
    lin = Linear(w.cuda(), b.cuda(), act=act, max_rows=M, backward=True)
    x, dy, z = x.cuda(), randn(g, M, N).cuda(), None if act == "none" else randn(g, M, R, dtype=BF16).cuda()
    new = lambda: (torch.empty_like(x), torch.empty(R, device="cuda"))  # noqa: E731
    with_x, without = new(), new()
    lin.backward(x, dy, z, dx=with_x[0], dbias=with_x[1])
    lin.backward(None, dy, z, dx=without[0], dbias=without[1])
    for a, c in zip(with_x, without):
        assert torch.equal(a, c)
    with pytest.raises(ValueError, match="x"):
        lin.backward(None, dy, z, dw=torch.empty_like(w).cuda())
    with pytest.raises(ValueError, match="rows"):
        lin.backward(None, torch.empty(M + 1, N, device="cuda"), z, dx=torch.empty(M + 1, K, dtype=BF16, device="cuda"))
