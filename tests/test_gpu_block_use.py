"""The norm, the router, rows in 8 bits and the block as programs use them: the experts' step back from 8 bits, the whole block
and its gradients, layers that share their buffers, streams, graphs, long rows."""
import math

import pytest
import torch

import block_ref as ref
import dense_ref
from bit_vector_quantised_amd.block import ExpertChoice, MoeBlock, RmsNorm, Router
from bit_vector_quantised_amd.dense import DenseExperts, ExpertRows, Linear, Rows8

from gpu_util import say
from test_gpu_dense import BF16, F32, gen, randn, routing

pytestmark = pytest.mark.gpu


def experts(g, E, H, I, dtype):
    return randn(g, E, 2 * I, H, dtype=dtype, scale=H ** -0.5).cuda(), randn(g, E, H, I, dtype=dtype, scale=I ** -0.5).cuda()


def grads_of(step, dy, T, dtype):
    E, R, H, k = step.sizes[:4]
    dx, dw = torch.full((T, H), -3.0, dtype=dtype, device="cuda"), torch.full((T, k), -3.0, device="cuda")
    dw1, dw2 = torch.full((E, R, H), -3.0, dtype=dtype, device="cuda"), torch.full((E, H, R // 2), -3.0, dtype=dtype, device="cuda")
    step.backward(dy, dx, dw, dw1, dw2)
    return {"dx": dx, "dw": dw, "dw1": dw1, "dw2": dw2}


@pytest.mark.parametrize("T,H,I,E,k,dtype,dy_dtype,lim,dropped", [
    (37, 96, 64, 7, 3, F32, F32, 0.0, 0.1), (37, 96, 64, 7, 3, BF16, F32, 1.0, 0.1), (1, 128, 32, 4, 2, BF16, BF16, 0.0, 0.0),
    (20, 33, 21, 5, 2, F32, F32, 0.7, 0.2), (50, 72, 41, 3, 2, BF16, F32, 0.0, 0.0), (9, 64, 48, 4, 2, BF16, BF16, 0.0, 1.0)])
def test_experts_backward_from_8_bits(T, H, I, E, k, dtype, dy_dtype, lim, dropped):
    """The gradients are those of the values that were kept, which are x and z rounded to 8 bits."""
    say(f"experts from 8 bits T={T} H={H} I={I} {dtype}")
    g = gen(T + H)
    w1, w2 = experts(g, E, H, I, dtype)
    step = DenseExperts(w1, w2, k, T + 3, swiglu_limit=lim, backward=True, kept8=True)
    x, ids, w = randn(g, T, H, dtype=dtype).cuda(), routing(g, T, k, E, dropped), torch.rand(T, k, generator=g)
    if dropped:
        ids[T // 2] = -1  # a token without experts
    dy = randn(g, T, H, dtype=dy_dtype)
    plain = DenseExperts(w1, w2, k, T + 3, swiglu_limit=lim)
    y = step.forward(x, ids.cuda(), w.cuda(), keep=True)
    assert torch.equal(y, plain.forward(x, ids.cuda(), w.cuda()))  # keeping changes nothing of the result
    q, e = ref.to8(x.float().cpu())
    assert torch.equal(step.x8.q[:T].cpu(), q) and torch.equal(step.x8.e[:T].cpu(), e)
    kept = ref.from8(step.x8.q[:T], step.x8.e[:T], H), ref.from8(step.z8.q[:T * k], step.z8.e[:T * k], 2 * I)
    pair_row, start = step.rows.pair_row[:T * k].cpu(), step.rows.expert_start.tolist()
    x.fill_(9.0)  # (what backward needs of the pass is kept)
    got = grads_of(step, dy.cuda(), T, dtype)
    want = ref.experts_backward8_64(*kept, dy, pair_row, start, w, w1.cpu(), w2.cpu(), lim, dtype)
    for name in want:
        dense_ref.check(got[name], *want[name], name)
    with pytest.raises(ValueError, match="kept nothing"):
        step.backward(dy.cuda(), *got.values())


def test_values_kept_are_those_of_the_pass():
    """z in 8 bits is z rounded, z the first product's values before the activation."""
    say("z in 8 bits")
    T, H, I, E, k = 25, 64, 48, 4, 2
    g = gen(3)
    w1, w2 = experts(g, E, H, I, BF16)
    step = DenseExperts(w1, w2, k, T, backward=True, kept8=True)
    x, ids = randn(g, T, H, dtype=BF16).cuda(), routing(g, T, k, E, 0.1)
    step.forward(x, ids.cuda(), torch.rand(T, k, generator=g).cuda(), keep=True)
    rows = ExpertRows(E, k, T)
    start = rows.sort(ids.cuda())
    xs = rows.gather(x, torch.zeros(T * k, H, dtype=BF16, device="cuda"))
    z = torch.zeros(T * k, 2 * I, dtype=BF16, device="cuda")
    Linear(w1, max_rows=T * k).forward(xs, start, out=z)
    q, e = ref.to8(z.float().cpu())
    n = int(start[-1])
    assert torch.equal(step.z8.q[:n].cpu(), q[:n]) and torch.equal(step.z8.e[:n].cpu(), e[:n])


def block(g, T, H, I, E, k, dtype, kept8, work=None, **choice):
    w1, w2 = experts(g, E, H, I, dtype)
    step = DenseExperts(w1, w2, k, T, backward=True, kept8=kept8, work=None if work is None else work.experts)
    norm = RmsNorm((1 + 0.2 * randn(g, H)).cuda(), max_rows=T, backward=True)
    router = Router(randn(g, E, H, dtype=dtype, scale=2 * H ** -0.5).cuda(), k, T, backward=True, **choice)
    return MoeBlock(norm, router, step, work)


def block_grads(b, s, dy, ds):
    E, R, H = b.experts.sizes[:3]
    dtype = b.experts.sizes[5]
    new = lambda *shape, t=dtype: torch.full(shape, -3.0, dtype=t, device="cuda")  # noqa: E731
    out = {"dx": new(*s.shape, t=s.dtype), "dgain": new(H, t=F32), "drouter": new(E, H), "dw1": new(E, R, H), "dw2": new(E, H, R // 2)}
    b.backward(s, dy, ds, *out.values())
    return out


BIASED = dict(score="sigmoid", groups=4, top_groups=2, scale=2.5)


@pytest.mark.parametrize("choice", [dict(), dict(score="softmax", renorm=False), BIASED], ids=["softmax", "scores", "groups"])
def test_block_and_its_gradients(choice):
    """In fp32, against 64 bits with the same experts chosen.  The longest chain is dx: norm, product, product, sum, of at
    most 96 terms each; 4 * 96 * 2^-23 = 4.6e-5 of sums of sizes, which exceed a value's by about the root of their
    number (10): within 5e-4 of the largest value of each tensor's norm."""
    say(f"block {choice}")
    T, H, I, E, k = 31, 96, 40, 8, 3
    g = gen(4)
    b = block(g, T, H, I, E, k, F32, False, **choice)
    if choice.get("groups"):
        b.router.choice.bias = (0.1 * randn(g, E)).cuda()
    x, r, dy, ds = (randn(g, T, H) for _ in range(4))
    s = torch.empty(T, H, device="cuda")
    y = b.forward(x.cuda(), r.cuda(), s, keep=True)
    got = block_grads(b, s, dy.cuda(), ds.cuda())
    ids = b.router.ids[:T].cpu().long()
    leaf = lambda t: t.detach().cpu().double().requires_grad_(True)  # noqa: E731
    x64, gain, wr, w1, w2 = leaf(x), leaf(b.norm.gain), leaf(b.router.linear.w), leaf(b.experts.fc1.w), leaf(b.experts.fc2.w)
    s64 = x64 + r.double()
    n = s64 / torch.sqrt((s64 * s64).mean(1, keepdim=True) + 1e-6) * gain
    logits = n @ wr.t()
    score = torch.sigmoid(logits) if choice.get("score") == "sigmoid" else torch.softmax(logits, 1)
    p = score.gather(1, ids)
    w = choice.get("scale", 1.0) * (p / p.sum(1, keepdim=True) if choice.get("renorm", True) else p)
    rows = []
    for t in range(T):
        acc = 0
        for i in range(k):
            e = int(ids[t, i])
            gate, up = (w1[e] @ n[t]).chunk(2)
            acc = acc + w[t, i] * (w2[e] @ (gate * torch.sigmoid(gate) * up))
        rows.append(acc)
    y64 = torch.stack(rows)
    ((y64 * dy.double()).sum() + (s64 * ds.double()).sum()).backward()
    pairs = {"y": (y, y64.detach()), "dx": (got["dx"], x64.grad), "dgain": (got["dgain"], gain.grad), "drouter": (got["drouter"], wr.grad),
             "dw1": (got["dw1"], w1.grad), "dw2": (got["dw2"], w2.grad)}
    for name, (a, want) in pairs.items():
        off = ((a.double().cpu() - want).norm() / want.norm()).item()
        say(f"  {name}: {off:.2e}")
        assert off <= 5e-4, name


@pytest.mark.parametrize("kept8", [False, True])
def test_block_is_its_parts(kept8):
    """To the bit what its parts give one after the other; with padding tokens that take no expert."""
    say(f"block by parts kept8={kept8}")
    T, H, I, E, k = 40, 160, 48, 16, 4
    g = gen(6)
    bias = torch.zeros(E)
    bias[3] = -math.inf  # an expert that is off
    b = block(g, T + 5, H, I, E, k, BF16, kept8, score="sigmoid", groups=4, top_groups=2, bias=bias.cuda())
    x, r = randn(g, T, H, dtype=BF16).cuda(), randn(g, T, H, dtype=BF16).cuda()
    dy, ds = randn(g, T, H, dtype=BF16).cuda(), randn(g, T, H, dtype=BF16).cuda()
    s, y = torch.empty_like(x), torch.empty_like(x)
    b.forward(x, r, s, y, keep=True)
    got = block_grads(b, s, dy, ds)
    c = b.router.choice.c
    norm, step = b.norm, b.experts
    one = DenseExperts(step.fc1.w, step.fc2.w, k, T, backward=True, kept8=kept8)
    n, s2, x8 = torch.empty_like(x), torch.empty_like(x), one.x8
    norm.forward(x, r, s2, n, x8)
    logits = Linear(b.router.linear.w, max_rows=T).forward(n, out=torch.empty(T, E, device="cuda"))
    choice = ExpertChoice(E, k, "sigmoid", bias.cuda(), 4, 2)
    ids, w = choice.forward(logits)
    assert not (ids == 3).any() and c.n_groups == 4
    y2 = one.forward(n, ids, w, torch.empty_like(x), keep=True, x8_there=kept8)
    assert torch.equal(s, s2) and torch.equal(y, y2)
    back = grads_of(one, dy, T, BF16)
    lin = Linear(b.router.linear.w, max_rows=T, backward=True, kept8=True)
    dn2, drouter = torch.empty_like(x), torch.empty_like(lin.w)
    lin.backward(x8 if kept8 else n, choice.backward(logits, ids, back["dw"]), dx=dn2, dw=drouter)
    dx, dgain = torch.empty_like(x), torch.empty(H, device="cuda")
    norm.backward(s, back["dx"], dn2, ds, dx, dgain)
    for name, want in {"dx": dx, "dgain": dgain, "drouter": drouter, "dw1": back["dw1"], "dw2": back["dw2"]}.items():
        assert torch.equal(got[name], want), name


def test_layers_that_share_buffers():
    """Two blocks one after the other, forward and then back, give with shared buffers what they give with their own."""
    say("layers that share buffers")
    T, H, I, E, k = 33, 128, 64, 8, 2
    x = randn(gen(1), T, H, dtype=BF16).cuda()
    dy = randn(gen(2), T, H, dtype=BF16).cuda()
    results = []
    for shared in (False, True):
        g = gen(7)
        first = block(g, T, H, I, E, k, BF16, True)
        second = block(g, T, H, I, E, k, BF16, True, work=first if shared else None)
        assert (second.experts.xs is first.experts.xs) == shared and second.experts.x8 is not first.experts.x8
        s1, s2 = torch.empty_like(x), torch.empty_like(x)
        y1, y2 = torch.empty_like(x), torch.empty_like(x)
        first.forward(x, torch.zeros_like(x), s1, y1, keep=True)
        second.forward(y1, s1, s2, y2, keep=True)
        back2 = block_grads(second, s2, dy, dy)   # (the stack's result is s2 + y2)
        back1 = block_grads(first, s1, back2["dx"], back2["dx"])
        results.append([y2, s2, *back2.values(), *back1.values()])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="work"):
        block(gen(7), T + 1, H, I, E, k, BF16, True, work=first)
    with pytest.raises(ValueError, match="work"):
        block(gen(7), T, H, I, E, k, BF16, False, work=first)


@pytest.mark.parametrize("kept8", [False, True])
def test_block_in_a_graph(kept8):
    """Forward and back captured into one graph: every replay, on new inputs and with eager work of the same objects between,
    gives the eager results' bits."""
    say(f"block in a graph kept8={kept8}")
    T, H, I, E, k = 29, 128, 96, 16, 4
    g = gen(5)
    b = block(g, T, H, I, E, k, BF16, kept8, **BIASED)
    x, r, dy, ds, s, y = (torch.empty(T, H, dtype=BF16, device="cuda") for _ in range(6))
    b.router.choice.bias = (0.1 * randn(g, E)).cuda()
    out = [torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(H, device="cuda"), torch.empty(E, H, dtype=BF16, device="cuda"),
           torch.empty(E, 2 * I, H, dtype=BF16, device="cuda"), torch.empty(E, H, I, dtype=BF16, device="cuda")]

    def fill(seed):
        q = gen(seed)
        for t in (x, r, dy, ds):
            t.copy_(randn(q, T, H))

    def run():
        b.forward(x, r, s, y, keep=True)
        b.backward(s, dy, ds, *out)

    fill(0)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(1, 5):
        fill(seed)
        run()
        want = [t.clone() for t in (s, y, *out)]
        for t in (s, y, *out):
            t.fill_(-3.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip((s, y, *out), want):
            assert torch.equal(a, c)


def test_two_graphs_of_two_objects_at_once():
    """Two norms with their workspaces, captured and replayed on two streams at once, do not touch each other."""
    say("two graphs at once")
    M, C = 700, 1000
    g = gen(9)
    gain = (1 + randn(g, C)).cuda()
    work = []
    for i in range(2):
        norm = RmsNorm(gain, max_rows=M, backward=True)
        s, dy = randn(g, M, C, dtype=BF16).cuda(), randn(g, M, C, dtype=BF16).cuda()
        dx, dg = torch.empty_like(s), torch.empty(C, device="cuda")
        norm.backward(s, dy, dx=dx, dgain=dg)
        work.append((norm, s, dy, dx, dg, dx.clone(), dg.clone()))
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in work]
    for norm, s, dy, dx, dg, _, _ in work:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norm.backward(s, dy, dx=dx, dgain=dg)
        graphs.append(graph)
    for _ in range(5):
        for _, _, _, dx, dg, _, _ in work:
            dx.fill_(-3.0)
            dg.fill_(-3.0)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, _, dx, dg, want, wg in work:
            assert torch.equal(dx, want) and torch.equal(dg, wg)


def test_on_another_stream():
    """An object's calls on a side stream, and the object dropped while they are under way."""
    say("block on a side stream")
    T, H, I, E, k = 64, 256, 64, 8, 2
    x = randn(gen(2), T, H, dtype=BF16).cuda()
    b = block(gen(3), T, H, I, E, k, BF16, True)
    s, y = torch.empty_like(x), torch.empty_like(x)
    b.forward(x, x, s, y, keep=True)
    want = [y.clone(), *(t.clone() for t in block_grads(b, s, x, x).values())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = block(gen(3), T, H, I, E, k, BF16, True)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        s2, y2 = torch.empty_like(x), torch.empty_like(x)
        b.forward(x, x, s2, y2, keep=True)
        got = [y2, *block_grads(b, s2, x, x).values()]
        del b
        for _ in range(20):
            torch.empty(1 << 20, device="cuda").fill_(5.0)  # (may take what the object has given back)
    torch.cuda.synchronize()
    for a, c in zip(got, want):
        assert torch.equal(a, c)


def test_buffers_outlive_the_calls_of_a_dropped_object():
    """An object used on a side stream and dropped at once, also one that only other objects' calls have used there: its
    buffers are not given out again while the side stream's work is under way."""
    say("buffers of dropped objects")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    T, H, I, E, k = 64, 64, 32, 4, 2
    x = randn(gen(2), T, H, dtype=BF16).cuda()
    s, y = torch.empty_like(x), torch.empty_like(x)
    gain = torch.ones(H, device="cuda")
    norm = RmsNorm(gain, max_rows=T)
    out = {}

    def parts(o, seen, met):
        if id(o) in met:
            return seen
        met.add(id(o))
        for v in vars(o).values():
            if isinstance(v, torch.Tensor):
                seen[v.data_ptr()] = v.numel() * v.element_size()
            elif type(v).__module__.startswith("bit_vector_quantised_amd") and hasattr(v, "__dict__") and not isinstance(v, type):
                parts(v, seen, met)
        return seen

    def whole(b):
        b.forward(x, x, s, y, keep=True)
        b.backward(s, x, x, *out.values())

    b = block(gen(3), T, H, I, E, k, BF16, True)
    out = {"dx": torch.empty_like(x), "dgain": torch.empty(H, device="cuda"), "drouter": torch.empty_like(b.router.linear.w),
           "dw1": torch.empty_like(b.experts.fc1.w), "dw2": torch.empty_like(b.experts.fc2.w)}
    w = [b.norm.gain, b.router.linear.w, b.experts.fc1.w, b.experts.fc2.w]  # (what a caller owns)
    del b

    def new_block():
        step = DenseExperts(w[2], w[3], k, T, backward=True, kept8=True)
        return MoeBlock(RmsNorm(w[0], max_rows=T, backward=True), Router(w[1], k, T, backward=True), step)

    makers = [(lambda: Rows8(T, H), lambda o: norm.forward(x, rows8=o, dense=False)),
              (lambda: RmsNorm(gain, max_rows=T, backward=True), lambda o: o.backward(x, x, dgain=out["dgain"])),
              (lambda: Router(w[1], k, T, backward=True), lambda o: o.forward(x)), (new_block, whole)]
    mine = {t.data_ptr() for t in (x, s, y, gain, *w, *out.values())}
    for make, call in makers:
        o = make()
        own = {p: n for p, n in parts(o, {}, set()).items() if p not in mine and n}
        assert own
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
            call(o)
        del o
        again = [torch.empty(size, dtype=torch.uint8, device="cuda") for size in own.values() for _ in range(3)]
        assert not side.query()  # (the wait is still under way, so the answer means something)
        for t in again:
            assert not any(p <= t.data_ptr() < p + size for p, size in own.items())
        side.synchronize()


def test_router_for_one_token_and_for_none():
    say("router: one token, none")
    g = gen(10)
    E, H, k = 256, 512, 8
    router = Router(randn(g, E, H, dtype=BF16).cuda(), k, 4, backward=True, **BIASED)
    x = randn(g, 4, H, dtype=BF16).cuda()
    all_ids, all_w = (t.clone() for t in router.forward(x))
    for t in range(4):
        ids, w = router.forward(x[t:t + 1])
        want, ww, rel = ref.choose64(router.logits[:1].cpu(), None, k, "sigmoid", 4, 2, 2, True, 2.5)
        assert torch.equal(ids.cpu().long(), want) and ids.shape == (1, k)
        dense_ref.check(w, ww, rel * ww, "w")
    ids, w = router.forward(x[:0])
    assert ids.shape == w.shape == (0, k)
    dweight = torch.full((E, H), -3.0, dtype=BF16, device="cuda")
    router.backward(x[:0], w, dweight=dweight)
    assert not dweight.any()  # no rows: zeros
    with pytest.raises(ValueError, match="tokens"):
        router.forward(randn(g, 5, H, dtype=BF16).cuda())
    with pytest.raises(ValueError, match="no forward"):
        router.backward(x, all_w)
    assert all_ids.shape == (4, k)


def test_empty_batches():
    say("no rows")
    e = lambda *s, t=BF16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    norm = RmsNorm(torch.ones(64, device="cuda"), max_rows=8, backward=True)
    assert norm.forward(e(0, 64), e(0, 64)).shape == (0, 64)
    dgain = torch.full((64,), 7.0, device="cuda")
    norm.backward(e(0, 64), e(0, 64), dgain=dgain)
    assert not dgain.any()
    r = Rows8(0, 64)
    assert r.pack(e(0, 64)).unpack().shape == (0, 64)
    rows = ExpertRows(4, 2, 8)
    rows.sort(e(0, 2, t=torch.int32))
    assert rows.gather(r).shape == (0, 64)
    rows.act_backward(r, e(0, 32), act="swiglu", dz=e(0, 64), y=e(0, 32), dw=e(0, 2, t=F32))
    b = block(gen(1), 4, 64, 32, 4, 2, BF16, True)
    s = e(0, 64)
    assert b.forward(s, s, e(0, 64), keep=True).shape == (0, 64)
    got = block_grads(b, s, s, s)
    assert got["dx"].shape == (0, 64) and not got["dw1"].any() and not got["drouter"].any() and not got["dgain"].any()


def test_refusals():
    """What the library cannot see: shapes, types, devices, buffers that were not made."""
    say("block: refusals")
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    gain = torch.ones(64, device="cuda")
    norm = RmsNorm(gain, max_rows=4)
    for call in (lambda: norm.forward(x[:, ::2]), lambda: norm.forward(torch.zeros(5, 64, device="cuda")), lambda: norm.forward(x.cpu()),
                 lambda: norm.forward(x, residual=x[:3]), lambda: norm.forward(x, x, s=torch.zeros(4, 64, device="cuda")),
                 lambda: norm.forward(x, out=x, dense=False), lambda: norm.forward(x, rows8=Rows8(4, 32)), lambda: norm.forward(x, rows8=Rows8(3, 64)),
                 lambda: norm.backward(x, x, dgain=gain), lambda: norm.backward(x, x, ds=x, dx=torch.zeros(4, 64, device="cuda")),
                 lambda: RmsNorm(gain.double()), lambda: RmsNorm(gain, eps=0.0), lambda: RmsNorm(torch.ones(16385, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    rows = ExpertRows(4, 2, 4)
    rows.sort(torch.zeros(4, 2, dtype=torch.int32, device="cuda"))
    z8, dy = Rows8(8, 64), torch.zeros(8, 32, dtype=BF16, device="cuda")
    for call in (lambda: rows.act_backward(z8, dy, act="relu"), lambda: rows.act_backward(z8, dy[:4], dz=dy),
                 lambda: rows.act_backward(z8, dy, dz=dy), lambda: rows.act_backward(Rows8(7, 64), dy, y=dy.clone()),
                 lambda: rows.act_backward(z8, dy, dz=torch.zeros(8, 64, device="cuda"), y=torch.zeros(8, 32, dtype=BF16, device="cuda")),
                 lambda: rows.gather(Rows8(3, 64)), lambda: Rows8(4, 0), lambda: Rows8(4, 40000), lambda: Rows8(-1, 64),
                 lambda: z8.pack(torch.zeros(9, 64, device="cuda")), lambda: z8.pack(x.half()), lambda: z8.unpack(9),
                 lambda: z8.unpack(2, out=torch.zeros(3, 64, device="cuda")),
                 lambda: rows.act_backward(z8, dy, dz=torch.zeros(8, 64, dtype=torch.float16, device="cuda")),
                 lambda: rows.act_backward(z8, dy.half(), dw=torch.zeros(4, 2, device="cuda")),
                 lambda: norm.backward(x, x, dx=x.half()), lambda: norm.forward(x, s=x.half()), lambda: norm.forward(x, out=x.half())):
        with pytest.raises((ValueError, TypeError)):
            call()
    lin = Linear(torch.zeros(32, 64, dtype=BF16, device="cuda"), max_rows=4, backward=True)
    with pytest.raises(ValueError, match="kept8"):
        lin.backward(Rows8(4, 64), torch.zeros(4, 32, dtype=BF16, device="cuda"), dw=torch.zeros(32, 64, dtype=BF16, device="cuda"))
    for kw in (dict(n_experts=0, top_k=1), dict(n_experts=8, top_k=9), dict(n_experts=8, top_k=3, groups=4, top_groups=1), dict(n_experts=9, top_k=1, groups=2),
               dict(n_experts=8, top_k=1, score="relu"), dict(n_experts=8, top_k=1, best=3), dict(n_experts=8, top_k=1, bias=torch.zeros(9, device="cuda"))):
        with pytest.raises(ValueError):
            ExpertChoice(**kw)
    w1, w2 = torch.zeros(4, 64, 32, dtype=BF16, device="cuda"), torch.zeros(4, 32, 32, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="kept8"):
        DenseExperts(w1, w2, 2, 4, kept8=True)
    step = DenseExperts(w1, w2, 2, 4, backward=True)
    with pytest.raises(ValueError, match="x8_there"):
        step.forward(x[:, :32].contiguous(), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda"), keep=True, x8_there=True)
    small = RmsNorm(torch.ones(32, device="cuda"), max_rows=4, backward=True)
    for norm, router in ((RmsNorm(gain, max_rows=4), Router(torch.zeros(4, 32, dtype=BF16, device="cuda"), 2, 4)),
                         (small, Router(torch.zeros(4, 32, device="cuda"), 2, 4)), (small, Router(torch.zeros(8, 32, dtype=BF16, device="cuda"), 2, 4)),
                         (small, Router(torch.zeros(4, 32, dtype=BF16, device="cuda"), 1, 4)), (small, Router(torch.zeros(4, 32, dtype=BF16, device="cuda"), 2, 3))):
        with pytest.raises(ValueError):
            MoeBlock(norm, router, step)
    forward_only = MoeBlock(RmsNorm(torch.ones(32, device="cuda"), max_rows=4), Router(torch.zeros(4, 32, dtype=BF16, device="cuda"), 2, 4, backward=True), step)
    x32 = torch.zeros(4, 32, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="backward"):
        forward_only.forward(x32, keep=True)
    assert forward_only.forward(x32).shape == (4, 32)


def test_far_rows():
    """Rows behind 2^32 bytes and 2^31 values."""
    say("far rows")
    M, C = 300000, 16384
    x = torch.zeros(M, C, dtype=BF16, device="cuda")
    some = torch.tensor([0, 1, 131071, 131072, 262143, 262144, M - 1], device="cuda")
    g = gen(12)
    x[some] = randn(g, len(some), C, dtype=BF16).cuda()
    r = Rows8(M, C).pack(x)
    q, e = ref.to8(x[some].float().cpu())
    assert torch.equal(r.q[some].cpu(), q) and torch.equal(r.e[some].cpu(), e)
    want = ref.from8(q, e, C)
    x.fill_(3.0)
    r.unpack(out=x)
    assert torch.equal(x[some].double().cpu(), want) and not x[2].any() and not x[M - 2].any()
    gain = 1 + 0.1 * randn(g, C)
    norm = RmsNorm(gain.cuda(), max_rows=M, backward=True)
    s = x[some].cpu()
    norm.forward(x, out=x, rows8=r)
    y = ref.norm64(s, None, gain, 1e-6, BF16, BF16)
    dense_ref.check(x[some], y[2], y[3], "y")
    ref.check8(r.q[some], r.e[some], y[2], y[4], "8 bits")
    dy = torch.zeros_like(x)
    dy[some] = randn(g, len(some), C, dtype=BF16).cuda()
    x[some] = s.cuda()
    dgain = torch.empty(C, device="cuda")
    back = ref.norm_backward64(s, gain, 1e-6, dy[some].cpu(), None, None, BF16)
    norm.backward(x, dy, ds=None, dx=(dx := torch.empty_like(x)), dgain=dgain)
    dense_ref.check(dx[some], back[0], back[1], "dx")
    dense_ref.check(dgain, back[2], back[3], "dgain")
