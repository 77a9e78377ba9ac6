"""Measured cases of the operators around the experts, forward and back: the norm with the
residual's addition and an output in 8 bits, the choice of experts, and rows kept in 8 bits
for the backward pass.

A case's "op" is one of
  norm         s = x + residual, y = s / sqrt(mean(s^2) + eps) * gain, in bf16 or fp32 and (or) kept in 8 bits
  norm_grad    its gradients: of x and the residual, of the gain
  choose       logits -> the experts of each token and their weights
  choose_grad  the gradient of the logits from the weights'
  keep         rows into 8 bits with a scale for each 32 columns, and back
  spread       tokens' rows out of 8 bits into the order of their experts
  act_grad     dz, the activation and the routing weights' gradient from z in 8 bits
  grad8        gradients of the dense product from x and z in 8 bits: of x, of W, of b

8 bits: blocks of 32 columns (from a row's first) as e4m3 values times the smallest power of two,
2^-110 or more, that brings the block's largest magnitude to 448 or less.  Outputs in 8 bits are
returned as the values they stand for, which bf16 holds exactly.

Sizes: hidden 7168, inner 2048, 256 experts, top-8 is this repository's layer shape; 1 and 4096
tokens are its decode and prefill batches.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEVICE = "cuda"
LIMIT = 7.0  # the SwiGLU clamp of the cases that have that activation
EPS = 1e-6


# ---------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------

def listed():
    return [
        # one decoded token before the router: nothing but latency
        {"name": "norm-one", "op": "norm", "rows": 1, "cols": 7168, "type": "bf16", "s_type": "bf16", "y_type": "bf16",
         "residual": True, "dense": True, "kept": True},
        # a training chunk: what the products read, and in the same pass what the way back reads
        {"name": "norm-chunk", "op": "norm", "rows": 4096, "cols": 7168, "type": "bf16", "s_type": "bf16",
         "y_type": "bf16", "residual": True, "dense": True, "kept": True},
        # odd in both sizes, an fp32 stream
        {"name": "norm-odd", "op": "norm", "rows": 1021, "cols": 2047, "type": "bf16", "s_type": "f32", "y_type": "f32",
         "residual": True, "dense": True, "kept": False},
        # a training chunk's way back: the experts' and the router's gradients of y, the stream's of s
        {"name": "norm-grad-chunk", "op": "norm_grad", "rows": 4096, "cols": 7168, "type": "bf16", "s_type": "bf16",
         "two": True, "stream": True},
        # one decoded token, scores by sigmoid, groups of experts and a bias for balance
        {"name": "choose-one", "op": "choose", "tokens": 1, "experts": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "best": 2, "renorm": True, "scale": 2.5, "closed": 0.0, "padded": 0},
        # four prefill chunks at once, the same way
        {"name": "choose-chunk", "op": "choose", "tokens": 16384, "experts": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "best": 2, "renorm": True, "scale": 2.5, "closed": 0.0, "padded": 100},
        # their way back for softmax without renormalisation, which reaches every logit
        {"name": "choose-grad-chunk", "op": "choose_grad", "tokens": 16384, "experts": 256, "k": 8, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "best": 1, "renorm": False, "scale": 1.0, "closed": 0.0,
         "padded": 100},
        # gate and up values of a training chunk's pairs
        {"name": "keep-chunk", "op": "keep", "rows": 32768, "cols": 4096, "type": "bf16"},
        # the kept tokens of that chunk to their experts again
        {"name": "spread-chunk", "op": "spread", "tokens": 4096, "k": 8, "experts": 256, "cols": 7168, "type": "bf16",
         "dropped": 0.0},
        # the way back through the activation of that chunk
        {"name": "act-grad-chunk", "op": "act_grad", "tokens": 4096, "k": 8, "experts": 256, "n_out": 2048,
         "act": "swiglu", "type": "bf16", "dropped": 0.0},
        # the gradients of a share of the experts
        {"name": "grad8-experts", "op": "grad8", "rows": 8192, "groups": 16, "n_in": 7168, "n_out": 2048,
         "act": "swiglu", "type": "bf16", "bias": True, "skew": 0.25, "behind": 0},
        # a small odd layer in fp32
        {"name": "grad8-odd", "op": "grad8", "rows": 515, "groups": 0, "n_in": 1000, "n_out": 333, "act": "gelu",
         "type": "f32", "bias": True, "skew": 0.0, "behind": 0},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even in its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A width: mostly a multiple of 128 as the layers have, else of 8, else any."""
    n = _spread(rng, low, high)
    step = rng.choice((128, 128, 128, 8, 1))
    return max(step, n // step * step)


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_grad", "norm_grad", "choose", "choose", "choose_grad", "keep", "spread",
                     "act_grad", "grad8", "grad8"))
    kind = rng.choice(("bf16", "bf16", "bf16", "f32"))
    other = rng.choice((kind, "f32"))
    if op in ("norm", "norm_grad"):
        cols = _width(rng, 64, 16384)
        rows = _spread(rng, 1, max(1, 4096 * 7168 // cols))
        case = {"op": op, "rows": rows, "cols": cols, "type": kind, "s_type": other}
        if op == "norm":
            out = rng.choice(((True, False), (True, True), (False, True)))
            return case | {"y_type": rng.choice((kind, "f32")), "residual": rng.random() < 0.7, "dense": out[0],
                           "kept": out[1]}
        return case | {"two": rng.random() < 0.5, "stream": rng.random() < 0.7}
    if op in ("choose", "choose_grad"):
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * _spread(rng, 4, 1024 // groups)
        top_groups = rng.randint(1, groups)
        k = min(top_groups * (experts // groups), rng.choice((1, 2, 4, 6, 8, 9, 16, 32)))
        tokens = _spread(rng, 1, max(1, min(65536, 16384 * 256 // experts)))
        return {"op": op, "tokens": tokens, "experts": experts, "k": k, "score": rng.choice(("softmax", "sigmoid")),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups, "best": rng.choice((1, 2)),
                "renorm": rng.random() < 0.6, "scale": rng.choice((1.0, 2.5)), "closed": rng.choice((0.0, 0.0, 0.1)),
                "padded": rng.choice((0, 0, tokens // 3))}
    if op == "keep":
        cols = _width(rng, 64, 16384)
        return {"op": op, "rows": _spread(rng, 1, max(1, 32768 * 4096 // cols)), "cols": cols, "type": kind}
    if op in ("spread", "act_grad"):
        experts = _spread(rng, 4, 1024)
        k = min(experts, rng.choice((1, 2, 4, 6, 8, 9)))
        cols = _width(rng, 64, 8192 if op == "spread" else 4096)
        most = 4096 * 8 * (7168 if op == "spread" else 2048) // (k * cols * (1 if kind == "bf16" else 2))
        case = {"op": op, "tokens": _spread(rng, 1, max(1, min(16384, most))), "k": k, "experts": experts, "type": kind,
                "dropped": rng.choice((0.0, 0.0, 0.05, 0.3))}
        return case | ({"cols": cols} if op == "spread" else {"n_out": cols, "act": rng.choice(("swiglu", "swiglu", "silu", "gelu"))})
    n_in, n_out = _width(rng, 128, 8192), _width(rng, 64, 4096)
    act = rng.choice(("none", "silu", "gelu", "swiglu", "swiglu"))
    wide = n_out * (2 if act == "swiglu" else 1)
    groups = rng.choice((0, 0, _spread(rng, 2, 64)))
    while groups * n_in * wide > 16 * 7168 * 4096:
        groups //= 2
    most = (9e11 if kind == "bf16" else 6e10) / (4 * n_in * wide)
    return {"op": op, "rows": _spread(rng, 1, max(1, min(32768, int(most)))), "groups": groups, "n_in": n_in,
            "n_out": n_out, "act": act, "type": kind, "bias": rng.random() < 0.6, "skew": rng.choice((0.0, 0.25, 0.5)),
            "behind": rng.choice((0, 0, 5)) if groups else 0}


# ---------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------

def _normal(g, shape, dtype, scale=1.0):
    # (drawn in fp32 slices: a share of the experts is gigabytes)
    out = torch.empty(shape, dtype=dtype, device=DEVICE)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - at)
        flat[at:at + n] = torch.randn(n, generator=g, device=DEVICE).mul_(scale)
    return out


def _stream(g, rows, cols, dtype):
    """Rows of a residual stream: a few columns far larger than the others, rows of several sizes."""
    x = _normal(g, (rows, cols), torch.float32)
    x *= torch.where(torch.rand(cols, generator=g, device=DEVICE) < 0.01, 20.0, 1.0)
    x *= torch.exp(torch.randn(rows, 1, generator=g, device=DEVICE))
    return x.to(dtype)


def _routing(case, g):
    """Distinct experts for each token, some far more popular than others, and weights
    that sum to one; dropped pairs have expert -1."""
    T, k, E = case["tokens"], case["k"], case["experts"]
    popular = -1.1 * torch.log(1.0 + torch.randperm(E, generator=g, device=DEVICE).float())
    gumbel = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEVICE).clamp_(1e-9, 1 - 1e-7)))
    score, ids = torch.topk(popular + gumbel, k, dim=1)
    w = torch.softmax(score, dim=1)
    ids = torch.where(torch.rand(T, k, generator=g, device=DEVICE) < case["dropped"], -1, ids).to(torch.int32)
    return ids.contiguous(), w.float().contiguous()


def _pair_row(ids, experts):
    """Where the sort by expert, which ran on the way there, put each pair; -1 for a dropped one."""
    flat = ids.view(-1).long()
    key = torch.where(flat < 0, experts, flat)
    order = torch.argsort(key, stable=True)
    at = torch.empty_like(order)
    at[order] = torch.arange(flat.numel(), device=DEVICE)
    return torch.where(flat < 0, -1, at).to(torch.int32)


def _group_start(case, g):
    """The rows of each group: sizes by a power of the group's rank; "behind" rows at the
    end belong to none."""
    G, rows = case["groups"], case["rows"] - min(case["behind"], case["rows"] - 1)
    p = (1.0 + torch.randperm(G, generator=g, device=DEVICE).double()) ** -case["skew"]
    group = torch.multinomial(p / p.sum(), rows, replacement=True, generator=g)
    start = torch.zeros(G + 1, dtype=torch.int64, device=DEVICE)
    start[1:] = torch.cumsum(torch.bincount(group, minlength=G), 0)
    return start.to(torch.int32)


def _to8(x):
    """Rows in 8 bits: bytes of e4m3 [M, cols rounded up to 32], and the scales' exponents + 127 [M, a 32nd of that]."""
    M, C = x.shape
    blocks = torch.nn.functional.pad(x.float(), (0, -C % 32)).view(M, -1, 32)
    part, exponent = torch.frexp(blocks.abs().amax(2))
    exponent = torch.where(part == 0, -110, torch.where(part <= 0.875, exponent - 9, exponent - 8).clamp(min=-110))
    q = torch.ldexp(blocks, -exponent[..., None]).to(torch.float8_e4m3fn)
    return q.view(M, -1).view(torch.uint8), (exponent + 127).to(torch.uint8)


def _from8(q, e, cols):
    """The values that they stand for, in fp32."""
    blocks = q.view(torch.float8_e4m3fn).float().view(q.shape[0], -1, 32)
    return torch.ldexp(blocks, e.int()[..., None] - 127).view(q.shape[0], -1)[:, :cols]


def _rows8(x):
    """x in 8 bits, as a program that kept it has it in hand."""
    q, e = _to8(x)
    if not own:
        return q, e
    from bit_vector_quantised_amd.dense import Rows8
    kept = Rows8(x.shape[0], x.shape[1], device=DEVICE)
    kept.q.copy_(q)
    kept.e.copy_(e)
    return kept


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 7919 + 29)
    op, kind = case["op"], TYPES[case.get("type", "f32")]
    s = {"case": dict(case)}
    if op in ("norm", "norm_grad"):
        M, C, stream = case["rows"], case["cols"], TYPES[case["s_type"]]
        s["gain"] = 1.0 + _normal(g, (C,), torch.float32, 0.2)
        if op == "norm":
            s["residual"] = _stream(g, M, C, stream) if case["residual"] else None
            s["x"] = _stream(g, M, C, kind)
            s["s_out"] = torch.zeros(M, C, dtype=stream, device=DEVICE) if case["residual"] else None
            s["y_out"] = torch.zeros(M, C, dtype=TYPES[case["y_type"]], device=DEVICE) if case["dense"] else None
            s["kept_out"] = torch.zeros(M, C, dtype=torch.bfloat16, device=DEVICE) if case["kept"] else None
        else:
            s["s"] = _stream(g, M, C, stream)
            s["dy"] = _normal(g, (M, C), kind)
            s["dy2"] = _normal(g, (M, C), kind, 0.3) if case["two"] else None
            s["ds"] = _normal(g, (M, C), stream) if case["stream"] else None
            s["dx_out"] = torch.zeros(M, C, dtype=stream, device=DEVICE)
            s["dgain_out"] = torch.zeros(C, dtype=torch.float32, device=DEVICE)
    elif op in ("choose", "choose_grad"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        logits = _normal(g, (T, E), torch.float32, 1.5) + _normal(g, (E,), torch.float32, 0.5)
        # experts that are off for all tokens, and padding tokens that take none
        logits = torch.where(torch.rand(E, generator=g, device=DEVICE) < case["closed"], -math.inf, logits)
        if case["padded"]:
            logits[T - case["padded"]:] = -math.inf
        s["logits"] = logits.contiguous()
        s["bias"] = _normal(g, (E,), torch.float32, 0.1) if case["bias"] else None
        if op == "choose":
            s["ids_out"] = torch.zeros(T, k, dtype=torch.int32, device=DEVICE)
            s["w_out"] = torch.zeros(T, k, dtype=torch.float32, device=DEVICE)
        else:
            s["ids"] = _plain_choose(s)["ids"]
            s["dw"] = _normal(g, (T, k), torch.float32)
            s["dlogits_out"] = torch.zeros(T, E, dtype=torch.float32, device=DEVICE)
    elif op == "keep":
        s["x"] = _stream(g, case["rows"], case["cols"], kind)
        s["out"] = torch.zeros(case["rows"], case["cols"], dtype=kind, device=DEVICE)
    elif op in ("spread", "act_grad"):
        T, k = case["tokens"], case["k"]
        s["ids"], s["w"] = _routing(case, g)
        s["pair_row"] = _pair_row(s["ids"], case["experts"])
        if op == "spread":
            s["x"] = _rows8(_stream(g, T, case["cols"], torch.float32))
            s["rows_out"] = torch.zeros(T * k, case["cols"], dtype=kind, device=DEVICE)
        else:
            N = case["n_out"]
            R = 2 * N if case["act"] == "swiglu" else N
            s["z"] = _rows8(_normal(g, (T * k, R), torch.float32, 1.5))
            s["dy"] = _normal(g, (T * k, N), kind)
            s["dz_out"] = torch.zeros(T * k, R, dtype=kind, device=DEVICE)
            s["y_out"] = torch.zeros(T * k, N, dtype=kind, device=DEVICE)
            s["dw_out"] = torch.zeros(T, k, dtype=torch.float32, device=DEVICE)
    else:
        M, K, N = case["rows"], case["n_in"], case["n_out"]
        R = 2 * N if case["act"] == "swiglu" else N
        G = case["groups"]
        lead = (G,) if G else ()
        s["start"] = _group_start(case, g) if G else None
        s["longest"] = int((s["start"][1:] - s["start"][:-1]).max()) if G else M
        s["weight"] = _normal(g, lead + (R, K), kind, 1.2 / math.sqrt(K))
        s["bias"] = _normal(g, lead + (R,), torch.float32, 0.1) if case["bias"] else None
        s["x"] = _rows8(_normal(g, (M, K), torch.float32))
        s["z"] = _rows8(_normal(g, (M, R), torch.float32, 1.2)) if case["act"] != "none" else None
        s["dy"] = _normal(g, (M, N), kind)
        s["dx_out"] = torch.zeros(M, K, dtype=kind, device=DEVICE)
        s["dweight_out"] = torch.zeros_like(s["weight"])
        s["dbias_out"] = torch.zeros(lead + (R,), dtype=torch.float32, device=DEVICE) if case["bias"] else None
    if own:
        s["plan"] = _plan(s)
    return s


def _plan(s):
    """The object whose calls a program makes, and what it keeps for them."""
    from bit_vector_quantised_amd.block import ExpertChoice, RmsNorm
    from bit_vector_quantised_amd.dense import ExpertRows, Linear, Rows8
    c = s["case"]
    op = c["op"]
    if op in ("norm", "norm_grad"):
        if op == "norm" and c["kept"]:
            s["kept"] = Rows8(c["rows"], c["cols"], device=DEVICE)
        return RmsNorm(s["gain"], eps=EPS, max_rows=c["rows"], backward=op == "norm_grad")
    if op in ("choose", "choose_grad"):
        return ExpertChoice(c["experts"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                            top_groups=c["top_groups"], best=c["best"], renorm=c["renorm"], scale=c["scale"], device=DEVICE)
    if op == "keep":
        return Rows8(c["rows"], c["cols"], device=DEVICE)
    if op in ("spread", "act_grad"):
        plan = ExpertRows(c["experts"], c["k"], c["tokens"], device=DEVICE)
        plan.sort(s["ids"])
        return plan
    return Linear(s["weight"], s["bias"], act=c["act"], swiglu_limit=LIMIT, max_rows=c["rows"], backward=True, kept8=True)


# ---------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------

def run(s):
    if own:
        return _RUN_OWN[s["case"]["op"]](s)
    return _RUN_PLAIN[s["case"]["op"]](s)


def _there(**outputs):
    return {name: v for name, v in outputs.items() if v is not None}


def _own_norm(s):
    kept = s.get("kept")
    s["plan"].forward(s["x"], residual=s["residual"], s=s["s_out"], out=s["y_out"], rows8=kept,
                      dense=s["y_out"] is not None)
    return _there(s=s["s_out"], y=s["y_out"], kept=None if kept is None else kept.unpack(out=s["kept_out"]))


def _own_norm_grad(s):
    s["plan"].backward(s["s"], s["dy"], dy2=s["dy2"], ds=s["ds"], dx=s["dx_out"], dgain=s["dgain_out"])
    return {"dx": s["dx_out"], "dgain": s["dgain_out"]}


def _own_choose(s):
    s["plan"].forward(s["logits"], ids=s["ids_out"], w=s["w_out"])
    return {"ids": s["ids_out"], "w": s["w_out"]}


def _own_choose_grad(s):
    return {"dlogits": s["plan"].backward(s["logits"], s["ids"], s["dw"], dlogits=s["dlogits_out"])}


def _own_keep(s):
    return {"x": s["plan"].pack(s["x"]).unpack(out=s["out"])}


def _own_spread(s):
    return {"rows": s["plan"].gather(s["x"], s["rows_out"])}


def _own_act_grad(s):
    c = s["case"]
    s["plan"].act_backward(s["z"], s["dy"], s["w"], act=c["act"], swiglu_limit=LIMIT, dz=s["dz_out"], y=s["y_out"],
                           dw=s["dw_out"])
    return {"dz": s["dz_out"], "y": s["y_out"], "dw": s["dw_out"]}


def _own_grad8(s):
    s["plan"].backward(s["x"], s["dy"], z=s["z"], group_start=s["start"], dx=s["dx_out"], dw=s["dweight_out"],
                       dbias=s["dbias_out"])
    return _there(dx=s["dx_out"], dw=s["dweight_out"], dbias=s["dbias_out"])


_RUN_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "choose": _own_choose, "choose_grad": _own_choose_grad,
            "keep": _own_keep, "spread": _own_spread, "act_grad": _own_act_grad, "grad8": _own_grad8}


def _plain_norm(s):
    c = s["case"]
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["gain"]
    return _there(s=v.to(TYPES[c["s_type"]]) if c["residual"] else None, y=y.to(TYPES[c["y_type"]]) if c["dense"] else None,
                  kept=_from8(*_to8(y), c["cols"]).to(torch.bfloat16) if c["kept"] else None)


def _plain_norm_grad(s):
    v = s["s"].float()
    unit = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    dy = s["dy"].float()
    if s["dy2"] is not None:
        dy = dy + s["dy2"].float()
    t = dy * s["gain"]
    dx = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * (t - unit * (t * unit).mean(1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return {"dx": dx.to(TYPES[s["case"]["s_type"]]), "dgain": (dy * unit).sum(0)}


def _scores(s):
    """Scores in 64 bits, as which experts come first may hang on their last places; 0 where an expert is off."""
    logits = s["logits"].double()
    on = logits > -math.inf
    if s["case"]["score"] == "sigmoid":
        return torch.where(on, 1.0 / (1.0 + torch.exp(-logits)), 0.0), on
    top = torch.where(on, logits, -math.inf).amax(1, keepdim=True)
    p = torch.where(on, torch.exp(logits - top), 0.0)
    return torch.where(on, p / p.sum(1, keepdim=True), 0.0), on


def _plain_choose(s):
    c = s["case"]
    T, E, G = c["tokens"], c["experts"], c["groups"]
    score, on = _scores(s)
    value = score if s["bias"] is None else score + s["bias"].double()
    # (without a bias by the logits, which have the scores' order)
    rank = torch.where(on, s["logits"].double() if s["bias"] is None else value, -math.inf)
    if c["top_groups"] < G:
        best = torch.sort(torch.where(on, value, -math.inf).view(T, G, E // G), dim=2, descending=True).values[..., :c["best"]]
        of_group = torch.where(best == -math.inf, 0.0, best).sum(2)
        of_group = torch.where(best[..., 0] == -math.inf, -math.inf, of_group)
        first = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        taken = torch.zeros(T, G, dtype=torch.bool, device=DEVICE).scatter_(1, first, True)
        rank = torch.where(taken.repeat_interleave(E // G, 1), rank, -math.inf)
    rank, ids = torch.sort(rank, dim=1, descending=True, stable=True)
    rank, ids = rank[:, :c["k"]], ids[:, :c["k"]]
    there = rank > -math.inf
    w = torch.where(there, score.gather(1, ids), 0.0)
    if c["renorm"]:
        w = torch.where(there, w / w.sum(1, keepdim=True), 0.0)
    return {"ids": torch.where(there, ids, -1).int(), "w": (w * c["scale"]).float()}


def _plain_choose_grad(s):
    c = s["case"]
    score, _ = _scores(s)
    ids = s["ids"].long()
    there, at = ids >= 0, ids.clamp(min=0)
    p = torch.where(there, score.gather(1, at), 0.0)
    dw = torch.where(there, s["dw"].double() * c["scale"], 0.0)
    if c["renorm"]:
        share = torch.where(there, p / p.sum(1, keepdim=True), 0.0)
        part = share * (dw - (dw * share).sum(1, keepdim=True))
    else:
        part = p * dw
    if c["score"] == "sigmoid":
        part = part * (1.0 - p)
    dlogits = torch.zeros_like(score).scatter_add_(1, at, part)
    if c["score"] == "softmax" and not c["renorm"]:
        dlogits = dlogits - score * part.sum(1, keepdim=True)
    return {"dlogits": dlogits.float()}


def _plain_keep(s):
    return {"x": _from8(*_to8(s["x"]), s["case"]["cols"]).to(TYPES[s["case"]["type"]])}


def _plain_spread(s):
    c = s["case"]
    T, k = c["tokens"], c["k"]
    at = s["pair_row"].long()
    rows = torch.zeros(T * k + 1, c["cols"], dtype=TYPES[c["type"]], device=DEVICE)
    rows[torch.where(at >= 0, at, T * k)] = _from8(*s["x"], c["cols"]).to(rows.dtype).repeat_interleave(k, 0)
    return {"rows": rows[:T * k]}


def _plain_act(z, act):
    """(the activation, its derivative with respect to z or the gate, that with respect to up)"""
    if act == "none":
        return z, torch.ones_like(z), None
    if act == "gelu":
        half = 0.5 * torch.erfc(z * -math.sqrt(0.5))
        return z * half, half + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi), None
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p)), None
    gate, up = z.chunk(2, dim=-1)
    g, u = gate.clamp(max=LIMIT), up.clamp(-LIMIT, LIMIT)
    p = 1.0 / (1.0 + torch.exp(-g))
    return g * p * u, torch.where(gate <= LIMIT, u * p * (1.0 + g * (1.0 - p)), 0.0), torch.where(up.abs() <= LIMIT, g * p, 0.0)


def _plain_dz(z, dy, act):
    y, by_gate, by_up = _plain_act(z, act)
    return y, dy * by_gate if by_up is None else torch.cat((dy * by_gate, dy * by_up), dim=-1)


def _plain_act_grad(s):
    c, kind = s["case"], TYPES[s["case"]["type"]]
    T, k, N = c["tokens"], c["k"], c["n_out"]
    R = 2 * N if c["act"] == "swiglu" else N
    at = s["pair_row"].long()
    there = at >= 0
    # each row's weight; the rows that no pair names are left as they were (zeros)
    w = torch.zeros(T * k + 1, dtype=torch.float32, device=DEVICE)
    w[torch.where(there, at, T * k)] = s["w"].view(-1)
    named = torch.zeros(T * k + 1, dtype=torch.bool, device=DEVICE)
    named[torch.where(there, at, T * k)] = True
    w, named = w[:T * k, None], named[:T * k, None]
    dy = s["dy"].float()
    y, dz = _plain_dz(_from8(*s["z"], R), dy, c["act"])
    dw = torch.where(there, (dy * y).sum(1)[at.clamp(min=0)], 0.0).view(T, k)
    return {"dz": torch.where(named, w * dz, 0.0).to(kind), "y": torch.where(named, w * y, 0.0).to(kind), "dw": dw}


def _padded(s):
    """The rows of each group as [G, longest], and which of them are there."""
    start = s["start"].long()
    at = start[:-1, None] + torch.arange(s["longest"], device=start.device)
    there = at < start[1:, None]
    return torch.where(there, at, 0), there


def _into_groups(s, x):
    at, there = _padded(s)
    return torch.where(there[..., None], x[at], 0.0)


def _from_groups(s, y, rows):
    at, there = _padded(s)
    out = torch.zeros(rows + 1, y.shape[-1], dtype=torch.float32, device=y.device)
    out[torch.where(there, at, rows).view(-1)] = y.reshape(-1, y.shape[-1])
    return out[:rows]


def _plain_grad8(s):
    c, kind = s["case"], TYPES[s["case"]["type"]]
    w, x, dz = s["weight"].float(), _from8(*s["x"], c["n_in"]), s["dy"].float()
    if c["act"] != "none":
        dz = _plain_dz(_from8(*s["z"], w.shape[-2]), dz, c["act"])[1]
    if s["start"] is None:
        dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    else:
        dz = _into_groups(s, dz)
        dx = _from_groups(s, torch.bmm(dz, w), c["rows"])
        dw, db = torch.bmm(dz.transpose(1, 2), _into_groups(s, x)), dz.sum(1)
    return _there(dx=dx.to(kind), dw=dw.to(kind), dbias=db if c["bias"] else None)


_RUN_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "choose": _plain_choose,
              "choose_grad": _plain_choose_grad, "keep": _plain_keep, "spread": _plain_spread,
              "act_grad": _plain_act_grad, "grad8": _plain_grad8}


# ---------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------

def _bytes8(rows, cols):
    return rows * (cols + (cols + 31) // 32)


def work(case):
    op = case["op"]
    size = 2 if case.get("type") == "bf16" else 4
    s_size = 2 if case.get("s_type") == "bf16" else 4
    if op == "norm":
        n = case["rows"] * case["cols"]
        b = n * (size + (2 * s_size if case["residual"] else 0)) + 4 * case["cols"]
        b += n * (2 if case["y_type"] == "bf16" else 4) if case["dense"] else 0
        # (the 8 bits, and the values that are read from them)
        b += _bytes8(case["rows"], case["cols"]) + 2 * n if case["kept"] else 0
        return {"bytes": b, "flops": 5.0 * n}
    if op == "norm_grad":
        n = case["rows"] * case["cols"]
        b = n * (size * (2 if case["two"] else 1) + s_size * (3 if case["stream"] else 2)) + 8 * case["cols"]
        return {"bytes": b, "flops": 10.0 * n}
    if op == "choose":
        T, E, k = case["tokens"], case["experts"], case["k"]
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 4.0 * T * E}
    if op == "choose_grad":
        T, E, k = case["tokens"], case["experts"], case["k"]
        # (which logits are read: all where all have a part in a weight)
        read = T * E if case["score"] == "softmax" and not case["renorm"] else T * k
        return {"bytes": 4 * (read + T * E) + 8 * T * k, "flops": 4.0 * read}
    if op == "keep":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * size * n + _bytes8(case["rows"], case["cols"]), "flops": 2.0 * n}
    if op == "spread":
        P = case["tokens"] * case["k"]
        kept = P * (1.0 - case["dropped"])
        return {"bytes": 4 * P + _bytes8(case["tokens"], case["cols"]) + kept * case["cols"] * size, "flops": kept * case["cols"]}
    N = case["n_out"]
    R = 2 * N if case["act"] == "swiglu" else N
    if op == "act_grad":
        P = case["tokens"] * case["k"]
        kept = P * (1.0 - case["dropped"])
        return {"bytes": 12 * P + _bytes8(kept, R) + kept * (2 * N + R) * size, "flops": 20.0 * kept * N}
    M, K = case["rows"] - min(case["behind"], case["rows"] - 1), case["n_in"]
    G = case["groups"] or 1
    met = G  # groups that have rows, as expected of the draw
    if case["groups"]:
        p = [(1.0 + i) ** -case["skew"] for i in range(G)]
        met = sum(1.0 - (1.0 - v / sum(p)) ** M for v in p)
    b = size * (M * K + met * R * K + G * R * K + M * N) + _bytes8(M, K) + (4 * G * R if case["bias"] else 0)
    b += _bytes8(M, R) if case["act"] != "none" else 0
    return {"bytes": b, "flops": 4.0 * M * R * K}


# ---------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------

def _value8(kept, cols):
    """What the bytes stand for, from the bits: sign, four of exponent, three of fraction."""
    q, e = (t.long() for t in kept)
    high, low = (q >> 3) & 15, (q & 7).double()
    size = torch.where(high == 0, low / 512.0, (1.0 + low / 8.0) * torch.exp2(high.double() - 7.0))
    scale = torch.exp2(e.double() - 127.0).repeat_interleave(32, 1)
    return (torch.where(q >= 128, -size, size) * scale)[:, :cols]


def _round8(x):
    """x rounded to what its bytes would stand for: each value to a multiple of its step, an eighth of the power of
    two at or below it, but at least 2^-9 scales."""
    M, C = x.shape
    out = torch.empty_like(x)
    for at in range(0, C, 32):
        block = x[:, at:at + 32]
        top = block.abs().max(1, keepdim=True).values
        scale = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(min=-110.0))
        scale = torch.where(top > 448.0 * scale, 2.0 * scale, torch.where((top <= 224.0 * scale) & (scale > 2.0 ** -110), 0.5 * scale, scale))
        v = block / scale
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
        out[:, at:at + 32] = torch.round(v / step) * step * scale
    return out


def _exact_norm(s):
    v = s["x"].double()
    if s["residual"] is not None:
        v += s["residual"].double()
    y = v / torch.sqrt(torch.sum(v ** 2, 1) / v.shape[1] + EPS)[:, None] * s["gain"].double()
    c = s["case"]
    return _there(s=v if c["residual"] else None, y=y if c["dense"] else None, kept=_round8(y) if c["kept"] else None)


def _exact_norm_grad(s):
    v, gain = s["s"].double(), s["gain"].double()
    dy = s["dy"].double() + (0.0 if s["dy2"] is None else s["dy2"].double())
    length = torch.sqrt(torch.sum(v ** 2, 1) / v.shape[1] + EPS)[:, None]
    # d(v / length) = dv / length - v (v . dv) / (cols length^3)
    dx = dy * gain / length - v * torch.sum(dy * gain * v, 1)[:, None] / (v.shape[1] * length ** 3)
    if s["ds"] is not None:
        dx += s["ds"].double()
    return {"dx": dx, "dgain": torch.sum(dy * v / length, 0)}


def _exact_score(s):
    l = s["logits"].double()
    if s["case"]["score"] == "sigmoid":
        return torch.sigmoid(l)
    return torch.exp(l - torch.logsumexp(l, 1)[:, None]).nan_to_num(0.0)  # (0 all along where all are off)


def _exact_choose(s):
    """The largest one taken, k times (as many groups first)."""
    c = s["case"]
    T, E, G, k = c["tokens"], c["experts"], c["groups"], c["k"]
    score = _exact_score(s)
    value = score + (0.0 if s["bias"] is None else s["bias"].double())
    value[s["logits"] == -math.inf] = -math.inf
    order = s["logits"].double().clone() if s["bias"] is None else value.clone()
    row = torch.arange(T, device=DEVICE)

    def take(v):
        top = v.amax(1, keepdim=True)
        i = (v == top).to(torch.uint8).argmax(1)  # the first of them
        out = torch.where(top[:, 0] > -math.inf, i, -1)
        v[row, i] = -math.inf
        return out, top[:, 0]

    if c["top_groups"] < G:
        left = value.view(T, G, E // G).reshape(T * G, -1).clone()
        at = torch.arange(T * G, device=DEVICE)
        total, any_there = torch.zeros(T * G, dtype=torch.float64, device=DEVICE), left.amax(1) > -math.inf
        for _ in range(min(c["best"], E // G)):
            top, i = left.max(1)
            total += torch.where(top > -math.inf, top, 0.0)
            left[at, i] = -math.inf
        total[~any_there] = -math.inf
        total = total.view(T, G)
        open_ = torch.zeros(T, G + 1, dtype=torch.bool, device=DEVICE)
        for _ in range(c["top_groups"]):
            i, _top = take(total)
            open_[row, torch.where(i < 0, G, i)] = True
        order[~open_[:, :G].repeat_interleave(E // G, 1)] = -math.inf
    ids = torch.stack([take(order)[0] for _ in range(k)], 1)
    w = torch.zeros(T, k, dtype=torch.float64, device=DEVICE)
    for i in range(k):
        w[:, i] = torch.where(ids[:, i] >= 0, score[row, ids[:, i].clamp(min=0)], 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return {"ids": ids.to(torch.int32), "w": w * c["scale"]}


def _exact_choose_grad(s):
    """By the Jacobian's rows: d score_j / d logit_e, weight by weight."""
    c = s["case"]
    T, E, k = c["tokens"], c["experts"], c["k"]
    score = _exact_score(s)
    row = torch.arange(T, device=DEVICE)
    there = s["ids"] >= 0
    ids = s["ids"].long().clamp(min=0)
    picked = torch.stack([torch.where(there[:, i], score[row, ids[:, i]], 0.0) for i in range(k)], 1)
    back = s["dw"].double() * there * c["scale"]
    if c["renorm"]:
        # w_i = p_i / P: P dp_i = dw_i - sum_j dw_j p_j / P
        P = picked.sum(1, keepdim=True).clamp(min=1e-300)
        back = (back - (back * (picked / P)).sum(1, keepdim=True)) * there / P
    out = torch.zeros(T, E, dtype=torch.float64, device=DEVICE)
    for i in range(k):
        if c["score"] == "sigmoid":
            out[row, ids[:, i]] += back[:, i] * picked[:, i] * (1.0 - picked[:, i])
        else:
            part = back[:, i] * picked[:, i]
            out -= part[:, None] * score
            out[row, ids[:, i]] += part
    return {"dlogits": out}


def _exact_act(z, act):
    """(act(z), its derivative with respect to z or gate, with respect to up) in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z), None
    if act == "gelu":
        half = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * half, half + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi), None
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z), None
    n = z.shape[1] // 2
    gate, up = z[:, :n], z[:, n:]
    g, u = torch.minimum(gate, torch.full_like(gate, LIMIT)), torch.clamp(up, -LIMIT, LIMIT)
    p = torch.sigmoid(g)
    return g * p * u, (gate <= LIMIT) * u * (p + g * p * torch.sigmoid(-g)), ((up >= -LIMIT) & (up <= LIMIT)) * g * p


def _exact_act_grad(s):
    c = s["case"]
    T, k, N = c["tokens"], c["k"], c["n_out"]
    R = 2 * N if c["act"] == "swiglu" else N
    out = {"dz": torch.zeros(T * k, R, dtype=torch.float64, device=DEVICE),
           "y": torch.zeros(T * k, N, dtype=torch.float64, device=DEVICE),
           "dw": torch.zeros(T, k, dtype=torch.float64, device=DEVICE)}
    z = _value8(s["z"], R)
    for i in range(k):
        at = s["pair_row"].view(T, k)[:, i].long()
        t = torch.nonzero(at >= 0).view(-1)
        r = at[t]
        dy, w = s["dy"][r].double(), s["w"][t, i, None].double()
        y, by_gate, by_up = _exact_act(z[r], c["act"])
        out["dw"][t, i] = (dy * y).sum(1)
        out["y"][r] = w * y
        out["dz"][r] = w * dy * by_gate if by_up is None else torch.cat((w * dy * by_gate, w * dy * by_up), dim=1)
    return out


def _exact_grad8(s):
    c = s["case"]
    M, K, N = c["rows"], c["n_in"], c["n_out"]
    R = s["weight"].shape[-2]
    dx = torch.zeros(M, K, dtype=torch.float64, device=DEVICE)
    dw, db = [], []
    at = [0, M] if s["start"] is None else s["start"].tolist()
    q, e = s["x"]
    for g in range(len(at) - 1):
        rows = slice(at[g], at[g + 1])
        w = s["weight"] if s["start"] is None else s["weight"][g]
        dz = s["dy"][rows].double()
        if c["act"] != "none":
            _, by_gate, by_up = _exact_act(_value8((s["z"][0][rows], s["z"][1][rows]), R), c["act"])
            dz = dz * by_gate if by_up is None else torch.cat((dz * by_gate, dz * by_up), dim=1)
        dx[rows] = torch.mm(dz, w.double())
        dw.append(torch.mm(dz.t(), _value8((q[rows], e[rows]), K)))
        db.append(dz.sum(0))
    dw, db = (torch.stack(v) if s["start"] is not None else v[0] for v in (dw, db))
    return _there(dx=dx, dw=dw, dbias=db if c["bias"] else None)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op == "keep":
        return {"x": _round8(s["x"].double())}
    if op == "spread":
        T, k = case["tokens"], case["k"]
        rows = torch.zeros(T * k, case["cols"], dtype=torch.float64, device=DEVICE)
        x = _value8(s["x"], case["cols"])
        for i in range(k):
            at = s["pair_row"].view(T, k)[:, i].long()
            t = torch.nonzero(at >= 0).view(-1)
            rows[at[t]] = x[t]
        return {"rows": rows}
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "choose": _exact_choose,
            "choose_grad": _exact_choose_grad, "act_grad": _exact_act_grad, "grad8": _exact_grad8}[op](s)
