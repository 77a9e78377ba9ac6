"""Measured cases of the row and dense-product operators: tokens sorted by expert and
back (with their gradients), and the product with bias, activation and residual in its
epilogue, plain or per expert (with its gradients).

A case's "op" is one of
  dispatch   sort the routed pairs by expert, gather the tokens' rows
  collect    y[t] = residual[t] + sum_i w[t, i] rows[pair_row[t, i]]
  rows_grad  the gradients of both: of the rows, of the weights, of the tokens
  linear     y = act(x W^T + b) + residual, with the rows of group g times W[g]
  linear_grad  its gradients: of x, of W, of b

Sizes: hidden 7168, inner 2048, 256 experts, top-8 is this repository's layer shape; 32
experts are an eighth of its layer, as eight devices would hold it; 1, 32 and 4096 tokens
are its decode and prefill batches.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEVICE = "cuda"


# ---------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------

def listed():
    return [
        # one decoded token to its eight experts: nothing but latency
        {"name": "dispatch-one", "op": "dispatch", "tokens": 1, "k": 8, "experts": 256, "cols": 7168, "type": "bf16",
         "dropped": 0.0},
        # a prefill chunk of the layer
        {"name": "dispatch-chunk", "op": "dispatch", "tokens": 4096, "k": 8, "experts": 256, "cols": 7168, "type": "bf16",
         "dropped": 0.0},
        # a decode batch's fp32 expert outputs back to its tokens
        {"name": "collect-batch", "op": "collect", "tokens": 32, "k": 8, "experts": 256, "cols": 7168, "type": "f32",
         "y_type": "f32", "dropped": 0.0, "weighted": True, "residual": False},
        # a prefill chunk added to the shared expert's output
        {"name": "collect-chunk", "op": "collect", "tokens": 4096, "k": 8, "experts": 256, "cols": 7168, "type": "bf16",
         "y_type": "f32", "dropped": 0.0, "weighted": True, "residual": True},
        # a training chunk's way back through both
        {"name": "rows-grad-chunk", "op": "rows_grad", "tokens": 4096, "k": 8, "experts": 256, "cols": 7168, "type": "bf16",
         "y_type": "bf16", "dropped": 0.0},
        # odd in every size, with pairs over an expert's capacity dropped
        {"name": "rows-grad-odd", "op": "rows_grad", "tokens": 1021, "k": 6, "experts": 40, "cols": 2047, "type": "f32",
         "y_type": "f32", "dropped": 0.1},
        # the shared expert's gate and up product for one decoded token
        {"name": "linear-one", "op": "linear", "rows": 1, "groups": 0, "n_in": 7168, "n_out": 2048, "act": "swiglu",
         "type": "bf16", "y_type": "bf16", "bias": False, "residual": False, "keep": False, "skew": 0.0, "behind": 0},
        # a decode batch's pairs at one device's share of the experts, the down product
        {"name": "linear-decode", "op": "linear", "rows": 64, "groups": 32, "n_in": 2048, "n_out": 7168, "act": "none",
         "type": "bf16", "y_type": "f32", "bias": False, "residual": False, "keep": False, "skew": 0.25, "behind": 0},
        # a dense layer's or the shared expert's product in training: bias, and z kept
        {"name": "linear-dense", "op": "linear", "rows": 4096, "groups": 0, "n_in": 7168, "n_out": 2048, "act": "swiglu",
         "type": "bf16", "y_type": "bf16", "bias": True, "residual": False, "keep": True, "skew": 0.0, "behind": 0},
        # a prefill chunk's pairs at one device's share of the experts, unevenly routed
        {"name": "linear-experts", "op": "linear", "rows": 32768, "groups": 32, "n_in": 7168, "n_out": 2048,
         "act": "swiglu", "type": "bf16", "y_type": "bf16", "bias": False, "residual": False, "keep": False, "skew": 0.25,
         "behind": 0},
        # the gradients of a share of the experts
        {"name": "linear-grad-experts", "op": "linear_grad", "rows": 8192, "groups": 16, "n_in": 7168, "n_out": 2048,
         "act": "swiglu", "type": "bf16", "y_type": "bf16", "bias": True, "skew": 0.25, "behind": 0},
        # a small odd layer in fp32
        {"name": "linear-grad-odd", "op": "linear_grad", "rows": 515, "groups": 0, "n_in": 1000, "n_out": 333,
         "act": "gelu", "type": "f32", "y_type": "f32", "bias": True, "skew": 0.0, "behind": 0},
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
    op = rng.choice(("dispatch", "collect", "rows_grad", "linear", "linear", "linear", "linear_grad", "linear_grad"))
    kind = rng.choice(("bf16", "bf16", "bf16", "f32"))
    y_kind = rng.choice((kind, "f32"))
    if op in ("dispatch", "collect", "rows_grad"):
        experts = _spread(rng, 4, 1024)
        k = min(experts, rng.choice((1, 2, 4, 6, 8, 9, 16)))
        cols = _width(rng, 128, 8192)
        most = 4096 * 8 * 7168 * 2 // (k * cols * (2 if kind == "bf16" else 4))
        tokens = _spread(rng, 1, max(1, min(16384, most)))
        case = {"op": op, "tokens": tokens, "k": k, "experts": experts, "cols": cols, "type": kind,
                "dropped": rng.choice((0.0, 0.0, 0.05, 0.3))}
        if op != "dispatch":
            case["y_type"] = y_kind
        if op == "collect":
            case["weighted"], case["residual"] = rng.random() < 0.8, rng.random() < 0.5
        return case
    grad = op == "linear_grad"
    n_in, n_out = _width(rng, 128, 8192), _width(rng, 64, 4096)
    act = rng.choice(("none", "silu", "gelu", "swiglu", "swiglu"))
    wide = n_out * (2 if act == "swiglu" else 1)
    groups = rng.choice((0, 0, _spread(rng, 2, 64)))
    while groups * n_in * wide > 16 * 7168 * 4096:
        groups //= 2
    most = (9e11 if kind == "bf16" else 6e10) / ((4 if grad else 2) * n_in * wide)
    rows = _spread(rng, 1, max(1, min(32768, int(most))))
    case = {"op": op, "rows": rows, "groups": groups, "n_in": n_in, "n_out": n_out, "act": act, "type": kind,
            "y_type": y_kind, "bias": rng.random() < 0.6, "skew": rng.choice((0.0, 0.25, 0.5)),
            "behind": rng.choice((0, 0, 5)) if groups else 0}
    if not grad:
        case["residual"], case["keep"] = rng.random() < 0.5, rng.random() < 0.4
    return case


# ---------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------

def _normal(g, shape, dtype, scale=1.0):
    # (drawn in fp32 slices: a device's experts are gigabytes)
    out = torch.empty(shape, dtype=dtype, device=DEVICE)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - at)
        flat[at:at + n] = torch.randn(n, generator=g, device=DEVICE).mul_(scale)
    return out


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


def _group_start(case, g):
    """The rows of each group: sizes by a power of the group's rank; "behind" rows at the
    end belong to none."""
    G, rows = case["groups"], case["rows"] - min(case["behind"], case["rows"] - 1)
    p = (1.0 + torch.randperm(G, generator=g, device=DEVICE).double()) ** -case["skew"]
    group = torch.multinomial(p / p.sum(), rows, replacement=True, generator=g)
    start = torch.zeros(G + 1, dtype=torch.int64, device=DEVICE)
    start[1:] = torch.cumsum(torch.bincount(group, minlength=G), 0)
    return start.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 7919 + 17)
    op, kind = case["op"], TYPES[case["type"]]
    y_kind = TYPES[case.get("y_type", case["type"])]
    s = {"case": dict(case)}
    if op in ("dispatch", "collect", "rows_grad"):
        T, k, C = case["tokens"], case["k"], case["cols"]
        s["ids"], s["w"] = _routing(case, g)
        if op == "dispatch":
            s["x"] = _normal(g, (T, C), kind)
            s["rows_out"] = torch.zeros(T * k, C, dtype=kind, device=DEVICE)
        else:
            s["rows"] = _normal(g, (T * k, C), kind)
            # where the sort, which ran before the experts, put each pair
            ids = s["ids"].view(-1).long()
            key = torch.where(ids < 0, case["experts"], ids)
            order = torch.argsort(key, stable=True)
            at = torch.empty_like(order)
            at[order] = torch.arange(T * k, device=DEVICE)
            s["pair_row"] = torch.where(ids < 0, -1, at).to(torch.int32)
            s["y_out"] = torch.zeros(T, C, dtype=y_kind, device=DEVICE)
            if op == "collect":
                s["residual"] = _normal(g, (T, C), y_kind) if case["residual"] else None
            else:
                s["dy"] = _normal(g, (T, C), y_kind)
                s["drows"] = _normal(g, (T * k, C), kind)
                s["rows_out"] = torch.zeros(T * k, C, dtype=kind, device=DEVICE)
                s["dx_out"] = torch.zeros(T, C, dtype=kind, device=DEVICE)
                s["dw_out"] = torch.zeros(T, k, dtype=torch.float32, device=DEVICE)
    else:
        M, K, N = case["rows"], case["n_in"], case["n_out"]
        R = 2 * N if case["act"] == "swiglu" else N
        G = case["groups"]
        lead = (G,) if G else ()
        s["start"] = _group_start(case, g) if G else None
        s["longest"] = int((s["start"][1:] - s["start"][:-1]).max()) if G else M
        s["filled"] = int(s["start"][-1]) if G else M
        s["x"] = _normal(g, (M, K), kind)
        s["weight"] = _normal(g, lead + (R, K), kind, 1.2 / math.sqrt(K))
        s["bias"] = _normal(g, lead + (R,), torch.float32, 0.1) if case["bias"] else None
        if op == "linear":
            s["residual"] = _normal(g, (M, N), y_kind) if case["residual"] else None
            s["y_out"] = torch.zeros(M, N, dtype=y_kind, device=DEVICE)
            s["z_out"] = torch.zeros(M, R, dtype=kind, device=DEVICE) if case["keep"] else None
        else:
            s["z"] = _normal(g, (M, R), kind, 1.2)
            s["dy"] = _normal(g, (M, N), y_kind)
            s["dx_out"] = torch.zeros(M, K, dtype=kind, device=DEVICE)
            s["dweight_out"] = torch.zeros_like(s["weight"])
            s["dbias_out"] = torch.zeros(lead + (R,), dtype=torch.float32, device=DEVICE) if case["bias"] else None
    if own:
        from bit_vector_quantised_amd.dense import ExpertRows, Linear
        if op in ("dispatch", "collect", "rows_grad"):
            s["plan"] = ExpertRows(case["experts"], case["k"], case["tokens"], device=DEVICE)
            if op != "dispatch":
                s["plan"].sort(s["ids"])
        else:
            s["plan"] = Linear(s["weight"], s["bias"], act=case["act"], swiglu_limit=LIMIT, max_rows=case["rows"],
                               backward=op == "linear_grad")
    return s


LIMIT = 7.0  # the SwiGLU clamp of the cases that have that activation


# ---------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------

def run(s):
    if own:
        return _RUN_OWN[s["case"]["op"]](s)
    return _RUN_PLAIN[s["case"]["op"]](s)


def _own_dispatch(s):
    p = s["plan"]
    p.sort(s["ids"])
    p.gather(s["x"], s["rows_out"])
    T = s["ids"].shape[0]
    P = T * s["case"]["k"]
    return {"start": p.expert_start, "pair_row": p.pair_row[:P], "row_pair": p.row_pair[:P], "rows": s["rows_out"]}


def _own_collect(s):
    w = s["w"] if s["case"]["weighted"] else None
    return {"y": s["plan"].combine(s["rows"], w, s["residual"], s["y_out"])}


def _own_rows_grad(s):
    p = s["plan"]
    p.combine_backward(s["dy"], s["w"], s["rows"], s["rows_out"], s["dw_out"])
    p.gather_backward(s["drows"], s["dx_out"])
    return {"drows": s["rows_out"], "dw": s["dw_out"], "dx": s["dx_out"]}


def _own_linear(s):
    s["plan"].forward(s["x"], group_start=s["start"], residual=s["residual"], out=s["y_out"], z=s["z_out"])
    return {"y": s["y_out"]} if s["z_out"] is None else {"y": s["y_out"], "z": s["z_out"]}


def _own_linear_grad(s):
    s["plan"].backward(s["x"], s["dy"], z=s["z"], group_start=s["start"], dx=s["dx_out"], dw=s["dweight_out"],
                       dbias=s["dbias_out"])
    out = {"dx": s["dx_out"], "dw": s["dweight_out"]}
    return out if s["dbias_out"] is None else out | {"dbias": s["dbias_out"]}


_RUN_OWN = {"dispatch": _own_dispatch, "collect": _own_collect, "rows_grad": _own_rows_grad, "linear": _own_linear,
            "linear_grad": _own_linear_grad}


def _plain_dispatch(s):
    E, k = s["case"]["experts"], s["case"]["k"]
    ids = s["ids"].view(-1).long()
    P = ids.numel()
    key = torch.where((ids < 0) | (ids >= E), E, ids)
    order = torch.argsort(key, stable=True)
    at = torch.empty_like(order)
    at[order] = torch.arange(P, device=ids.device)
    counts = (key[None, :] == torch.arange(E, device=ids.device)[:, None]).sum(1) if P <= 1 << 14 else \
        torch.zeros(E + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))[:E]
    start = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    start[1:] = torch.cumsum(counts, 0)
    valid = torch.arange(P, device=ids.device) < start[E]
    rows = torch.where(valid[:, None], s["x"][order // k], 0)
    return {"start": start.int(), "pair_row": torch.where(key == E, -1, at).int(),
            "row_pair": torch.where(valid, order, -1).int(), "rows": rows}


def _plain_back(rows, pair_row, w, T, k):
    """sum_i w[t, i] rows[pair_row[t, i]] in fp32; a dropped pair adds nothing."""
    at = pair_row.long()
    part = torch.where((at >= 0)[:, None], rows[at.clamp(min=0)].float(), 0.0)
    if w is not None:
        part = part * w.reshape(-1, 1)
    return part.view(T, k, -1).sum(1)


def _plain_collect(s):
    c = s["case"]
    y = _plain_back(s["rows"], s["pair_row"], s["w"] if c["weighted"] else None, c["tokens"], c["k"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(TYPES[c["y_type"]])}


def _plain_rows_grad(s):
    c = s["case"]
    T, k, kind = c["tokens"], c["k"], TYPES[c["type"]]
    at = s["pair_row"].long()
    kept = at >= 0
    dy = s["dy"].float().repeat_interleave(k, 0)
    dw = torch.where(kept, (dy * s["rows"][at.clamp(min=0)].float()).sum(1), 0.0).view(T, k)
    drows = torch.zeros(T * k + 1, c["cols"], dtype=kind, device=dy.device)
    drows[torch.where(kept, at, T * k)] = (dy * s["w"].reshape(-1, 1)).to(kind)
    dx = _plain_back(s["drows"], s["pair_row"], None, T, k).to(kind)
    return {"drows": drows[:T * k], "dw": dw, "dx": dx}


def _padded(s):
    """The rows of each group as [G, longest], and which of them are there."""
    start = s["start"].long()
    at = start[:-1, None] + torch.arange(s["longest"], device=start.device)
    there = at < start[1:, None]
    return torch.where(there, at, 0), there


def _into_groups(s, x):
    at, there = _padded(s)
    return torch.where(there[..., None], x[at].float(), 0.0)


def _from_groups(s, y, rows):
    at, there = _padded(s)
    out = torch.zeros(rows + 1, y.shape[-1], dtype=torch.float32, device=y.device)
    out[torch.where(there, at, rows).view(-1)] = y.reshape(-1, y.shape[-1])
    return out[:rows]


def _plain_act(z, act):
    if act == "none":
        return z
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    gate, up = z.chunk(2, dim=-1)
    gate, up = gate.clamp(max=LIMIT), up.clamp(-LIMIT, LIMIT)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_linear(s):
    c = s["case"]
    w = s["weight"].float()
    if s["start"] is None:
        z = s["x"].float() @ w.t()
        z = z if s["bias"] is None else z + s["bias"]
    else:
        z = torch.bmm(_into_groups(s, s["x"]), w.transpose(1, 2))
        z = z if s["bias"] is None else z + s["bias"][:, None, :]
        z = _from_groups(s, z, c["rows"])
    y = _plain_act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if s["filled"] < c["rows"]:  # rows that belong to no group stay as they were
        y[s["filled"]:] = 0.0
    y = y.to(TYPES[c["y_type"]])
    return {"y": y, "z": z.to(TYPES[c["type"]])} if c["keep"] else {"y": y}


def _plain_dz(z, dy, act):
    if act == "none":
        return dy
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return dy * p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return dy * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    gate, up = z.chunk(2, dim=-1)
    g, u = gate.clamp(max=LIMIT), up.clamp(-LIMIT, LIMIT)
    p = 1.0 / (1.0 + torch.exp(-g))
    dgate = torch.where(gate <= LIMIT, dy * u * p * (1.0 + g * (1.0 - p)), 0.0)
    dup = torch.where(up.abs() <= LIMIT, dy * g * p, 0.0)
    return torch.cat((dgate, dup), dim=-1)


def _plain_linear_grad(s):
    c, kind = s["case"], TYPES[s["case"]["type"]]
    w, dz = s["weight"].float(), _plain_dz(s["z"].float(), s["dy"].float(), c["act"])
    if s["start"] is None:
        dx, dw, db = dz @ w, dz.t() @ s["x"].float(), dz.sum(0)
    else:
        dz = _into_groups(s, dz)
        dx = _from_groups(s, torch.bmm(dz, w), c["rows"])
        dw, db = torch.bmm(dz.transpose(1, 2), _into_groups(s, s["x"])), dz.sum(1)
    out = {"dx": dx.to(kind), "dw": dw.to(kind)}
    return out | {"dbias": db} if c["bias"] else out


_RUN_PLAIN = {"dispatch": _plain_dispatch, "collect": _plain_collect, "rows_grad": _plain_rows_grad,
              "linear": _plain_linear, "linear_grad": _plain_linear_grad}


# ---------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------

def work(case):
    size = 2 if case["type"] == "bf16" else 4
    y_size = 2 if case.get("y_type", case["type"]) == "bf16" else 4
    op = case["op"]
    if op in ("dispatch", "collect", "rows_grad"):
        T, P, C = case["tokens"], case["tokens"] * case["k"], case["cols"]
        kept = P * (1.0 - case["dropped"])
        if op == "dispatch":
            return {"bytes": 12 * P + 4 * case["experts"] + T * C * size + kept * C * size, "flops": 0}
        if op == "collect":
            return {"bytes": (8 if case["weighted"] else 4) * P + kept * C * size
                    + T * C * y_size * (2 if case["residual"] else 1), "flops": 2.0 * kept * C}
        return {"bytes": 16 * P + T * C * y_size + 3 * kept * C * size + T * C * size, "flops": 4.0 * kept * C}
    M, K, N = case["rows"], case["n_in"], case["n_out"]
    M -= min(case["behind"], M - 1)
    R = 2 * N if case["act"] == "swiglu" else N
    G = case["groups"] or 1
    met = G  # groups that have rows, as expected of the draw
    if case["groups"]:
        p = [(1.0 + i) ** -case["skew"] for i in range(G)]
        met = sum(1.0 - (1.0 - v / sum(p)) ** M for v in p)
    if op == "linear":
        b = size * (M * K + met * R * K) + y_size * M * N * (2 if case["residual"] else 1)
        b += size * M * R if case["keep"] else 0
        return {"bytes": b + (4 * R * met if case["bias"] else 0), "flops": 2.0 * M * R * K}
    b = size * (2 * M * K + met * R * K + G * R * K) + y_size * M * N + (4 * G * R if case["bias"] else 0)
    b += size * M * R if case["act"] != "none" else 0
    return {"bytes": b, "flops": 4.0 * M * R * K}


# ---------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------

def _exact_back(rows, pair_row, w, T, k):
    """Added up slot by slot of a token."""
    y = torch.zeros(T, rows.shape[1], dtype=torch.float64, device=rows.device)
    for i in range(k):
        at = pair_row.view(T, k)[:, i].long()
        t = torch.nonzero(at >= 0).view(-1)
        part = rows[at[t]].double()
        y[t] += part if w is None else part * w[t, i, None].double()
    return y


def _exact_dispatch(s):
    c = s["case"]
    T, k, E = c["tokens"], c["k"], c["experts"]
    rows = torch.zeros(T * k, c["cols"], dtype=torch.float64, device=DEVICE)
    ids = s["ids"].view(-1).tolist()
    lists = [[] for _ in range(E)]
    for p, e in enumerate(ids):
        if 0 <= e < E:
            lists[e].append(p)
    row_pair = [p for pairs in lists for p in pairs]
    if row_pair:
        rows[:len(row_pair)] = s["x"][torch.tensor(row_pair, device=DEVICE) // k].double()
    start, pair_row = [0], [-1] * (T * k)
    for pairs in lists:
        start.append(start[-1] + len(pairs))
    for r, p in enumerate(row_pair):
        pair_row[p] = r
    row_pair += [-1] * (T * k - len(row_pair))
    whole = [torch.tensor(v, dtype=torch.int32) for v in (start, pair_row, row_pair)]
    return {"start": whole[0], "pair_row": whole[1], "row_pair": whole[2], "rows": rows}


def _exact_rows_grad(s):
    c = s["case"]
    T, k = c["tokens"], c["k"]
    drows = torch.zeros(T * k, c["cols"], dtype=torch.float64, device=DEVICE)
    dw = torch.zeros(T, k, dtype=torch.float64, device=DEVICE)
    for i in range(k):
        at = s["pair_row"].view(T, k)[:, i].long()
        t = torch.nonzero(at >= 0).view(-1)
        dy = s["dy"][t].double()
        dw[t, i] = (dy * s["rows"][at[t]].double()).sum(1)
        drows[at[t]] = dy * s["w"][t, i, None].double()
    return {"drows": drows, "dw": dw, "dx": _exact_back(s["drows"], s["pair_row"], None, T, k)}


def _exact_product(s):
    """(group's weight, its rows' slice, its bias) of every group."""
    if s["start"] is None:
        return [(s["weight"], slice(0, s["case"]["rows"]), s["bias"])]
    at = s["start"].tolist()
    return [(s["weight"][g], slice(at[g], at[g + 1]), None if s["bias"] is None else s["bias"][g])
            for g in range(len(at) - 1)]


def _exact_act(z, act):
    """(act(z), its derivative with respect to gate, with respect to up) in 64 bits."""
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


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op == "dispatch":
        return _exact_dispatch(s)
    if op == "collect":
        y = _exact_back(s["rows"], s["pair_row"], s["w"] if case["weighted"] else None, case["tokens"], case["k"])
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    if op == "rows_grad":
        return _exact_rows_grad(s)
    M, K, N = case["rows"], case["n_in"], case["n_out"]
    R = 2 * N if case["act"] == "swiglu" else N
    if op == "linear":
        y = torch.zeros(M, N, dtype=torch.float64, device=DEVICE)
        z = torch.zeros(M, R, dtype=torch.float64, device=DEVICE)
        for w, rows, bias in _exact_product(s):
            z[rows] = torch.mm(s["x"][rows].double(), w.double().t())
            if bias is not None:
                z[rows] += bias.double()
            y[rows] = _exact_act(z[rows], case["act"])[0]
            if s["residual"] is not None:
                y[rows] += s["residual"][rows].double()
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    dx = torch.zeros(M, K, dtype=torch.float64, device=DEVICE)
    dw, db = [], []
    for w, rows, _ in _exact_product(s):
        dy = s["dy"][rows].double()
        _, by_gate, by_up = _exact_act(s["z"][rows].double(), case["act"])
        dz = dy * by_gate if by_up is None else torch.cat((dy * by_gate, dy * by_up), dim=1)
        dx[rows] = torch.mm(dz, w.double())
        dw.append(torch.mm(dz.t(), s["x"][rows].double()))
        db.append(dz.sum(0))
    dw, db = (torch.stack(v) if s["start"] is not None else v[0] for v in (dw, db))
    return {"dx": dx, "dw": dw, "dbias": db} if case["bias"] else {"dx": dx, "dw": dw}
