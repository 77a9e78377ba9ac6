"""The norm, the choice of experts and rows in 8 bits in 64 bits (plain torch on the CPU), with the error that an fp32
evaluation of each may have, element by element.  As in dense_ref.py: HALF[t] is half a step of type t, U an fp32
operation that may truncate; a sum of n terms t_i added in a chain of at most d additions is off by d U sum |t_i|."""
import math

import torch

from dense_ref import HALF, U, act64, act_grad64

# A row's sum: at most 16 terms in a thread, six steps over the wave, sixteen waves.
DEPTH = 16 + 6 + 16


def to8(x):
    """(q, e) of rows x (fp32), by definition; in a block with a value that is not finite only e counts."""
    M, C = x.shape
    pitch = (C + 31) // 32 * 32
    v = torch.zeros(M, pitch, dtype=torch.float64)
    v[:, :C] = x.double()
    v = v.view(M, -1, 32)
    top = v.abs().amax(2)
    fine = torch.isfinite(top)
    e = torch.full(top.shape, -110, dtype=torch.int64)
    for k in range(-110, 121):  # the smallest one that is large enough, found by trying
        e = torch.where(top > 448.0 * 2.0 ** k, k + 1, e)
    q = (v / torch.exp2(e.double())[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(M, pitch), torch.where(fine, e + 127, 255).to(torch.uint8)


def from8(q, e, cols):
    """The values, from the bits."""
    q, e = q.cpu().long(), e.cpu().long()
    high, low = (q >> 3) & 15, (q & 7).double()
    size = torch.where(high == 0, low / 512, (1 + low / 8) * torch.exp2(high.double() - 7))
    size = torch.where((q & 127) == 127, math.nan, size)
    scale = torch.where(e == 255, math.nan, torch.exp2(e.double() - 127)).repeat_interleave(32, 1)
    return (torch.where(q >= 128, -size, size) * scale)[:, :cols]


def norm64(x, res, gain, eps, s_dtype, y_dtype):
    """(s, bound, y, bound of the rounded y, relative bound of the unrounded one)."""
    s = x.double() + (0 if res is None else res.double())
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * gain.double()
    # s: one addition.  Its square's sum is off by DEPTH + 2 U of itself (the terms have one sign) and by twice s's
    # own error; the root halves that; mean, eps, root, division, two products: a few U
    rel = (DEPTH + 2) * U / 2 + 8 * U
    return s, (U + HALF[s_dtype]) * s.abs(), y, (rel + HALF[y_dtype] * (1 + rel)) * y.abs(), rel


def check8(q, e, y, rel, what):
    """Rows in 8 bits against y, whose fp32 evaluation is off by rel |y|: the scale is that of a largest magnitude within
    rel, and each value within half a step of y."""
    cols = y.shape[1]
    low, high = (to8((y * (1 + d)).float())[1].long() for d in (-2 * rel, 2 * rel))
    got = e.cpu().long()
    assert ((got >= low) & (got <= high)).all(), what
    scale = torch.exp2(got.double() - 127).repeat_interleave(32, 1)[:, :cols]
    off = (from8(q, e, cols) - y).abs()
    bound = torch.maximum(y.abs() * (1 + rel) / 16, scale * 2.0 ** -10) + rel * y.abs()
    assert (off <= bound).all(), (what, (off - bound).max())
    pad = q.cpu()[:, cols:]
    assert (pad == 0).all(), what  # the columns behind the last


def norm_backward64(s, gain, eps, dy, dy2, ds, dx_dtype):
    """(dx, bound, dgain, bound)."""
    s, g = s.double(), gain.double()
    M, C = s.shape
    d = dy.double() + (0 if dy2 is None else dy2.double())
    rho = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    t = d * g
    dot, size = (t * s).mean(1, keepdim=True), (t * s).abs().mean(1, keepdim=True)
    through = rho * (t - s * rho * rho * dot)
    rel = (DEPTH + 2) * U / 2 + 8 * U  # of rho
    e = rho * ((rel + 6 * U) * t.abs() + s.abs() * rho * rho * ((3 * rel + 8 * U) * dot.abs() + (DEPTH + 4) * U * size))
    dx = through + (0 if ds is None else ds.double())
    e = e + U * dx.abs()
    part = d * s * rho
    # dgain: at most M rows in a workgroup, as many parts again in 32 shares
    return dx, e + HALF[dx_dtype] * (dx.abs() + e), part.sum(0), (rel + (M + 40) * U) * part.abs().sum(0)


def choose64(logits, bias, k, score="softmax", groups=1, top_groups=1, best=2, renorm=True, scale=1.0):
    """(ids, w, relative bound of w), one token after the other."""
    T, E = logits.shape
    ids, w, rel = torch.full((T, k), -1), torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        l = logits[t].double().tolist()
        b = [0.0] * E if bias is None else bias.double().tolist()
        on = [e for e in range(E) if l[e] > -math.inf and b[e] > -math.inf]
        s = score64(l, on, score)
        value = {e: s[e] + b[e] for e in on}
        order = {e: l[e] if bias is None else value[e] for e in on}
        if top_groups < groups:
            size = E // groups
            of = {}
            for e in on:
                of.setdefault(e // size, []).append(value[e])
            of = {g: sum(sorted(v, reverse=True)[:best]) for g, v in of.items()}
            stay = sorted(of, key=lambda g: (-of[g], g))[:top_groups]
            order = {e: v for e, v in order.items() if e // size in stay}
        first = sorted(order, key=lambda e: (-order[e], e))[:k]
        for j, e in enumerate(first):
            ids[t, j] = e
        for j, (v, r) in enumerate(weights64(l, on, first, score, renorm)):
            w[t, j], rel[t, j] = v * scale, r + 2 * U
    return ids, w, rel


def score64(l, on, score):
    if score == "sigmoid":
        return {e: 1 / (1 + math.exp(-l[e])) if l[e] > -700 else 0.0 for e in on}
    if not on:
        return {}
    top = max(l[e] for e in on)
    p = {e: 1.0 if l[e] == top else math.exp(l[e] - top) for e in on}
    total = sum(p.values())
    return {e: v / total for e, v in p.items()}


def weights64(l, on, first, score, renorm):
    """[(weight before scale, relative bound)] of the chosen experts, by logarithms so that nothing is lost."""
    if not first:
        return []
    if not renorm:
        s = score64(l, on, score)
        if score == "sigmoid":
            return [(s[e], 16 * U) for e in first]
        top = max(l[e] for e in on)
        away = lambda e: 0.0 if l[e] == top else abs(l[e] - top)  # noqa: E731
        return [(s[e], (2 * away(e) + 48) * U) for e in first]
    logs = [l[e] for e in first] if score == "softmax" else \
        [min(l[e], 0.0) - math.log1p(math.exp(-abs(l[e]))) for e in first]
    top = max(logs)
    p = [1.0 if v == top else math.exp(v - top) for v in logs]
    total = sum(p)
    # the logarithms are off by a few U of themselves, their differences by that of both
    most = [0.0 if v == top else max(abs(v), abs(top)) for v in logs]
    return [(v / total, (8 * m + 8 * max(most) + 24 + len(first)) * U) for v, m in zip(p, most)]


def choose_backward64(logits, bias, ids, dw, score="softmax", renorm=True, scale=1.0):
    """(dlogits, bound)."""
    T, E = logits.shape
    out, bound = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        l = logits[t].double().tolist()
        b = [0.0] * E if bias is None else bias.double().tolist()
        on = [e for e in range(E) if l[e] > -math.inf and b[e] > -math.inf]
        at = [j for j, e in enumerate(ids[t].tolist()) if 0 <= e < E and l[e] > -math.inf]
        first = [int(ids[t, j]) for j in at]
        got = weights64(l, on, first, score, renorm)
        d = [float(dw[t, j]) * scale for j in at]
        mean = sum(p * v for (p, _), v in zip(got, d)) if renorm else 0.0
        size = sum(p * abs(v) for (p, _), v in zip(got, d)) if renorm else 0.0
        parts, errs = [], []
        worst = max([r for _, r in got], default=0.0)
        for e, (p, r), v in zip(first, got, d):
            f = 1.0
            if score == "sigmoid":
                f = 1 / (1 + math.exp(l[e])) if l[e] < 700 else 0.0
            parts.append(p * (v - mean) * f)
            errs.append(p * f * (abs(v) + size) * (r + worst + (len(first) + 24) * U))
        for e, v, r in zip(first, parts, errs):
            out[t, e] += v
            bound[t, e] += r
        if score == "softmax" and not renorm:
            s = score64(l, on, score)
            top = max((l[e] for e in on), default=0.0)
            for e in on:
                away = 0.0 if l[e] == top else abs(l[e] - top)
                out[t, e] -= s[e] * sum(parts)
                bound[t, e] += s[e] * (sum(errs) + sum(map(abs, parts)) * (2 * away + 64) * U) + 2 * U * abs(out[t, e])
    return out, bound


def act_backward64(z, dy, pair_row, w, act, lim, dtype):
    """{name: (value, bound)} and the rows that pairs name; z [P, R] as values."""
    P, N = dy.shape
    w = torch.ones(P, dtype=torch.float64) if w is None else w.double().reshape(-1)
    dz, bz = torch.zeros(P, z.shape[1], dtype=torch.float64), torch.zeros(P, z.shape[1], dtype=torch.float64)
    y, by = torch.zeros(P, N, dtype=torch.float64), torch.zeros(P, N, dtype=torch.float64)
    dw, bw = torch.zeros(P, dtype=torch.float64), torch.zeros(P, dtype=torch.float64)
    pairs = [p for p in range(P) if 0 <= int(pair_row[p]) < P]
    rows = [int(pair_row[p]) for p in pairs]
    if pairs:
        zz, d, ww = z[rows].double(), dy[rows].double(), w[pairs][:, None]
        h, eh, _ = act64(zz, act, lim)
        f, ef = act_grad64(zz, act, lim)
        dd = torch.cat((d, d), 1) if act == "swiglu" else d
        v = ww * dd * f
        e = (ww * dd).abs() * ef + 4 * U * v.abs()
        dz[rows], bz[rows] = v, e + HALF[dtype] * (v.abs() + e)
        v, e = ww * h, ww.abs() * eh + 2 * U * (ww * h).abs()
        y[rows], by[rows] = v, e + HALF[dtype] * (v.abs() + e)
        dw[pairs] = (d * h).sum(1)
        bw[pairs] = (d.abs() * eh).sum(1) + (N // 64 + 24) * U * (d * h).abs().sum(1)
    return {"dz": (dz, bz), "y": (y, by), "dw": (dw, bw)}, rows


def experts_backward8_64(x, z, dy, pair_row, start, w, w1, w2, lim, dtype):
    """{name: (value, bound)} of dx, dw, dw1, dw2 of the step from what it kept, as values: tokens x [T, H] and rows z
    [P, R].  Rounded to dtype on the way: dy's rows, dh, w h, dz, dx's rows."""
    T, H = x.shape
    k = w.shape[1]
    P, half = T * k, HALF[dtype]
    pair_row = pair_row.view(T, k)
    x, z, dy, w = x.double(), z.double(), dy.double(), w.double()
    dx, bx = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    dw, bw = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    dw1, b1, dw2, b2 = (torch.zeros(t.shape, dtype=torch.float64) for t in (w1, w1, w2, w2))
    of_row = {int(pair_row[t, i]): (t, i) for t in range(T) for i in range(k) if int(pair_row[t, i]) >= 0}
    for e in range(w1.shape[0]):
        rows = list(range(start[e], start[e + 1]))
        if not rows:
            continue
        tok, place = [of_row[r][0] for r in rows], [of_row[r][1] for r in rows]
        v1, v2 = w1[e].double(), w2[e].double()
        ww = w[tok, place][:, None]
        do = dy[tok]
        edo = half * do.abs()
        dh, size = do @ v2, do.abs() @ v2.abs()
        edh = edo @ v2.abs() + (H + 4) * U * size
        edh = edh + half * (dh.abs() + edh)
        h, eh, _ = act64(z[rows], "swiglu", lim)
        f, ef = act_grad64(z[rows], "swiglu", lim)
        dw[tok, place] = (dh * h).sum(1)
        bw[tok, place] = (edh * (h.abs() + eh) + dh.abs() * eh).sum(1) + (h.shape[1] // 64 + 24) * U * (dh * h).abs().sum(1)
        wh = ww * h
        ewh = ww * eh + 2 * U * wh.abs()
        ewh = ewh + half * (wh.abs() + ewh)
        dd, edd = torch.cat((dh, dh), 1), torch.cat((edh, edh), 1)
        dz = ww * dd * f
        edz = ww * (edd * (f.abs() + ef) + dd.abs() * ef) + 4 * U * dz.abs()
        edz = edz + half * (dz.abs() + edz)
        n = len(rows) + 40

        def product(a, ea, b, eb, n):
            size = a.abs() @ b.abs()
            err = ea @ (b.abs() + eb) + a.abs() @ eb + n * U * size
            v = a @ b
            return v, err + half * (v.abs() + err)

        zero = torch.zeros_like
        dw2[e], b2[e] = product(do.t(), edo.t(), wh, ewh, n)
        dw1[e], b1[e] = product(dz.t(), edz.t(), x[tok], zero(x[tok]), n)
        part, epart = product(dz, edz, v1, zero(v1), v1.shape[0] + 4)
        for r in range(len(rows)):
            dx[tok[r]] += part[r]
            bx[tok[r]] += epart[r] + (k + 1) * U * part[r].abs()
    bx = bx + half * (dx.abs() + bx)
    return {"dx": (dx, bx), "dw": (dw, bw), "dw1": (dw1, b1), "dw2": (dw2, b2)}
