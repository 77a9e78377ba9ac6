"""The row operators and the dense product in 64 bits (plain torch on the CPU), with the
error that an fp32 evaluation of each may have, element by element.

Every bound counts roundings: HALF[t] is half a step of type t relative to a value (the
one rounding of an output), U one fp32 operation that may truncate (the matrix cores' adds
need not round to nearest).  A sum of n terms t_i is off by at most n U sum |t_i|.
"""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -23
# fp32 (and bf16) hold nothing between 0 and 2^-126 but subnormals, which may be flushed: a value
# of exp(-300) times a finite factor is 0 in fp32 and 1e-128 in 64 bits, off by less than this.
TINY = 2.0 ** -126


def act64(z, act, lim=0.0):
    """(value, bound of its evaluation's own error, Lipschitz bound) of rows z [M, R]; for swiglu the
    Lipschitz bounds of gate and up side by side."""
    if act == "none":
        return z, torch.zeros_like(z), torch.ones_like(z)
    if act == "swiglu":
        g, u = z.chunk(2, dim=1)
        if lim > 0:
            g, u = g.clamp(max=lim), u.clamp(-lim, lim)
        h = g * torch.sigmoid(g) * u
        return h, (g.abs() + 8) * 2 * U * h.abs(), torch.cat((1.1 * u.abs(), (g * torch.sigmoid(g)).abs()), 1)
    if act == "silu":
        h = z * torch.sigmoid(z)
        # exp(-z) has a relative error of |z| U from its argument, and a few U from the rest
        return h, (z.abs() + 8) * 2 * U * h.abs(), torch.full_like(z, 1.1)
    h = 0.5 * z * torch.special.erfc(-z / 2.0 ** 0.5)
    # 1 + erf loses what the 1 hides: an absolute error of a few U times |z|
    return h, 8 * U * z.abs(), torch.full_like(z, 1.13)


def act_grad64(z, act, lim=0.0):
    """(factors of dy in dz [M, R], bound of their error) at z [M, R]."""
    if act == "none":
        return torch.ones_like(z), torch.zeros_like(z)
    if act == "swiglu":
        g, u = z.chunk(2, dim=1)
        gin = uin = torch.ones_like(g)
        if lim > 0:
            gin, uin = (g <= lim).to(z), ((u <= lim) & (u >= -lim)).to(z)
            g, u = g.clamp(max=lim), u.clamp(-lim, lim)
        s = torch.sigmoid(g)
        f = torch.cat((gin * u * s * (1 + g * (1 - s)), uin * g * s), 1)
        size = torch.cat((u.abs() * s * (1 + g.abs()), g.abs() * s), 1)
        return f, (torch.cat((g, g), 1).abs() + 8) * 4 * U * size
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s)), (z.abs() + 8) * 4 * U * s * (1 + z.abs())
    phi = torch.exp(-0.5 * z * z) * 0.3989422804014327
    f = 0.5 * torch.special.erfc(-z / 2.0 ** 0.5) + z * phi
    return f, 8 * U * (1 + z.abs()) + (z * z + 8) * 2 * U * z.abs() * phi


def groups_of(M, start):
    return [(0, 0, M)] if start is None else [(g, start[g], start[g + 1]) for g in range(len(start) - 1)]


def linear_forward64(x, w, bias, start, act, lim, residual, y_dtype, z_dtype):
    """(y, bound of y, z, bound of z) on the rows that belong to a group (elsewhere zeros)."""
    x = x.double()
    w3 = w.double().reshape(-1, w.shape[-2], w.shape[-1])
    b2 = None if bias is None else bias.double().reshape(w3.shape[0], -1)
    M, K, R = x.shape[0], x.shape[1], w3.shape[1]
    N = R // 2 if act == "swiglu" else R
    y, by = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    z, bz = torch.zeros(M, R, dtype=torch.float64), torch.zeros(M, R, dtype=torch.float64)
    for g, r0, r1 in groups_of(M, start):
        if r1 <= r0:
            continue
        s = slice(r0, r1)
        zz = x[s] @ w3[g].t()
        size = x[s].abs() @ w3[g].abs().t()
        if b2 is not None:
            zz, size = zz + b2[g], size + b2[g].abs()
        ez = (K + 4) * U * size
        h, eh, lip = act64(zz, act, lim)
        if act == "swiglu":
            # (the second-order term of a product of two slightly wrong factors)
            eh = eh + 1.01 * (lip * ez)[:, :N] + 1.01 * (lip * ez)[:, N:] + 2 * ez[:, :N] * ez[:, N:]
        else:
            eh = eh + lip * ez
        if residual is not None:
            h = h + residual[s].double()
        y[s], by[s] = h, eh + U * h.abs() + HALF[y_dtype] * (h.abs() + eh)
        z[s], bz[s] = zz, ez + HALF[z_dtype] * (zz.abs() + ez)
    return y, by, z, bz


def linear_backward64(x, w, start, act, lim, z, dy, dtype):
    """{name: (value, bound)} of dx, dw, dbias; dz is rounded to dtype for the products."""
    x, dy = x.double(), dy.double()
    shape = w.shape
    w3 = w.double().reshape(-1, shape[-2], shape[-1])
    M, K, R = x.shape[0], x.shape[1], w3.shape[1]
    dx, bx = torch.zeros(M, K, dtype=torch.float64), torch.zeros(M, K, dtype=torch.float64)
    dw, bw = torch.zeros_like(w3), torch.zeros_like(w3)
    db, bb = torch.zeros(w3.shape[0], R, dtype=torch.float64), torch.zeros(w3.shape[0], R, dtype=torch.float64)
    for g, r0, r1 in groups_of(M, start):
        if r1 <= r0:
            continue
        s = slice(r0, r1)
        d = torch.cat((dy[s], dy[s]), 1) if act == "swiglu" else dy[s]
        f, ef = act_grad64(z[s].double(), act, lim) if act != "none" else (torch.ones_like(d), torch.zeros_like(d))
        dz = d * f
        ez = d.abs() * ef + 2 * U * dz.abs()          # unrounded dz (dbias)
        er = ez + HALF[dtype] * (dz.abs() + ez)       # rounded dz (products)
        v, size = dz @ w3[g], dz.abs() @ w3[g].abs()
        e = er @ w3[g].abs() + (R + 4) * U * size
        dx[s], bx[s] = v, e + HALF[dtype] * (v.abs() + e)
        v, size = dz.t() @ x[s], dz.abs().t() @ x[s].abs()
        e = er.t() @ x[s].abs() + (r1 - r0 + 40) * U * size  # (splits of the rows add up to 32 more terms)
        dw[g], bw[g] = v, e + HALF[dtype] * (v.abs() + e)
        db[g] = dz.sum(0)
        bb[g] = ez.sum(0) + (r1 - r0 + 8) * U * dz.abs().sum(0)
    return {"dx": (dx, bx), "dw": (dw.reshape(shape), bw.reshape(shape)),
            "dbias": (db.reshape(shape[:-1]), bb.reshape(shape[:-1]))}


def sort64(ids, n_experts):
    """(start, pair_row, row_pair) as lists, by definition."""
    ids = [int(v) for v in ids]
    pairs = [[p for p, e in enumerate(ids) if e == x] for x in range(n_experts)]
    start = [0]
    for v in pairs:
        start.append(start[-1] + len(v))
    row_pair = [p for v in pairs for p in v]
    pair_row = [-1] * len(ids)
    for r, p in enumerate(row_pair):
        pair_row[p] = r
    return start, pair_row, row_pair + [-1] * (len(ids) - len(row_pair))


def combine64(rows, pair_row, w, residual, T, k, y_dtype):
    """(y, bound)."""
    C = rows.shape[1]
    y = torch.zeros(T, C, dtype=torch.float64) if residual is None else residual.double().clone()
    size = y.abs()
    for t in range(T):
        for i in range(k):
            r = int(pair_row[t * k + i])
            if 0 <= r < T * k:
                part = rows[r].double() * (1.0 if w is None else float(w[t, i]))
                y[t] += part
                size[t] += part.abs()
    e = (k + 1) * U * size
    return y, e + HALF[y_dtype] * (y.abs() + e)


def combine_backward64(dy, pair_row, w, rows, T, k):
    """(drows, bound, named rows, dw, bound)."""
    C = rows.shape[1]
    dt = rows.dtype
    d, bd = torch.zeros(T * k, C, dtype=torch.float64), torch.zeros(T * k, C, dtype=torch.float64)
    dw, bw = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    named = []
    for t in range(T):
        g = dy[t].double()
        for i in range(k):
            r = int(pair_row[t * k + i])
            if not 0 <= r < T * k:
                continue
            named.append(r)
            d[r] = g * (1.0 if w is None else float(w[t, i]))
            bd[r] = (U + HALF[dt]) * d[r].abs()
            p = g * rows[r].double()
            dw[t, i], bw[t, i] = p.sum(), (C + 4) * U * p.abs().sum()
    return d, bd, named, dw, bw


def check(got, want, bound, what):
    got = got.detach().double().cpu()
    off = (got - want).abs()
    bad = ~(off <= bound + TINY)  # (NaN fails)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, off - bound, -1.0).nan_to_num(nan=1e300)).item())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, the worst at {i}: "
                             f"{got.reshape(-1)[i].item()} for {want.reshape(-1)[i].item()}, bound {bound.reshape(-1)[i].item()}")
