"""The state space operators in 64 bits on the CPU, from their definitions, token by token,
with the sizes that bound a 32-bit evaluation's error.

u = 2^-24 is fp32's unit roundoff.  What the kernels' functions are off by, relative:
  sigmoid(p)      (12 + 2 |p|) u: an exponential of a rounded product (2.5 + 1.3 |p|), 1 + e, the
                  reciprocal, and the rounding of its use
  D = softplus(v) (12 + |v|) u: the exponential (4), the polynomial (3) and three roundings; v = dt +
                  bias itself is rounded, which moves D by |v| u at most (softplus' <= 1 and D >=
                  |v| for v >= 0, D' / D <= 1 for v < 0)
  exp(D A)        (4 + 2 |D A|) u + |D A| times D's
First-order bounds of everything else follow from these; they are doubled at the end for the
second order and for the parts in which long rows are worked on (a part's decay is the exponential
of a sum of D, off by no more than the product of its tokens' decays).
"""
import torch

from lm_reference import U, wide

SLACK = 2.0


def _shift(starts, b, t):
    """Tokens since the document's start, a large number where none has begun."""
    age = torch.full((b, t), 1 << 20, dtype=torch.int64)
    if starts is not None:
        s = starts.cpu() != 0
        for r in range(b):
            n = 1 << 20
            for k in range(t):
                n = 0 if s[r, k] else n + 1
                age[r, k] = n
    return age


def _silu_slope(p):
    s = torch.sigmoid(p)
    return s + p * s * (1 - s)


def _r_sig(p):
    return (12 + 2 * p.abs()) * U


def conv(x, w, bias, state, starts, silu=True):
    """y, last, the bound of y's error, and what the gradient needs."""
    x, w, bias, state = map(wide, (x, w, bias, state))
    (b, t, d), k = x.shape, w.shape[1]
    full = torch.cat([torch.zeros(b, k - 1, d, dtype=torch.float64) if state is None else state, x], 1)
    age = _shift(starts, b, t)
    p = torch.zeros(b, t, d, dtype=torch.float64) + (0.0 if bias is None else bias)
    m = p.abs()
    for j in range(k):  # x_{t-j}
        v = torch.where((age >= j).unsqueeze(-1), full[:, k - 1 - j:k - 1 - j + t], torch.zeros((), dtype=torch.float64))
        p, m = p + v * w[:, k - 1 - j], m + (v * w[:, k - 1 - j]).abs()
    ep = (k + 2) * U * m
    if silu:
        y = p * torch.sigmoid(p)
        bound = 1.1 * ep + y.abs() * _r_sig(p)
    else:
        y, bound = p, ep
    last = full[:, t:].clone()
    if t:
        for i in range(k - 1):
            last[age[:, -1] < k - 2 - i, i] = 0.0
    return y, last, SLACK * bound, (p, ep, full, age)


def conv_grad(dy, x, w, bias, state, starts, dlast, silu=True):
    """(dx, dw, db, dstate) and their bounds."""
    _, _, _, (p, ep, full, age) = conv(x, w, bias, state, starts, silu)
    dy, w, dlast = wide(dy), wide(w), wide(dlast)
    (b, t, d), k = p.shape, w.shape[1]
    if silu:
        s = torch.sigmoid(p)
        q = dy * _silu_slope(p)
        eq = dy.abs() * (0.5 * ep + _r_sig(p) * (s + p.abs() * s) + 4 * U * (s + p.abs() * s))
    else:
        q, eq = dy, 0 * dy
    dfull, efull, mfull = torch.zeros_like(full), torch.zeros_like(full), torch.zeros_like(full)
    dw, ew = torch.zeros_like(w), torch.zeros_like(w)
    n = b * t + 40  # roundings on the way of a sum over tokens
    for j in range(k):
        on = (age >= j).unsqueeze(-1).double()
        at = slice(k - 1 - j, k - 1 - j + t)
        tap = w[:, k - 1 - j]
        dfull[:, at] += on * q * tap
        efull[:, at] += on * eq * tap.abs()
        mfull[:, at] += on * (q * tap).abs()
        v = torch.where(on > 0, full[:, at], torch.zeros((), dtype=torch.float64))
        dw[:, k - 1 - j] = (q * v).sum((0, 1))
        ew[:, k - 1 - j] = (eq * v.abs() + n * U * (q * v).abs()).sum((0, 1))
    if dlast is not None:
        for i in range(k - 1):
            on = (age[:, -1] >= k - 2 - i).double().unsqueeze(-1) if t else 1.0
            dfull[:, t + i] += on * dlast[:, i]
            mfull[:, t + i] += (on * dlast[:, i]).abs()
    efull += (k + 3) * U * mfull
    out = (dfull[:, k - 1:], dw, q.sum((0, 1)), dfull[:, :k - 1])
    bounds = (efull[:, k - 1:], ew, (eq + n * U * q.abs()).sum((0, 1)), efull[:, :k - 1])
    return out, tuple(SLACK * e for e in bounds)


def _per_channel(m, d):
    return m.repeat_interleave(d // m.shape[-2], -2)


def _step_sizes(dt, dt_bias, softplus):
    v = dt if dt_bias is None else dt + dt_bias
    if not softplus:
        return v, v, U * torch.ones_like(v)
    return v, torch.nn.functional.softplus(v, threshold=200.0), (12 + v.abs()) * U


def scan(x, dt, a, b, c, d, z, dt_bias, h0, starts, softplus=True, states=None):
    """y, last, their bounds; `states` collects each token's states for the
    gradient: before it (after a drop) and after it."""
    x, dt, a, b, c, d, z, dt_bias, h0 = map(wide, (x, dt, a, b, c, d, z, dt_bias, h0))
    (rows, t, width), n = x.shape, a.shape[1]
    v, step, rd = _step_sizes(dt, dt_bias, softplus)
    h = torch.zeros(rows, width, n, dtype=torch.float64) if h0 is None else h0
    m, e = h.abs(), torch.zeros_like(h)
    y, ey, my = (torch.zeros(rows, t, width, dtype=torch.float64) for _ in range(3))
    for k in range(t):
        if starts is not None:
            s = (starts[:, k].cpu() != 0)[:, None, None]
            zero = torch.zeros((), dtype=torch.float64)
            h, m, e = torch.where(s, zero, h), torch.where(s, zero, m), torch.where(s, zero, e)
        arg = step[:, k, :, None] * a
        ra = (4 + 2 * arg.abs()) * U + arg.abs() * rd[:, k, :, None]
        decay = torch.exp(arg)
        bk, ck = _per_channel(b[:, k], width), _per_channel(c[:, k], width)
        u = (step[:, k] * x[:, k])[..., None] * bk
        before = (h, m, e)
        h, mp = decay * h + u, m
        m = decay * m + u.abs()
        e = decay * (e + ra * mp) + u.abs() * (rd[:, k, :, None] + 3 * U) + 2 * U * m
        if states is not None:
            states.append((before, (h, m, e)))
        y[:, k] = (h * ck).sum(-1)
        ey[:, k] = (e * ck.abs()).sum(-1)
        my[:, k] = (m * ck.abs()).sum(-1)
    if d is not None:
        y, my = y + d * x, my + (d * x).abs()
    ey = ey + (n + 6) * U * my
    pre = (y, ey)
    if z is not None:
        s = torch.sigmoid(z)
        ey = ey * (z * s).abs() + (y * z * s).abs() * _r_sig(z)
        y = y * z * s
    if states is not None:
        return pre, h
    return y, h, SLACK * ey, SLACK * e


def scan_grad(dy, x, dt, a, b, c, d, z, dt_bias, h0, starts, dlast, softplus=True):
    """(dx, ddt, da, db, dc, dd, dz, ddt_bias, dh0) and their bounds."""
    states = []
    (y, ey), _ = scan(x, dt, a, b, c, d, z, dt_bias, h0, starts, softplus, states)
    dy, x, dt, a, b, c, d, z, dt_bias, dlast = map(wide, (dy, x, dt, a, b, c, d, z, dt_bias, dlast))
    (rows, t, width), n, groups = x.shape, a.shape[1], b.shape[2]
    v, step, rd = _step_sizes(dt, dt_bias, softplus)
    e, ee, dz, ez = dy, 0 * dy, None, None
    if z is not None:
        s = torch.sigmoid(z)
        slope = _silu_slope(z)
        e, ee = dy * z * s, (dy * z * s).abs() * _r_sig(z)
        dz = dy * y * slope
        ez = dy.abs() * (ey * slope.abs() + y.abs() * (_r_sig(z) + 6 * U) * (s + z.abs() * s))
    g = torch.zeros(rows, width, n, dtype=torch.float64) if dlast is None else dlast
    mg, eg = g.abs(), torch.zeros_like(g)
    dx, ddt, edx, eddt = (torch.zeros(rows, t, width, dtype=torch.float64) for _ in range(4))
    db, dc, edb, edc = (torch.zeros(rows, t, groups, n, dtype=torch.float64) for _ in range(4))
    da, eda = torch.zeros_like(a), torch.zeros_like(a)
    deep = rows * t + 60

    def fold(q):
        return q.unflatten(1, (groups, -1)).sum(2)

    for k in range(t - 1, -1, -1):
        bk, ck = _per_channel(b[:, k], width), _per_channel(c[:, k], width)
        sk, rk, xk = step[:, k, :, None], rd[:, k, :, None], x[:, k, :, None]
        ek, eek = e[:, k, :, None], ee[:, k, :, None]
        arg = sk * a
        ra, decay = (4 + 2 * arg.abs()) * U + arg.abs() * rk, torch.exp(arg)
        g, mg = g + ek * ck, mg + (ek * ck).abs()
        eg = eg + eek * ck.abs() + 2 * U * mg
        (hp, mp, ep), (hn, mn, en) = states[k]
        db[:, k] = fold(g * sk * xk)
        edb[:, k] = fold((sk * xk).abs() * (eg + mg * (rk + 200 * U)))
        dc[:, k] = fold(ek * hn)
        edc[:, k] = fold(ek.abs() * (en + mn * 200 * U) + eek * mn)
        along, ea, ma = (g * bk).sum(-1), (eg * bk.abs()).sum(-1), (mg * bk.abs()).sum(-1)
        ea = ea + (n + 8) * U * ma
        q, mq = decay * g * hp, decay * mg * mp
        eq = decay * (eg * mp + mg * ep + mg * mp * (ra + 4 * U))
        through, et = (q * a).sum(-1), ((eq + (n + 8) * U * mq) * a.abs()).sum(-1)
        da += (q * sk).sum(0)
        eda += (sk.abs() * (eq + mq * (rk + deep * U))).sum(0)
        dx[:, k] = step[:, k] * along
        edx[:, k] = step[:, k].abs() * (ea + ma * (rd[:, k] + 4 * U))
        ds, es = x[:, k] * along + through, x[:, k].abs() * (ea + 3 * U * ma) + et + 3 * U * (q * a).abs().sum(-1)
        if softplus:
            sv = torch.sigmoid(v[:, k])
            ddt[:, k], eddt[:, k] = ds * sv, sv * (es + ds.abs() * (_r_sig(v[:, k]) + v[:, k].abs() * U))
        else:
            ddt[:, k], eddt[:, k] = ds, es
        g, eg, mg = decay * g, decay * (eg + mg * (ra + 2 * U)), decay * mg
        if starts is not None:
            on = (starts[:, k].cpu() == 0).double()[:, None, None]
            g, eg, mg = on * g, on * eg, on * mg
    if d is not None:
        dx, edx = dx + d * e, edx + d.abs() * (ee + 3 * U * e.abs())
    out = (dx, ddt, da, db, dc, None if d is None else (e * x).sum((0, 1)), dz,
           None if dt_bias is None else ddt.sum((0, 1)), g)
    bounds = (edx, eddt, eda, edb, edc, ((ee + deep * U * e.abs()) * x.abs()).sum((0, 1)), ez,
              (eddt + deep * U * ddt.abs()).sum((0, 1)), eg)
    return out, tuple(None if q is None else SLACK * q for q in bounds)


def verify(drafts, target, draft, accept, sample, lengths=None):
    """(accepted, tokens), request by request, sums in 64 bits."""
    p, q = wide(target), wide(draft)
    p = torch.where(p > 0, p, torch.zeros_like(p))
    q = None if q is None else torch.where(q > 0, q, torch.zeros_like(q))
    n, k, v = p.shape
    k -= 1
    drafts, accept, sample = drafts.cpu().long(), wide(accept), wide(sample)
    lengths = [k] * n if lengths is None else lengths.cpu().clamp(0, k).tolist()
    tokens, accepted = torch.full((n, k + 1), -1, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)
    for r in range(n):
        i, rest = 0, None
        while i < lengths[r]:
            tok = int(drafts[r, i])
            ok = 0 <= tok < v
            if ok:
                qi = 1.0 if q is None else float(q[r, i, tok])
                ok = float(accept[r, i]) * qi < float(p[r, i, tok])
            if not ok:
                if q is None:
                    rest = p[r, i].clone()
                    if 0 <= tok < v:
                        rest[tok] = 0.0
                else:
                    rest = (p[r, i] - q[r, i]).clamp(min=0)
                break
            tokens[r, i] = tok
            i += 1
        if rest is None:
            rest = p[r, i]
        accepted[r] = i
        sums = rest.cumsum(0)
        if v and float(sums[-1]) > 0:
            tokens[r, i] = int((sums > float(sample[r]) * sums[-1]).int().argmax())
    return accepted, tokens
