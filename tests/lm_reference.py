"""The language-model operators in 64 bits on the CPU, from their definitions, token by
token and row by row, with the sizes that bound a 32-bit evaluation's error.

u = 2^-24 is fp32's unit roundoff.  The kernels' exponential is off by at most 2^-22 + |z| u
relative (the instruction's bound and its argument's rounding), the reciprocal by 2^-23, and
1 + e by u: a sigmoid of |z| <= 8 is off by at most (4 + 8 + 2 + 1) u < 16 u relative, at
either end.
"""
import torch

U = 2.0 ** -24
# The unit roundoff of each output type (24, 8 and 11 significant bits), and half the
# spacing below its normal range (an output may be subnormal).
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0 ** -25}


def wide(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def gates(f, i):
    a = torch.sigmoid(f)
    return a, torch.sigmoid(-f) if i is None else torch.sigmoid(i)


def recurrence(x, f, i, h0, starts):
    """h, last, and the bound of a 32-bit h's error: with every a_t off by 16 u and every
    product and sum by another few u, dh_t <= 20 u (E_t + M_t), M the recurrence of |u x|
    and E_t = a_t (E_{t-1} + M_{t-1}) its sensitivity to the a's."""
    x, f, i, h0 = wide(x), wide(f), wide(i), wide(h0)
    b, t, d = x.shape
    a, u = gates(f, i)
    if starts is not None:
        a = a * (starts.cpu() == 0).unsqueeze(-1)
    state = torch.zeros(b, d, dtype=torch.float64) if h0 is None else h0
    m, e = state.abs(), torch.zeros_like(state)
    hs, bound = torch.zeros(b, t, d, dtype=torch.float64), torch.zeros(b, t, d, dtype=torch.float64)
    for k in range(t):
        ux = u[:, k] * x[:, k]
        state = a[:, k] * state + ux
        e = a[:, k] * (e + m)
        m = a[:, k] * m + ux.abs()
        hs[:, k] = state
        bound[:, k] = 20 * U * (e + m)
    last = bound[:, -1] if t else torch.zeros_like(state)
    return hs, state, bound, last


def recurrence_grad(dh, x, f, h, i, h0, starts, dlast):
    """dx, df, di, dh0 and the bounds of their errors, h being the forward's stored output."""
    dh, x, f, h, i, h0, dlast = map(wide, (dh, x, f, h, i, h0, dlast))
    b, t, d = x.shape
    a, u = gates(f, i)
    keep = a if starts is None else a * (starts.cpu() == 0).unsqueeze(-1)
    c = torch.zeros(b, d, dtype=torch.float64) if dlast is None else dlast
    mc, ec = c.abs(), torch.zeros_like(c)
    g, mg, eg = (torch.zeros(b, t, d, dtype=torch.float64) for _ in range(3))
    for k in range(t - 1, -1, -1):
        g[:, k] = dh[:, k] + c
        mg[:, k] = dh[:, k].abs() + mc
        eg[:, k] = ec
        c, mc, ec = keep[:, k] * g[:, k], keep[:, k] * mg[:, k], keep[:, k] * (ec + mg[:, k])
    err = 20 * U * (eg + mg)
    before = torch.zeros_like(x)
    if t:
        before[:, 1:] = h[:, :-1]
        if h0 is not None:
            before[:, 0] = h0
        if starts is not None:
            before = before * (starts.cpu() == 0).unsqueeze(-1)
    s = a * torch.sigmoid(-f)
    if i is None:
        df, mf, di, mi = s * (before - x) * g, s * (before.abs() + x.abs()), None, None
    else:
        df, mf = s * before * g, s * before.abs()
        si = u * torch.sigmoid(-i)
        di, mi = si * x * g, si * x.abs()
    # Each factor of two sigmoids and a few products: 40 u of the magnitude.
    bounds = [u * err + 20 * U * u * g.abs(), mf * (err + 40 * U * g.abs()),
              None if i is None else mi * (err + 40 * U * g.abs()), 20 * U * (ec + mc)]
    return (u * g, df, di, c), bounds


def layer_norm(x, w, b, eps, depth=80):
    """y, mean, rstd and the bounds: sums of `depth` roundings at most along any path."""
    x, w, b = wide(x), wide(w), wide(b)
    d = x.shape[-1]
    mean = x.mean(-1)
    c = x - mean[:, None]
    var = (c * c).mean(-1)
    rstd = 1 / torch.sqrt(var + eps)
    dm = depth * U * x.abs().mean(-1)
    # var: its own sums, and the mean's error, which enters squared and through the sum of c.
    dv = (depth + 4) * U * var + 2 * dm * c.abs().mean(-1) + dm * dm
    dr = rstd * (dv / (2 * (var + eps)) + 4 * U)
    n = c * rstd[:, None]
    y = n if w is None else n * w + (b if b is not None else 0.0)
    ww = torch.ones(d, dtype=torch.float64) if w is None else w.abs()
    bound = ww * (rstd[:, None] * (dm[:, None] + 2 * U * x.abs()) + c.abs() * dr[:, None] + 2 * U * n.abs()) \
        + 2 * U * y.abs()
    return y, mean, rstd, bound, dm + U * mean.abs(), dr


def layer_norm_grad(dy, x, mean, rstd, w, rows_depth, depth=80):
    """dx, dw, db and bounds, from the given (32-bit) mean and rstd."""
    dy, x, mean, rstd, w = map(wide, (dy, x, mean, rstd, w))
    n = (x - mean[:, None]) * rstd[:, None]
    dn = 4 * U * (n.abs() + rstd[:, None] * x.abs() * U)
    g = dy if w is None else dy * w
    mg, mgn = g.mean(-1, keepdim=True), (g * n).mean(-1, keepdim=True)
    dx = rstd[:, None] * (g - mg - n * mgn)
    bg = depth * U * g.abs().mean(-1, keepdim=True)
    bgn = (depth + 4) * U * (g * n).abs().mean(-1, keepdim=True)
    bound = rstd[:, None] * (6 * U * (g.abs() + mg.abs() + (n * mgn).abs()) + bg + n.abs() * bgn + dn * mgn.abs())
    k = (rows_depth + 60) * U
    return (dx, (dy * n).sum(0), dy.sum(0)), (bound, (k + 8 * U) * (dy * n).abs().sum(0), k * dy.abs().sum(0))


def token_logprobs(logits, targets, top):
    """logprob, entropy, lse, top values and ids (ties to the lower id)."""
    v, t = wide(logits), targets.cpu().long()
    n, width = v.shape
    if width:
        m = v.max(1).values
        none = m == -torch.inf
        d = v - torch.where(none, torch.zeros_like(m), m)[:, None]
        e = d.exp()
        s = e.sum(1)
        lse = torch.where(none, torch.full_like(m, -torch.inf), m + s.log())
        some = torch.where(none, torch.ones_like(s), s)
        p = e / some[:, None]
        lp = d - some.log()[:, None]  # not v - lse: a row near the lowest number swallows log s
    else:
        lse, p, lp = torch.full((n,), -torch.inf, dtype=torch.float64), v, v
    entropy = -(p * torch.where(p > 0, lp, torch.zeros_like(lp))).sum(1)
    ok = (t >= 0) & (t < width)
    at = torch.where(ok, t, torch.zeros_like(t))
    logprob = torch.where(ok, lp.gather(1, at[:, None])[:, 0] if width else lse, torch.zeros_like(lse))
    ids = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :top] if top else None
    return logprob, entropy, lse, lp.gather(1, ids) if top else None, ids, p, lp


def token_logprobs_grad(logits, targets, dlogprob, dentropy):
    _, entropy, lse, _, _, p, lp = token_logprobs(logits, targets, 0)
    t = targets.cpu().long()
    ok = (t >= 0) & (t < p.shape[1]) & (lse > -torch.inf)
    w = torch.zeros(len(t), dtype=torch.float64) if dlogprob is None else wide(dlogprob) * ok
    h = torch.zeros(len(t), dtype=torch.float64) if dentropy is None else wide(dentropy) * (lse > -torch.inf)
    one = torch.zeros_like(p)
    one[torch.arange(len(t)), torch.where(ok, t, torch.zeros_like(t))] = ok.double()
    inner = torch.where(p > 0, lp + entropy[:, None], torch.zeros_like(lp))
    d = w[:, None] * (one - p) - h[:, None] * p * inner
    mag = w.abs()[:, None] * (one + p) + h.abs()[:, None] * p * torch.where(p > 0, lp.abs() + entropy[:, None],
                                                                             torch.zeros_like(lp))
    # p from an exponent lp of 32 bits: off by (4 + 2 |lp|) u relative, and by lse's error.
    lim = torch.where(p > 0, lp.abs(), torch.zeros_like(lp))
    at_lse = 4 * U * (1 + torch.where(lse > -torch.inf, lse.abs(), torch.zeros_like(lse)))
    bound = mag * U * (16 + 4 * lim) + p * (w.abs()[:, None] + h.abs()[:, None] * (1 + lim + entropy[:, None])) \
        * at_lse[:, None]
    return d, bound


def check(got, want, bound, what=""):
    """|got - want| within the bound plus one rounding to got's type, non-finite values equal."""
    g, dt = wide(got), got.dtype
    assert g.shape == want.shape, "%s: shape %s, not %s" % (what, tuple(g.shape), tuple(want.shape))
    fine = torch.isfinite(want)
    assert torch.equal(g[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), what
    assert torch.equal(g.isnan(), want.isnan()), what + ": NaN elsewhere"
    tol = bound + ROUND[dt] * (want.abs() + bound) + TINY[dt]
    bad = fine & ~((g - want).abs() <= tol)
    if bad.any():
        k = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError("%s: %d of %d off, first at %s: got %r want %r (tolerance %.3g)" % (
            what, int(bad.sum()), bad.numel(), k, float(g[k]), float(want[k]),
            float(tol.expand_as(want)[k] if torch.is_tensor(tol) else tol)))
