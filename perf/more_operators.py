"""Operators of state space language models in this package, as cases that can be timed and checked.

Three operators, in the forms that such a model uses them:

  causal_conv    y_t = silu(bias + sum_k w_k x_{t-K+1+k}), a short convolution of each channel
                 over time: forward ("conv"), gradient ("conv_grad") and the form for one token
                 a call on a pool of states ("conv_step")
  selective_scan h_t = exp(D_t A) h_{t-1} + D_t x_t B_t,  y_t = (C_t . h_t + d x_t) silu(z_t),
                 D_t = softplus(dt_t + bias): forward ("scan"), gradient ("scan_grad") and one
                 token a call ("scan_step")
  verify_drafts  which drafted tokens the target's probabilities accept, and the token after
                 them, from given random numbers ("verify")

listed() and draw() give cases, prepare() what a program holds before the call, run() one
call: of the package's own kernels where `own` is true, else of the plain form below,
elementary torch operations in 32 bits (64 for the verification's sums, whose values decide
between whole numbers).  exact() is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


# ------------------------------------------------------------------ cases ------

def listed():
    return [
        # A training batch through the convolution: its input is half of a projection's rows,
        # several documents in one row.
        {"name": "conv_train", "op": "conv", "dtype": "bf16", "batch": 8, "length": 2048, "channels": 2048,
         "taps": 4, "bias": True, "packed": True, "carried": False},
        # Its gradient, with the sums over all tokens for the weight and the bias.
        {"name": "conv_grad_train", "op": "conv_grad", "dtype": "bf16", "batch": 8, "length": 2048,
         "channels": 2048, "taps": 4, "bias": True, "packed": True, "carried": False},
        # Serving: one token for each of 64 requests, states in a larger pool, some rows padding.
        {"name": "conv_step_64", "op": "conv_step", "dtype": "bf16", "batch": 64, "channels": 4096, "taps": 4,
         "bias": True, "pool": 96},
        # A short prompt through one layer of a small model: latency.
        {"name": "scan_small", "op": "scan", "dtype": "fp32", "batch": 1, "length": 96, "channels": 256,
         "states": 16, "groups": 1, "gated": False, "packed": False, "carried": False, "keep": False},
        # A training batch, which keeps what its gradient needs.
        {"name": "scan_train", "op": "scan", "dtype": "bf16", "batch": 8, "length": 2048, "channels": 2048,
         "states": 16, "groups": 1, "gated": True, "packed": True, "carried": False, "keep": True},
        # One long document continued from a saved state: few rows, a long axis.
        {"name": "scan_long", "op": "scan", "dtype": "bf16", "batch": 1, "length": 32768, "channels": 2048,
         "states": 16, "groups": 1, "gated": True, "packed": False, "carried": True, "keep": False},
        # The gradient of the training batch.
        {"name": "scan_grad_train", "op": "scan_grad", "dtype": "bf16", "batch": 8, "length": 2048,
         "channels": 2048, "states": 16, "groups": 1, "gated": True, "packed": True, "carried": False},
        # A gradient at an odd width, length and number of states, in fp32, with a carried state.
        {"name": "scan_grad_odd", "op": "scan_grad", "dtype": "fp32", "batch": 3, "length": 777, "channels": 1001,
         "states": 13, "groups": 1, "gated": False, "packed": False, "carried": True},
        # Serving: one token for each of 64 requests.
        {"name": "scan_step_64", "op": "scan_step", "dtype": "bf16", "batch": 64, "channels": 4096, "states": 16,
         "groups": 1, "gated": True, "pool": 96},
        # A few requests with four drafted tokens each: latency.
        {"name": "verify_few", "op": "verify", "dtype": "fp32", "batch": 4, "drafts": 4, "vocab": 50021,
         "lookup": False},
        # A serving batch over a large vocabulary.
        {"name": "verify_batch", "op": "verify", "dtype": "fp32", "batch": 128, "drafts": 4, "vocab": 128000,
         "lookup": False},
        # Drafts looked up in the prompt: long, certain, without probabilities of their own.
        {"name": "verify_lookup", "op": "verify", "dtype": "bf16", "batch": 64, "drafts": 10, "vocab": 32000,
         "lookup": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a multiple of 64 mostly, else anything."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.4 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["conv", "conv_grad", "conv_step", "scan", "scan", "scan_grad", "scan_grad", "scan_step",
                     "verify", "verify"])
    case = {"op": op, "dtype": rng.choice(["fp32", "bf16", "bf16", "fp16"])}
    if op == "verify":
        vocab, drafts = _log(rng, 1000, 160000), rng.randint(1, 12)
        batch = min(_log(rng, 1, 256), max(1, (64 << 20) // (vocab * (drafts + 1))))
        return {**case, "batch": batch, "drafts": drafts, "vocab": vocab, "lookup": rng.random() < 0.3}
    if op in ("conv", "conv_grad"):
        channels = _width(rng, 64, 8192)
        room = (32 << 20) // channels
        length = min(_log(rng, 1, 65536), room)
        return {**case, "batch": min(_log(rng, 1, 64), max(1, room // length)), "length": length,
                "channels": channels, "taps": rng.choice([2, 3, 4, 4]), "bias": rng.random() < 0.8,
                "packed": rng.random() < 0.5, "carried": rng.random() < 0.5}
    if op == "conv_step":
        batch = _log(rng, 1, 512)
        return {**case, "batch": batch, "channels": _width(rng, 64, 8192), "taps": rng.choice([2, 3, 4, 4]),
                "bias": rng.random() < 0.8, "pool": batch + rng.randint(0, batch)}
    states, groups = rng.choice([16, 16, 16, 8, 32, 64, rng.randint(1, 40)]), rng.choice([1, 1, 1, 2, 4])
    channels = max(1, _width(rng, 64, 4096) // groups) * groups
    case.update(channels=channels, states=states, groups=groups, gated=rng.random() < 0.7)
    if op == "scan_step":
        batch = min(_log(rng, 1, 512), max(1, (64 << 20) // (channels * states)))
        return {**case, "batch": batch, "pool": batch + rng.randint(0, batch)}
    room = max(1, (256 << 20) // (channels * states))
    length = min(_log(rng, 1, 16384), room)
    case.update(batch=min(_log(rng, 1, 64), max(1, room // length)), length=length,
                packed=rng.random() < 0.5, carried=rng.random() < 0.5)
    if op == "scan":
        case["keep"] = rng.random() < 0.5
    return case


def work(case):
    """Each input read once, each output written once; the operations of the formulas."""
    op, es = case["op"], SIZE[case["dtype"]]
    b = case["batch"]
    if op == "verify":
        # A request's row of probabilities, and the drafter's where it has one.
        rows = 1 if case["lookup"] else 2
        return {"bytes": b * case["vocab"] * rows * es + b * case["drafts"] * (8 + 2 * es) + 4 * b * case["drafts"],
                "flops": 2 * rows * b * case["vocab"]}
    d = case["channels"]
    if op == "conv_step":
        k = case["taps"]
        return {"bytes": b * d * es * (2 + 2 * (k - 1)) + d * (k + 1) * es + 4 * b, "flops": b * d * (2 * k + 6)}
    if op in ("conv", "conv_grad"):
        t, k = case["length"], case["taps"]
        n = (2 if op == "conv" else 3) * b * t * d * es + (b * t if case["packed"] else 0)
        n += (1 if op == "conv" else 2) * d * (k + bool(case["bias"])) * es
        n += (2 if case["carried"] else 1) * b * (k - 1) * d * es
        return {"bytes": n, "flops": b * t * d * ((2 * k + 6) if op == "conv" else (6 * k + 16))}
    n, g, z = case["states"], case["groups"], bool(case["gated"])
    if op == "scan_step":
        return {"bytes": 8 * b * d * n + b * d * (3 + z) * es + 2 * b * g * n * es + 4 * d * (n + 2),
                "flops": b * d * (8 * n + 12)}
    t = case["length"]
    state = 4 * b * d * n
    if op == "scan":
        bytes_ = b * t * (d * (3 + z) * es + 2 * g * n * es) + state * (2 if case["carried"] else 1) + 4 * d * (n + 2)
        return {"bytes": bytes_ + (b * t if case["packed"] else 0), "flops": b * t * d * (8 * n + 12)}
    bytes_ = b * t * (d * (5 + 2 * z) * es + 4 * g * n * es) + state * (3 if case["carried"] else 1) + 8 * d * (n + 2)
    return {"bytes": bytes_ + (b * t if case["packed"] else 0), "flops": b * t * d * (26 * n + 30)}


# ----------------------------------------------------------------- inputs ------

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, mean=0.0, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).add_(mean).to(dtype)


def _slots(g, batch, pool):
    slots = torch.randperm(pool, generator=g, device="cuda")[:batch].to(torch.int32)
    slots[batch - batch // 8:] = -1  # the batch is padded to its size
    return slots


def _starts(g, case):
    if not case["packed"]:
        return None
    return (torch.rand((case["batch"], case["length"]), generator=g, device="cuda") < 1 / 400).to(torch.uint8)


def _prepare_conv(case, g):
    op, dtype = case["op"], DTYPES[case["dtype"]]
    b, d, k = case["batch"], case["channels"], case["taps"]
    s = {"case": case, "w": _normal(g, (d, k), dtype, 0.0, k ** -0.5),
         "bias": _normal(g, (d,), dtype, 0.0, 0.2) if case["bias"] else None}
    if op == "conv_step":
        s["x"] = _normal(g, (b, 2 * d), dtype)[:, :d]
        s["slots"], s["live"] = _slots(g, b, case["pool"]), torch.arange(b - b // 8, device="cuda")
        s["state"] = _normal(g, (case["pool"], k - 1, d), dtype)
        return s
    t = case["length"]
    s["x"] = _normal(g, (b, t, 2 * d), dtype)[..., :d]  # the other half is the gate z
    s["starts"] = _starts(g, case)
    s["state"] = _normal(g, (b, k - 1, d), dtype) if case["carried"] else None
    if op == "conv_grad":
        s["dy"] = _normal(g, (b, t, d), dtype)
        s["dlast"] = _normal(g, (b, k - 1, d), dtype) if case["carried"] else None
    return s


def _prepare_scan(case, g):
    op, dtype = case["op"], DTYPES[case["dtype"]]
    b, d, n, groups = case["batch"], case["channels"], case["states"], case["groups"]
    at = (b,) if op == "scan_step" else (b, case["length"])
    s = {"case": case, "x": _normal(g, at + (d,), dtype), "dt": _normal(g, at + (d,), dtype, 0.0, 0.7)}
    # B and C are slices of one projection's rows, whose first part dt comes from.
    rank = max(8, d // 128 * 8)
    proj = _normal(g, at + (rank + 2 * groups * n,), dtype)
    s["b"] = proj[..., rank:rank + groups * n].unflatten(-1, (groups, n))
    s["c"] = proj[..., rank + groups * n:].unflatten(-1, (groups, n))
    s["z"] = _normal(g, at + (2 * d,), dtype)[..., d:] if case["gated"] else None
    # Decay rates 1 .. states, steps of 0.001 to 0.1.
    s["a"] = -torch.arange(1, n + 1, device="cuda") * torch.exp(_normal(g, (d, n), torch.float32, 0.0, 0.2))
    step = torch.exp(torch.rand((d,), generator=g, device="cuda") * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["d"] = _normal(g, (d,), torch.float32, 1.0, 0.1)
    if op == "scan_step":
        s["slots"], s["live"] = _slots(g, b, case["pool"]), torch.arange(b - b // 8, device="cuda")
        s["state"] = _normal(g, (case["pool"], d, n), torch.float32)
        return s
    s["starts"] = _starts(g, case)
    s["h0"] = _normal(g, (b, d, n), torch.float32) if case["carried"] else None
    if op == "scan_grad":
        s["dy"] = _normal(g, at + (d,), dtype)
        s["dlast"] = _normal(g, (b, d, n), torch.float32) if case["carried"] else None
        if own:  # what the forward pass kept
            import stream_compaction_decoupled_gb300 as gb
            s["kept"] = gb.selective_scan(s["x"], s["dt"], s["a"], s["b"], s["c"], s["d"], s["z"], s["dt_bias"],
                                          h0=s["h0"], starts=s["starts"], keep=True)[2]
    return s


def _prepare_verify(case, g):
    dtype, b, k, v = DTYPES[case["dtype"]], case["batch"], case["drafts"], case["vocab"]
    drafts = torch.empty((b, k), dtype=torch.int64, device="cuda")
    target = torch.empty((b, k + 1, v), dtype=dtype, device="cuda")
    draft = None if case["lookup"] else torch.empty((b, k, v), dtype=dtype, device="cuda")
    for r in range(b):
        logits = _normal(g, (k + 1, v), torch.float32, 0.0, 3.0)
        q = torch.softmax(logits[:k] + _normal(g, (k, v), torch.float32, 0.0, 0.6), 1)
        if r % 5 == 0:  # the target keeps its likelier tokens only
            logits = torch.where(logits > 3.0, logits, float("-inf"))
        target[r] = torch.softmax(logits, 1).to(dtype)
        if case["lookup"]:  # a lookup is right at first, then goes astray
            best = target[r, :k].float().argmax(1)
            astray = torch.randint(0, v, (k,), generator=g, device="cuda")
            drafts[r] = torch.where(torch.rand((k,), generator=g, device="cuda") < 0.7, best, astray)
        else:
            draft[r] = q.to(dtype)
            u = torch.rand((k, 1), generator=g, device="cuda", dtype=torch.float64)
            drafts[r] = torch.searchsorted(q.double().cumsum(1), u * 0.999999).clamp_(max=v - 1).squeeze(1)
    lengths = torch.full((b,), k, dtype=torch.int32, device="cuda")
    lengths[::3] = torch.randint(0, k + 1, (len(lengths[::3]),), generator=g, device="cuda").to(torch.int32)
    return {"case": case, "drafts": drafts, "target": target, "draft": draft, "lengths": lengths,
            "accept": torch.rand((b, k), generator=g, device="cuda"),
            "sample": torch.rand((b,), generator=g, device="cuda")}


def prepare(case, seed):
    g, op = _rng(seed), case["op"]
    if op == "verify":
        return _prepare_verify(case, g)
    return _prepare_conv(case, g) if op.startswith("conv") else _prepare_scan(case, g)


# ------------------------------------------------------------ plain forms ------

def _document(starts):
    """The number of each token's document in its row."""
    return starts.long().cumsum(1)


def _shifted(x, state, k, starts):
    """(x_{t-j} for j = k - 1 .. 0), zero before the state and before the token's document."""
    b, t, d = x.shape
    head = torch.zeros((b, k - 1, d), dtype=torch.float32, device=x.device) if state is None else state.float()
    full = torch.cat([head, x.float()], 1)
    views = [full[:, i:i + t] for i in range(k)]
    if starts is not None:
        doc = _document(starts)
        doc_full = torch.cat([doc.new_zeros((b, k - 1)), doc], 1)
        views = [v * (doc_full[:, i:i + t] == doc).unsqueeze(-1) for i, v in enumerate(views)]
    return views


def _last_inputs(x, state, k, starts):
    b, t, d = x.shape
    head = x.new_zeros((b, k - 1, d)) if state is None else state
    full = torch.cat([head, x], 1)[:, t:]
    if starts is None:
        return full
    doc = _document(starts)
    doc_full = torch.cat([doc.new_zeros((b, k - 1)), doc], 1)
    return full * (doc_full[:, t:] == doc[:, -1:]).unsqueeze(-1).to(x.dtype)


def _pre(views, w, bias):
    p = torch.zeros_like(views[0]) if bias is None else bias.float().expand_as(views[0])
    for i, v in enumerate(views):
        p = p + v * w[:, i].float()
    return p


def _conv(x, w, bias, state, starts):
    k = w.shape[1]
    p = _pre(_shifted(x, state, k, starts), w, bias)
    return (p * torch.sigmoid(p)).to(x.dtype), _last_inputs(x, state, k, starts)


def _conv_grad(dy, x, w, bias, state, starts, dlast):
    (b, t, d), k = x.shape, w.shape[1]
    views = _shifted(x, state, k, starts)
    p = _pre(views, w, bias)
    sg = torch.sigmoid(p)
    dp = dy.float() * sg * (1 + p * (1 - sg))
    dw = torch.stack([(dp * v).sum((0, 1)) for v in views], 1).to(w.dtype)
    full = torch.zeros((b, t + k - 1, d), dtype=torch.float32, device=x.device)
    doc_full = None
    if starts is not None:
        doc = _document(starts)
        doc_full = torch.cat([doc.new_zeros((b, k - 1)), doc], 1)
    for i in range(k):
        c = dp * w[:, i].float()
        if doc_full is not None:
            c = c * (doc_full[:, i:i + t] == doc).unsqueeze(-1)
        full[:, i:i + t] += c
    if dlast is not None:
        c = dlast.float()
        if doc_full is not None:
            c = c * (doc_full[:, t:] == doc[:, -1:]).unsqueeze(-1)
        full[:, t:] += c
    return (full[:, k - 1:].to(x.dtype), dw, None if bias is None else dp.sum((0, 1)).to(bias.dtype),
            None if state is None else full[:, :k - 1].to(x.dtype))


def _conv_step(x, state, w, bias, slots, live):
    at = slots[live].long()
    window = torch.cat([state[at], x[live].unsqueeze(1)], 1)
    p = (window.float() * w.t().float()).sum(1)
    if bias is not None:
        p = p + bias.float()
    state[at] = window[:, 1:]
    y = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
    y[live] = (p * torch.sigmoid(p)).to(x.dtype)
    return y, state


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _per_channel(m, channels):
    """(..., groups, states) to (..., channels, states)."""
    return m.float().repeat_interleave(channels // m.shape[-2], -2)


def _block(batch, channels, states):
    """Tokens at a time: some 32 million states."""
    return max(1, (32 << 20) // (batch * channels * states))


def _affine_scan(a, u, state):
    """h_t = a_t h_{t-1} + u_t along dim 1 from `state`, in log2(T) doubling steps."""
    u[:, 0] += a[:, 0] * state
    s, t = 1, u.shape[1]
    while s < t:
        u = torch.cat([u[:, :s], a[:, s:] * u[:, :-s] + u[:, s:]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return u


def _decays(step, a, starts, lo, hi):
    """(exp(D_t A) with 0 at starts) of tokens lo .. hi."""
    e = torch.exp(step[:, lo:hi].unsqueeze(-1) * a)
    return e if starts is None else e * (starts[:, lo:hi] == 0)[..., None, None]


def _scan(x, dt, a, b, c, d, z, dt_bias, h0, starts, states_out=None):
    (batch, t, width), n = x.shape, a.shape[1]
    xf = x.float()
    step = _softplus(dt.float() + dt_bias)
    h = torch.zeros((batch, width, n), dtype=torch.float32, device=x.device) if h0 is None else h0
    y = torch.empty((batch, t, width), dtype=torch.float32, device=x.device)
    block = _block(batch, width, n)
    for lo in range(0, t, block):
        hi = min(t, lo + block)
        u = (step * xf)[:, lo:hi].unsqueeze(-1) * _per_channel(b[:, lo:hi], width)
        hs = _affine_scan(_decays(step, a, starts, lo, hi), u, h)
        y[:, lo:hi] = (hs * _per_channel(c[:, lo:hi], width)).sum(-1)
        if states_out is not None:
            states_out[:, lo:hi] = hs
        h = hs[:, -1].clone()
    y = y + d * xf
    if states_out is not None:
        return y
    if z is not None:
        y = y * z.float() * torch.sigmoid(z.float())
    return y.to(x.dtype), h


def _to_groups(m, groups):
    """Sums (..., channels, states) over the channels of each group."""
    return m.unflatten(-2, (groups, -1)).sum(-2)


def _scan_grad(dy, x, dt, a, b, c, d, z, dt_bias, h0, starts, dlast):
    (batch, t, width), n, groups = x.shape, a.shape[1], b.shape[2]
    hs = torch.empty((batch, t, width, n), dtype=torch.float32, device=x.device)
    y = _scan(x, dt, a, b, c, d, z, dt_bias, h0, starts, states_out=hs)
    xf, v = x.float(), dt.float() + dt_bias
    step, dy0, dz = _softplus(v), dy.float(), None
    if z is not None:
        zf = z.float()
        sg = torch.sigmoid(zf)
        dz = (dy0 * y * sg * (1 + zf * (1 - sg))).to(x.dtype)
        dy0 = dy0 * zf * sg
    dx, dstep = dy0 * d, torch.empty_like(xf)
    db, dc = (torch.empty((batch, t, groups, n), dtype=torch.float32, device=x.device) for _ in range(2))
    da = torch.zeros_like(a)
    carry = torch.zeros((batch, width, n), dtype=torch.float32, device=x.device) if dlast is None else dlast
    block = _block(batch, width, n)
    for lo in range((t - 1) // block * block, -1, -block):
        hi = min(t, lo + block)
        e = _decays(step, a, starts, lo, hi)
        # From the back: the decay of token k + 1 carries the gradient of its state to token k.
        back = torch.cat([torch.ones_like(e[:, :1]), e[:, 1:].flip(1)], 1)
        g = dy0[:, lo:hi].unsqueeze(-1) * _per_channel(c[:, lo:hi], width)
        g = _affine_scan(back, g.flip(1), carry).flip(1)
        first = hs[:, lo - 1:lo] if lo else (torch.zeros_like(hs[:, :1]) if h0 is None else h0.unsqueeze(1))
        q = g * e * torch.cat([first, hs[:, lo:hi - 1]], 1)  # g a h_{t-1}
        gb = (g * _per_channel(b[:, lo:hi], width)).sum(-1)
        dx[:, lo:hi] += step[:, lo:hi] * gb
        dstep[:, lo:hi] = xf[:, lo:hi] * gb + (q * a).sum(-1)
        da += (q * step[:, lo:hi].unsqueeze(-1)).sum((0, 1))
        db[:, lo:hi] = _to_groups(g * (step * xf)[:, lo:hi].unsqueeze(-1), groups)
        dc[:, lo:hi] = _to_groups(dy0[:, lo:hi].unsqueeze(-1) * hs[:, lo:hi], groups)
        carry = e[:, 0] * g[:, 0]
    ddt = dstep * torch.sigmoid(v)
    return (dx.to(x.dtype), ddt.to(x.dtype), da, db.to(x.dtype), dc.to(x.dtype), (dy0 * xf).sum((0, 1)), dz,
            ddt.sum((0, 1)), carry if h0 is not None else None)


def _scan_step(x, dt, a, b, c, d, z, dt_bias, state, slots, live):
    at, width = slots[live].long(), x.shape[1]
    xf = x[live].float()
    step = _softplus(dt[live].float() + dt_bias)
    h = torch.exp(step.unsqueeze(-1) * a) * state[at]
    h = h + (step * xf).unsqueeze(-1) * _per_channel(b[live], width)
    state[at] = h
    p = (h * _per_channel(c[live], width)).sum(-1) + d * xf
    if z is not None:
        p = p * z[live].float() * torch.sigmoid(z[live].float())
    y = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
    y[live] = p.to(x.dtype)
    return y, state


def _verify(drafts, target, draft, accept, sample, lengths):
    b, k = drafts.shape
    rows = torch.arange(b, device=drafts.device)
    p = target[:, :k].gather(2, drafts.unsqueeze(2)).squeeze(2).double()
    q = torch.ones_like(p) if draft is None else draft.gather(2, drafts.unsqueeze(2)).squeeze(2).double()
    place = torch.arange(k, device=drafts.device)
    ok = (accept.double() * q < p) & (place < lengths.unsqueeze(1))
    accepted = ok.long().cumprod(1).sum(1)
    rest = target[rows, accepted].double()
    if k:
        at = accepted.clamp(max=k - 1)
        if draft is None:
            other = torch.zeros_like(rest).scatter_(1, drafts.gather(1, at.unsqueeze(1)), float("inf"))
        else:
            other = draft[rows, at].double()
        rejected = (accepted < lengths).unsqueeze(1)
        rest = torch.where(rejected, torch.clamp(rest - other, min=0.0), rest)
    total = rest.cumsum(1)
    pick = (total <= sample.double().unsqueeze(1) * total[:, -1:]).sum(1)
    place = torch.arange(k + 1, device=drafts.device)
    tokens = torch.cat([drafts, drafts.new_zeros((b, 1))], 1)
    tokens = torch.where(place < accepted.unsqueeze(1), tokens, -1)
    tokens[rows, accepted] = pick
    return accepted.to(torch.int32), tokens.to(torch.int32)


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(op, s)
    if op == "conv":
        return _conv(s["x"], s["w"], s["bias"], s["state"], s["starts"])
    if op == "conv_grad":
        return _conv_grad(s["dy"], s["x"], s["w"], s["bias"], s["state"], s["starts"], s["dlast"])
    if op == "conv_step":
        return _conv_step(s["x"], s["state"], s["w"], s["bias"], s["slots"], s["live"])
    if op == "verify":
        return _verify(s["drafts"], s["target"], s["draft"], s["accept"], s["sample"], s["lengths"])
    args = [s[k] for k in ("x", "dt", "a", "b", "c", "d", "z", "dt_bias")]
    if op == "scan":
        return _scan(*args, s["h0"], s["starts"])
    if op == "scan_grad":
        return _scan_grad(s["dy"], *args, s["h0"], s["starts"], s["dlast"])
    return _scan_step(*args, s["state"], s["slots"], s["live"])


def _run_own(op, s):
    import stream_compaction_decoupled_gb300 as gb
    if op == "conv":
        return gb.causal_conv(s["x"], s["w"], s["bias"], state=s["state"], starts=s["starts"])
    if op == "conv_grad":
        return gb.causal_conv_backward(s["dy"], s["x"], s["w"], s["bias"], state=s["state"], starts=s["starts"],
                                       dlast=s["dlast"])
    if op == "conv_step":
        return gb.causal_conv_step(s["x"], s["state"], s["w"], s["bias"], slots=s["slots"]), s["state"]
    if op == "verify":
        r = gb.verify_drafts(s["drafts"], s["target"], s["draft"], s["accept"], s["sample"], lengths=s["lengths"])
        return r.accepted, r.tokens
    x, dt, a, b, c, d, z, dt_bias = (s[k] for k in ("x", "dt", "a", "b", "c", "d", "z", "dt_bias"))
    if op == "scan":
        return gb.selective_scan(x, dt, a, b, c, d, z, dt_bias, h0=s["h0"], starts=s["starts"],
                                 keep=s["case"]["keep"])[:2]
    if op == "scan_grad":
        r = gb.selective_scan_backward(s["dy"], x, dt, a, b, c, s["kept"], d, z, dt_bias, starts=s["starts"],
                                       dlast=s["dlast"])
        return (r.dx, r.ddt, r.da, r.db, r.dc, r.dd, r.dz, r.ddt_bias, r.dh0 if s["h0"] is not None else None)
    return gb.selective_scan_step(x, dt, a, b, c, s["state"], d, z, dt_bias, slots=s["slots"]), s["state"]


# ------------------------------------------------- the definition, 64 bits ------

def _silu64(v):
    return v / (1 + torch.exp(-v))


def _exact_conv(s, case):
    op, k = case["op"], case["taps"]
    x, w = s["x"], s["w"]
    if op == "conv_step":
        y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for r in s["live"].tolist():
            slot = int(s["slots"][r])
            v = torch.einsum("kd,dk->d", torch.vstack([s["state"][slot], x[r:r + 1]]), w)
            y[r] = _silu64(v if s["bias"] is None else v + s["bias"])
            s["state"][slot] = torch.vstack([s["state"][slot][1:], x[r:r + 1]])
        return y, s["state"]
    b, t, d = x.shape
    # Where in its document a token is, counting what the state holds before the first.
    place = torch.arange(t, device="cuda").expand(b, t) + (k if s["state"] is not None else 0)
    if s["starts"] is not None:
        begun = torch.where(s["starts"] != 0, torch.arange(t, device="cuda"), -1).cummax(1).values
        place = torch.where(begun >= 0, torch.arange(t, device="cuda") - begun, place)

    def before(j):
        """x_{t-j}, zero where it is not of the token's document."""
        v = torch.zeros((b, t, d), dtype=torch.float64, device="cuda")
        v[:, j:] = x[:, :max(t - j, 0)]
        if s["state"] is not None:
            for r in range(min(j, t)):
                v[:, r] = s["state"][:, k - 1 - j + r]
        return v * (place >= j).unsqueeze(-1)

    v = sum(before(j) * w[:, k - 1 - j] for j in range(k))
    if s["bias"] is not None:
        v = v + s["bias"]
    whole = torch.cat([torch.zeros((b, k - 1, d), dtype=torch.float64, device="cuda") if s["state"] is None
                       else s["state"], x], 1)
    # The newest input is its own place 0; the one r before it counts where the document reaches it.
    reach = torch.arange(k - 2, -1, -1, device="cuda") <= place[:, -1:]
    if op == "conv":
        return _silu64(v), whole[:, t:] * reach.unsqueeze(-1)
    sg = 1 / (1 + torch.exp(-v))
    dv = s["dy"] * (sg + v * sg * (1 - sg))
    dwhole = torch.zeros_like(whole)
    if s["dlast"] is not None:
        dwhole[:, t:] = s["dlast"] * reach.unsqueeze(-1)
    dw = []
    for j in range(k - 1, -1, -1):
        dw.append(torch.einsum("btd,btd->d", dv, before(j)))
        dwhole[:, k - 1 - j:k - 1 - j + t] += dv * w[:, k - 1 - j] * (place >= j).unsqueeze(-1)
    return (dwhole[:, k - 1:], torch.stack(dw, 1), None if s["bias"] is None else dv.sum((0, 1)),
            None if s["state"] is None else dwhole[:, :k - 1])


def _exact_scan(s, case):
    op, width, n, groups = case["op"], case["channels"], case["states"], case["groups"]
    x, a, d, z = s["x"], s["a"], s["d"], s["z"]
    v = s["dt"] + s["dt_bias"]
    step = torch.logaddexp(v, torch.zeros_like(v))
    if op == "scan_step":
        r, at = s["live"], s["slots"][s["live"]].long()
        h = s["state"][at].unflatten(1, (groups, -1)) * torch.exp(step[r].unsqueeze(-1) * a).unflatten(1, (groups, -1))
        h += (step * x)[r].unflatten(1, (groups, -1)).unsqueeze(-1) * s["b"][r].unsqueeze(2)
        s["state"][at] = h.flatten(1, 2)
        y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        y[r] = torch.einsum("bgcn,bgn->bgc", h, s["c"][r]).flatten(1) + d * x[r]
        if z is not None:
            y[r] *= _silu64(z[r])
        return y, s["state"]
    batch, t, _ = x.shape
    if t * batch * width * n > 1200 << 20 or t > 40000:
        return None
    starts = None if s["starts"] is None else (s["starts"] != 0).tolist()

    def drop(m, k):
        if starts is not None:
            for r in range(batch):
                if starts[r][k]:
                    m[r] = 0.0
        return m

    h = torch.zeros((batch, groups, width // groups, n), dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        h += s["h0"].unflatten(1, (groups, -1))
    an = a.unflatten(0, (groups, -1))
    stepg, ug = (m.unflatten(2, (groups, -1)).unsqueeze(-1) for m in (step, step * x))
    y = torch.empty((t, batch, groups, width // groups), dtype=torch.float64, device="cuda")
    grad = op == "scan_grad"
    befores = torch.empty((t,) + h.shape, dtype=torch.float64, device="cuda") if grad else None
    for k in range(t):
        h = drop(h.clone() if starts is not None else h, k)
        if grad:
            befores[k] = h
        h = torch.addcmul(torch.exp(stepg[:, k] * an) * h, ug[:, k], s["b"][:, k].unsqueeze(2))
        torch.matmul(h, s["c"][:, k].unsqueeze(-1), out=y[k].unsqueeze(-1))
    y = y.transpose(0, 1).flatten(2) + d * x
    if not grad:
        return y if z is None else y * _silu64(z), h.flatten(1, 2)
    dy0, dz = s["dy"], None
    if z is not None:
        sg = 1 / (1 + torch.exp(-z))
        dz = s["dy"] * y * (sg + z * sg * (1 - sg))
        dy0 = s["dy"] * z * sg
    dyg = dy0.unflatten(2, (groups, -1)).unsqueeze(-1)
    carry = torch.zeros_like(h) if s["dlast"] is None else s["dlast"].unflatten(1, (groups, -1)).clone()
    along, through = (torch.empty((batch, t, groups, width // groups), dtype=torch.float64, device="cuda")
                      for _ in range(2))
    db, dc = (torch.empty((batch, t, groups, n), dtype=torch.float64, device="cuda") for _ in range(2))
    da = torch.zeros_like(an)
    for k in range(t - 1, -1, -1):
        e = torch.exp(stepg[:, k] * an)
        g = torch.addcmul(carry, dyg[:, k], s["c"][:, k].unsqueeze(2))
        now = torch.addcmul(e * befores[k], ug[:, k], s["b"][:, k].unsqueeze(2))
        db[:, k] = (g * ug[:, k]).sum(2)
        dc[:, k] = (now * dyg[:, k]).sum(2)
        along[:, k] = torch.matmul(g, s["b"][:, k].unsqueeze(-1)).squeeze(-1)
        q = g * e * befores[k]
        through[:, k] = (q * an).sum(-1)
        da += (q * stepg[:, k]).sum(0)
        carry = drop(e * g, k)
    along, through = along.flatten(2), through.flatten(2)
    ddt = (x * along + through) / (1 + torch.exp(-v))
    return (d * dy0 + step * along, ddt, da.flatten(0, 1), db, dc, torch.einsum("btd,btd->d", dy0, x), dz,
            ddt.sum((0, 1)), carry.flatten(1, 2) if s["h0"] is not None else None)


def _exact_verify(s, case):
    """Request by request, draft by draft."""
    k, v = case["drafts"], case["vocab"]
    drafts, lengths, u = s["drafts"].tolist(), s["lengths"].tolist(), s["accept"].double().tolist()
    accepted = torch.zeros((len(drafts),), dtype=torch.int32, device="cuda")
    tokens = torch.full((len(drafts), k + 1), -1, dtype=torch.int32, device="cuda")
    for r, row in enumerate(drafts):
        n, rest = 0, None
        while n < lengths[r]:
            p = s["target"][r, n].double()
            q = torch.zeros_like(p) if s["draft"] is None else s["draft"][r, n].double()
            if s["draft"] is None:
                q[row[n]] = 1.0
            if not u[r][n] * float(q[row[n]]) < float(p[row[n]]):
                rest = torch.where(p > q, p - q, torch.zeros_like(p))
                break
            tokens[r, n] = row[n]
            n += 1
        if rest is None:
            rest = s["target"][r, n].double()
        sums = torch.cumsum(rest, 0)
        tokens[r, n] = int(torch.searchsorted(sums, sums[-1:] * s["sample"][r].double(), right=True)[0])
        accepted[r] = n
    return accepted, tokens


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s, case)
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return _exact_conv(s, case) if case["op"].startswith("conv") else _exact_scan(s, case)
