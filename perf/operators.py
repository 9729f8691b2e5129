"""The language-model operators of this package, as cases that can be timed and checked.

Three operators, in the forms a recurrent language model uses them:

  recurrence   h_t = a_t h_{t-1} + u_t x_t,  a = sigmoid(f),  u = sigmoid(i) or 1 - a:
               forward ("recurrence"), gradient ("recurrence_grad") and the form for one
               token a call on a pool of states ("recurrence_step")
  layer norm   y = (x - mean) rstd w + b: forward ("norm") and gradient ("norm_grad")
  log probabilities of given tokens with the entropy and the top alternatives of each row
               of logits: forward ("logprob") and gradient ("logprob_grad")

listed() and draw() give cases, prepare() what a program holds before the call, run() one
call: of the package's own kernels where `own` is true, else of the plain form below,
elementary torch operations in 32 bits.  exact() is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
EPS = 1e-5
NEG = float("-inf")


# ------------------------------------------------------------------ cases ------

def listed():
    return [
        # A short prompt through one layer of a small model: launch and latency.
        {"name": "recurrence_small", "op": "recurrence", "dtype": "fp32", "batch": 1, "length": 96,
         "channels": 256, "input_gate": False, "packed": False, "carried": False},
        # A training batch: gates and input are slices of one fused projection.
        {"name": "recurrence_train", "op": "recurrence", "dtype": "bf16", "batch": 8, "length": 2048,
         "channels": 2048, "input_gate": True, "packed": True, "carried": False},
        # One long document continued from a saved state: few channels' worth of rows, a long axis.
        {"name": "recurrence_long", "op": "recurrence", "dtype": "bf16", "batch": 1, "length": 65536,
         "channels": 2048, "input_gate": True, "packed": False, "carried": True},
        # The gradient of the training batch.
        {"name": "recurrence_grad_train", "op": "recurrence_grad", "dtype": "bf16", "batch": 8, "length": 2048,
         "channels": 2048, "input_gate": True, "packed": True, "carried": False},
        # A gradient at an odd width and length, in fp32, with a carried state.
        {"name": "recurrence_grad_odd", "op": "recurrence_grad", "dtype": "fp32", "batch": 3, "length": 1537,
         "channels": 1001, "input_gate": False, "packed": False, "carried": True},
        # Serving: one token for each of 64 requests, states in a larger pool, some rows padding.
        {"name": "recurrence_step_64", "op": "recurrence_step", "dtype": "bf16", "batch": 64,
         "channels": 2048, "input_gate": True, "pool": 96},
        # A few rows at decoding time: latency.
        {"name": "norm_decode", "op": "norm", "dtype": "bf16", "rows": 16, "cols": 2048, "affine": True},
        # All the tokens of a training batch.
        {"name": "norm_train", "op": "norm", "dtype": "bf16", "rows": 16384, "cols": 4096, "affine": True},
        # Their gradient, with the reduction over rows for the weight and the bias.
        {"name": "norm_grad_train", "op": "norm_grad", "dtype": "bf16", "rows": 16384, "cols": 4096,
         "affine": True},
        # Sampling: the logits of a few requests, 20 alternatives, some rows restricted by a grammar.
        {"name": "logprob_decode", "op": "logprob", "dtype": "fp32", "rows": 7, "vocab": 50021, "top": 20},
        # Scoring a training batch over a large vocabulary.
        {"name": "logprob_score", "op": "logprob", "dtype": "bf16", "rows": 4096, "vocab": 128000, "top": 8},
        # The gradient of log probabilities and entropy, as a policy-gradient step takes it.
        {"name": "logprob_grad_train", "op": "logprob_grad", "dtype": "bf16", "rows": 4096, "vocab": 32000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a multiple of 64 mostly, else anything."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.4 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["recurrence", "recurrence", "recurrence_grad", "recurrence_grad", "recurrence_step",
                     "norm", "norm_grad", "logprob", "logprob", "logprob_grad"])
    dtype = rng.choice(["fp32", "bf16", "bf16", "fp16"])
    if op in ("recurrence", "recurrence_grad"):
        channels = _width(rng, 64, 4096)
        room = (120 << 20) // (channels * SIZE[dtype])
        length = min(_log(rng, 1, 65536), room)
        return {"op": op, "dtype": dtype, "batch": min(_log(rng, 1, 64), max(1, room // length)), "length": length,
                "channels": channels, "input_gate": rng.random() < 0.5, "packed": rng.random() < 0.5,
                "carried": rng.random() < 0.5}
    if op == "recurrence_step":
        batch = _log(rng, 1, 512)
        return {"op": op, "dtype": dtype, "batch": batch, "channels": _width(rng, 64, 4096),
                "input_gate": rng.random() < 0.5, "pool": batch + rng.randint(0, batch)}
    if op in ("norm", "norm_grad"):
        cols = _width(rng, 64, 16384)
        return {"op": op, "dtype": dtype, "rows": min(_log(rng, 1, 65536), (1 << 26) // cols), "cols": cols,
                "affine": rng.random() < 0.8}
    vocab = _log(rng, 1000, 200000)
    case = {"op": op, "dtype": dtype, "rows": min(_log(rng, 1, 8192), (120 << 20) // vocab), "vocab": vocab}
    if op == "logprob":
        case["top"] = rng.choice([0, 1, 5, 8, 20, 32])
    return case


def work(case):
    """Each input read once, each output written once; a handful of operations an element."""
    op, es = case["op"], SIZE[case["dtype"]]
    if op in ("recurrence", "recurrence_grad"):
        b, t, d = case["batch"], case["length"], case["channels"]
        gate = 1 if case["input_gate"] else 0
        state = 4 * b * d
        if op == "recurrence":
            n = (3 + gate) * b * t * d * es + state  # x, f(, i) in; h and the last state out
        else:
            n = (6 + 2 * gate) * b * t * d * es + state  # dh, x, f, h(, i) in; dx, df(, di), dh0 out
        if case["carried"]:
            n += state if op == "recurrence" else 2 * state  # h0 (and the last state's gradient)
        if case["packed"]:
            n += b * t
        return {"bytes": n, "flops": (12 if op == "recurrence" else 24) * b * t * d}
    if op == "recurrence_step":
        b, d = case["batch"], case["channels"]
        return {"bytes": b * d * ((3 + bool(case["input_gate"])) * es + 8) + 4 * b, "flops": 12 * b * d}
    if op in ("norm", "norm_grad"):
        n, d, w = case["rows"], case["cols"], (case["cols"] if case["affine"] else 0)
        if op == "norm":
            return {"bytes": 2 * n * d * es + 2 * w * es + 8 * n, "flops": 8 * n * d}
        return {"bytes": 3 * n * d * es + 3 * w * es + 8 * n, "flops": 14 * n * d}
    n, v = case["rows"], case["vocab"]
    if op == "logprob":
        return {"bytes": n * v * es + 16 * n + 8 * n * case["top"], "flops": 6 * n * v}
    return {"bytes": 2 * n * v * es + 20 * n, "flops": 8 * n * v}


# ----------------------------------------------------------------- inputs ------

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, mean=0.0, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).add_(mean).to(dtype)


def _recurrence_inputs(case, g):
    b, t, d, dtype = case["batch"], case["length"], case["channels"], DTYPES[case["dtype"]]
    k = 3 if case["input_gate"] else 2
    # One projection gives the input and the gates: x, f(, i) are slices of its rows.
    proj = torch.empty((b, t, k * d), device="cuda", dtype=dtype)
    proj[..., :d] = _normal(g, (b, t, d), dtype)
    proj[..., d:2 * d] = _normal(g, (b, t, d), dtype, 2.0, 1.5)  # memories of a few to some hundred steps
    if k == 3:
        proj[..., 2 * d:] = _normal(g, (b, t, d), dtype, 0.0, 1.5)
    s = {"case": case, "x": proj[..., :d], "f": proj[..., d:2 * d], "i": proj[..., 2 * d:] if k == 3 else None,
         "h0": None, "starts": None}
    if case["packed"]:  # several documents in one row, some hundred tokens each
        s["starts"] = (torch.rand((b, t), generator=g, device="cuda") < 1 / 400).to(torch.uint8)
    if case["carried"]:
        s["h0"] = _normal(g, (b, d), torch.float32)
    return s


def prepare(case, seed):
    g, op, dtype = _rng(seed), case["op"], DTYPES[case["dtype"]]
    if op in ("recurrence", "recurrence_grad"):
        s = _recurrence_inputs(case, g)
        if op == "recurrence_grad":
            b, t, d = s["x"].shape
            s["h"] = _recurrence(s["x"], s["f"], s["i"], s["h0"], s["starts"])[0]  # what the forward pass left
            s["dh"] = _normal(g, (b, t, d), dtype)
            s["dlast"] = _normal(g, (b, d), torch.float32) if case["carried"] else None
        return s
    if op == "recurrence_step":
        b, d, pool = case["batch"], case["channels"], case["pool"]
        k = 3 if case["input_gate"] else 2
        proj = _normal(g, (b, k * d), dtype)
        proj[:, d:2 * d] += 2.0
        slots = torch.randperm(pool, generator=g, device="cuda")[:b].to(torch.int32)
        slots[b - b // 8:] = -1  # the batch is padded to its size
        return {"case": case, "x": proj[:, :d], "f": proj[:, d:2 * d], "i": proj[:, 2 * d:] if k == 3 else None,
                "slots": slots, "live": torch.arange(b - b // 8, device="cuda"),
                "state": _normal(g, (pool, d), torch.float32)}
    if op in ("norm", "norm_grad"):
        n, d = case["rows"], case["cols"]
        x = _normal(g, (n, d), torch.float32)
        x = (x * (0.5 + torch.rand((n, 1), generator=g, device="cuda")) + 0.3).to(dtype)
        s = {"case": case, "x": x, "w": None, "b": None}
        if case["affine"]:
            s["w"] = _normal(g, (d,), dtype, 1.0, 0.2)
            s["b"] = _normal(g, (d,), dtype, 0.0, 0.2)
        if op == "norm_grad":
            s["dy"] = _normal(g, (n, d), dtype)
            _, s["mean"], s["rstd"] = _norm(x, s["w"], s["b"])
        return s
    n, v = case["rows"], case["vocab"]
    logits = _normal(g, (n, v), dtype, 0.0, 2.5)
    rows = torch.arange(n, device="cuda")
    targets = torch.randint(0, v, (n,), generator=g, device="cuda")
    best = torch.randint(0, v, (n,), generator=g, device="cuda")
    logits[rows, best] = (12.0 + 3.0 * torch.rand((n,), generator=g, device="cuda")).to(dtype)
    targets = torch.where(torch.rand((n,), generator=g, device="cuda") < 0.6, best, targets)
    if op == "logprob":
        logits[::5, v // 3:] = NEG  # every fifth row: a grammar allows part of the vocabulary
    else:
        targets[::16] = -1  # prompt tokens take no part in the loss
    s = {"case": case, "logits": logits, "targets": targets}
    if op == "logprob_grad":
        _, s["entropy"], s["lse"], _, _ = _logprob(logits, targets, 0)
        s["dlogprob"] = _normal(g, (n,), torch.float32) / n
        s["dentropy"] = _normal(g, (n,), torch.float32, 0.01, 0.001) / n
    return s


# ------------------------------------------------------------ plain forms ------

def _scan(a, b):
    """y_t = a_t y_{t-1} + b_t along dim 1 from y_{-1} = 0, in log2(T) doubling steps."""
    s, t = 1, b.shape[1]
    while s < t:
        b = torch.cat([b[:, :s], a[:, s:] * b[:, :-s] + b[:, s:]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _gates(f, i):
    a = torch.sigmoid(f.float())
    return a, torch.sigmoid(-f.float()) if i is None else torch.sigmoid(i.float())


def _recurrence(x, f, i, h0, starts):
    a, u = _gates(f, i)
    b = u * x.float()
    if starts is not None:
        a = a * (starts == 0).unsqueeze(-1)
    if h0 is not None:
        b[:, 0] += a[:, 0] * h0
    h = _scan(a, b)
    return h.to(x.dtype), h[:, -1].contiguous()


def _recurrence_grad(dh, x, f, i, h, h0, starts, dlast):
    a, u = _gates(f, i)
    keep = a if starts is None else a * (starts == 0).unsqueeze(-1)
    g = dh.float()
    if dlast is not None:
        g = torch.cat([g[:, :-1], (g[:, -1] + dlast).unsqueeze(1)], 1)
    back = torch.cat([torch.zeros_like(keep[:, :1]), keep[:, 1:].flip(1)], 1)
    g = _scan(back, g.flip(1)).flip(1)
    first = torch.zeros_like(g[:, 0]) if h0 is None else h0
    before = torch.cat([first.unsqueeze(1), h[:, :-1].float()], 1)
    if starts is not None:
        before = before * (starts == 0).unsqueeze(-1)
    x = x.float()
    dx = u * g
    da = a * torch.sigmoid(-f.float())
    if i is None:
        df, di = da * (before - x) * g, None
    else:
        df, di = da * before * g, (u * torch.sigmoid(-i.float()) * x * g).to(h.dtype)
    return dx.to(h.dtype), df.to(h.dtype), di, keep[:, 0] * g[:, 0]


def _step(x, f, i, state, slots, live):
    a, u = _gates(f, i)
    at = slots[live].long()
    new = a[live] * state[at] + u[live] * x[live].float()
    state[at] = new
    h = torch.zeros_like(x, memory_format=torch.contiguous_format)
    h[live] = new.to(x.dtype)
    return h, state


def _norm(x, w, b):
    v = x.float()
    mean = v.mean(1)
    c = v - mean.unsqueeze(1)
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    y = c * rstd.unsqueeze(1)
    if w is not None:
        y = y * w.float() + b.float()
    return y.to(x.dtype), mean, rstd


def _norm_grad(dy, x, mean, rstd, w):
    g = dy.float()
    n = (x.float() - mean.unsqueeze(1)) * rstd.unsqueeze(1)
    dw, db = (None, None) if w is None else ((g * n).sum(0).to(w.dtype), g.sum(0).to(w.dtype))
    if w is not None:
        g = g * w.float()
    dx = (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True)) * rstd.unsqueeze(1)
    return dx.to(x.dtype), dw, db


def _ordered(v):
    """int64 keys that order as (value, then the lower index first)."""
    bits = (v + 0.0).view(torch.int32).long()
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    return (bits << 32) | (0x7FFFFFFF - torch.arange(v.shape[1], device=v.device))


def _logprob(logits, targets, top):
    v = logits.float()
    m = v.max(1, keepdim=True).values
    d = v - m
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    log_s = torch.log(s)
    lse = (m + log_s).squeeze(1)
    entropy = log_s.squeeze(1) - (e * torch.where(e > 0, d, 0.0)).sum(1) / s.squeeze(1)
    at = targets.clamp(min=0).unsqueeze(1)
    logprob = torch.where(targets < 0, 0.0, (d.gather(1, at) - log_s).squeeze(1))
    if not top:
        return logprob, entropy, lse, None, None
    ids = 0x7FFFFFFF - (_ordered(v).topk(top, 1).values & 0x7FFFFFFF)
    return logprob, entropy, lse, d.gather(1, ids) - log_s, ids.to(torch.int32)


def _logprob_grad(logits, targets, lse, entropy, dlogprob, dentropy):
    lp = logits.float() - lse.unsqueeze(1)
    p = torch.exp(lp)
    one = torch.arange(logits.shape[1], device=lp.device) == targets.unsqueeze(1)
    weight = torch.where(targets < 0, 0.0, dlogprob).unsqueeze(1)
    d = weight * (one.float() - p)
    d -= dentropy.unsqueeze(1) * p * torch.where(p > 0, lp + entropy.unsqueeze(1), 0.0)
    return d.to(logits.dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(op, s)
    if op == "recurrence":
        return _recurrence(s["x"], s["f"], s["i"], s["h0"], s["starts"])
    if op == "recurrence_grad":
        return _recurrence_grad(s["dh"], s["x"], s["f"], s["i"], s["h"], s["h0"], s["starts"], s["dlast"])
    if op == "recurrence_step":
        return _step(s["x"], s["f"], s["i"], s["state"], s["slots"], s["live"])
    if op == "norm":
        return _norm(s["x"], s["w"], s["b"])
    if op == "norm_grad":
        return _norm_grad(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    if op == "logprob":
        return _logprob(s["logits"], s["targets"], s["case"]["top"])
    return _logprob_grad(s["logits"], s["targets"], s["lse"], s["entropy"], s["dlogprob"], s["dentropy"])


def _run_own(op, s):
    import stream_compaction_decoupled_gb300 as gb
    if op == "recurrence":
        return gb.recurrence(s["x"], s["f"], s["i"], h0=s["h0"], starts=s["starts"])
    if op == "recurrence_grad":
        return gb.recurrence_backward(s["dh"], s["x"], s["f"], s["h"], s["i"], h0=s["h0"], starts=s["starts"],
                                      dlast=s["dlast"])
    if op == "recurrence_step":
        return gb.recurrence_step(s["x"], s["f"], s["state"], s["i"], slots=s["slots"]), s["state"]
    if op == "norm":
        return gb.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
    if op == "norm_grad":
        return gb.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    if op == "logprob":
        return tuple(gb.token_logprobs(s["logits"], s["targets"], top=s["case"]["top"]))
    return gb.token_logprobs_backward(s["logits"], s["targets"], s["lse"], s["entropy"], s["dlogprob"],
                                      s["dentropy"])


# ------------------------------------------------- the definition, 64 bits ------

def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op == "recurrence_step":
        live, at = s["live"], s["slots"][s["live"]].long()
        a = 1 / (1 + torch.exp(-s["f"][live]))
        u = 1 - a if s["i"] is None else 1 / (1 + torch.exp(-s["i"][live]))
        s["state"][at] = a * s["state"][at] + u * s["x"][live]
        h = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
        h[live] = s["state"][at]
        return h, s["state"]
    if op in ("recurrence", "recurrence_grad"):
        x, f, i, starts = s["x"], s["f"], s["i"], s["starts"]
        b, t, d = x.shape
        a = 1 / (1 + torch.exp(-f))
        u = 1 - a if i is None else 1 / (1 + torch.exp(-i))
        keep = a.clone()
        if starts is not None:
            keep[starts != 0] = 0.0
        zero = torch.zeros((b, d), dtype=torch.float64, device="cuda")
        h0 = zero if s["h0"] is None else s["h0"]
        y = torch.empty((t, b, d), dtype=torch.float64, device="cuda")  # token by token
        if op == "recurrence":
            ux, state = u * x, h0
            for k in range(t):
                state = torch.addcmul(ux[:, k], keep[:, k], state, out=y[k])
            return y.transpose(0, 1), state
        carry = zero if s["dlast"] is None else s["dlast"]  # a_{t+1} g_{t+1}
        for k in range(t - 1, -1, -1):
            torch.add(s["dh"][:, k], carry, out=y[k])
            carry = keep[:, k] * y[k]
        g = y.transpose(0, 1)
        before = torch.cat([h0.unsqueeze(1), s["h"][:, :-1]], 1)
        if starts is not None:
            before[starts != 0] = 0.0
        if i is None:
            return u * g, a * (1 - a) * (before - x) * g, None, carry
        return u * g, a * (1 - a) * before * g, u * (1 - u) * x * g, carry
    if op == "norm":
        x = s["x"]
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        y = (x - mean[:, None]) * rstd[:, None]
        return y if s["w"] is None else torch.addcmul(s["b"], y, s["w"]), mean, rstd
    if op == "norm_grad":
        d = case["cols"]
        n = (s["x"] - s["mean"][:, None]) * s["rstd"][:, None]
        g = s["dy"] if s["w"] is None else s["dy"] * s["w"]
        along = torch.einsum("nd,nd->n", g, n) / d
        dx = s["rstd"][:, None] * (g - g.sum(1, keepdim=True) / d - n * along[:, None])
        if s["w"] is None:
            return dx, None, None
        return dx, torch.einsum("nd,nd->d", s["dy"], n), s["dy"].sum(0)
    v, targets = s["logits"], s["targets"]
    logp = v - torch.logsumexp(v, 1, keepdim=True)
    p = logp.exp()
    at = targets.clamp(min=0)[:, None]
    if op == "logprob":
        entropy = torch.special.entr(p).sum(1)
        logprob = logp.gather(1, at)[:, 0]
        logprob[targets < 0] = 0.0
        top = logp.topk(case["top"], 1).values if case["top"] else None
        return logprob, entropy, torch.logsumexp(v, 1), top, None
    w = s["dlogprob"].clone()
    w[targets < 0] = 0.0
    # dH/dv_j = -p_j (log p_j + H) = entr(p_j) - p_j H
    d = -w[:, None] * p + s["dentropy"][:, None] * (torch.special.entr(p) - p * s["entropy"][:, None])
    d.scatter_add_(1, at, w[:, None])
    return d
