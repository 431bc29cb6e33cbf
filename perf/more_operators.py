"""The elementwise recurrence, the delta rule's single token and the norm after a block: the cases they are measured at.

Operators next to the chunked delta rule and the layer operators, each as a user's program calls it:

* the gated linear recurrence (per channel: h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t with
  a_t = exp(-c softplus(decay) sigmoid(r_t)), times SiLU of a gate), over prompts and packed prompts, with its gradient,
  and for one token a sequence with the cached state;
* one token of every running request through the gated delta rule, whose states the chunked prefill leaves behind;
* the norm of a block's output times SiLU of its gate, scaled and added to the residual stream, with the norm before the
  next block, and their gradients; without the stream it is the gated norm of each head's output.

``own`` selects between the plain form (elementary torch operations in 32 bits) and this package's kernels.
"""
import math

import torch

own = False  # set by whoever measures: False the plain forms, True the package's operators

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_C = 8.0  # the recurrence's decay scale


def _lengths(case):
    return [int(v) for v in case["lengths"].split(",")] if case.get("lengths") else None


def listed():
    return [
        # The smallest call: one new token for each of 64 running requests, whose states sit in a cache of 96.
        {"name": "linear_step_64", "op": "linear_step", "rows": 64, "slots": 96, "D": 4096, "z": False, "dtype": "bf16"},
        # The same for a larger batch in 32 bits, an odd width, with the output gate.
        {"name": "linear_step_f32", "op": "linear_step", "rows": 200, "slots": 211, "D": 2051, "z": True, "dtype": "f32"},
        # A long prompt of one request, and the state that decoding starts from.
        {"name": "linear_prompt_16384", "op": "linear", "B": 1, "T": 16384, "D": 4096, "z": False, "dtype": "bf16"},
        # Prompts of uneven lengths packed together (one of a single token), each continuing from a cached state, gated, odd width.
        {"name": "linear_packed_f32", "op": "linear", "B": 1, "T": 5003, "D": 1031, "z": True, "dtype": "f32", "lengths": "1021,1,2642,1339"},
        # A training step of two sequences: output and all gradients.
        {"name": "linear_train_2x4096", "op": "linear_train", "B": 2, "T": 4096, "D": 4096, "z": False, "dtype": "bf16"},
        # A training step over packed documents, gated, continuing from states and with a gradient of the final ones.
        {"name": "linear_train_packed", "op": "linear_train", "B": 1, "T": 8192, "D": 2048, "z": True, "dtype": "bf16",
         "lengths": "2500,1,2871,717,2103"},
        # One new token for each of 64 running requests: 16 query/key heads and 32 value heads of 128 channels.
        {"name": "delta_step_64", "op": "delta_step", "rows": 64, "slots": 72, "Hq": 16, "Hv": 32, "K": 128, "V": 128, "dtype": "bf16"},
        # One running request: a call's latency.
        {"name": "delta_step_1", "op": "delta_step", "rows": 1, "slots": 4, "Hq": 8, "Hv": 16, "K": 128, "V": 128, "dtype": "bf16"},
        # The other head sizes in 32 bits, an odd batch.
        {"name": "delta_step_f32", "op": "delta_step", "rows": 13, "slots": 17, "Hq": 4, "Hv": 8, "K": 64, "V": 192, "dtype": "f32"},
        # Between two blocks over a batch of prompts: the norm after one, the stream, the norm before the next.
        {"name": "block_norm_prompt", "op": "norm", "M": 16384, "D": 4096, "gate": False, "residual": True, "next": True, "dtype": "bf16"},
        # A training step of the same with the block's gate.
        {"name": "block_norm_train", "op": "norm_train", "M": 8192, "D": 4096, "gate": True, "residual": True, "next": True, "dtype": "bf16"},
        # A training step of the gated norm of each head's output: 32 heads of 128 channels of 8192 tokens.
        {"name": "head_norm_train", "op": "norm_train", "M": 262144, "D": 128, "gate": True, "residual": False, "next": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def _cut(rng, total, parts):
    cuts = sorted(rng.randint(0, total) for _ in range(parts - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_train", "linear_train", "linear_step", "delta_step", "norm", "norm_train"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op == "linear_step":
        rows = _log(rng, 1, 256)
        return {"op": op, "rows": rows, "slots": rows + rng.randint(0, 64), "D": _log(rng, 64, 8192), "z": rng.random() < 0.5, "dtype": dt}
    if op in ("linear", "linear_train"):
        d = _log(rng, 64, 4096)
        t = _log(rng, 1, min(16384, (1 << (25 if op == "linear" else 24)) // d))
        packed = rng.random() < 0.5
        b = 1 if packed else rng.choice([1, 1, 2, 3])
        t = max(1, t // b)
        c = {"op": op, "B": b, "T": t, "D": d, "z": rng.random() < 0.5, "dtype": dt}
        if packed:
            c["lengths"] = _cut(rng, t, rng.randint(1, 8))
        return c
    if op == "delta_step":
        hq, k, v = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128, 128, 192]), rng.choice([64, 128, 128, 192, 256])
        hv = hq * rng.choice([1, 2, 4])
        rows = _log(rng, 1, max(1, min(128, (1 << 24) // (hv * k * v))))
        return {"op": op, "rows": rows, "slots": rows + rng.randint(0, 8), "Hq": hq, "Hv": hv, "K": k, "V": v, "dtype": dt}
    d = _log(rng, 64, 8192)
    m = _log(rng, 1, min(65536, (1 << (25 if op == "norm" else 24)) // d))
    gate, residual, after = (rng.random() < 0.6 for _ in range(3))
    return {"op": op, "M": m, "D": d, "gate": gate, "residual": residual, "next": after, "dtype": dt}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    def rand(*s):
        return torch.rand(*s, device="cuda", generator=gen)

    op, dt = case["op"], _DT[case["dtype"]]
    s = {"op": op}
    lens = _lengths(case)
    if lens is not None:
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if "slots" in case:
        s["slots"] = torch.randperm(case["slots"], device="cuda", generator=gen)[: case["rows"]].to(torch.int32)
    if op in ("linear", "linear_train", "linear_step"):
        d = case["D"]
        head = (case["rows"],) if op == "linear_step" else (case["B"], case["T"])
        for k in ("x", "i", "r"):
            s[k] = randn(*head, d).to(dt)
        s["z"] = randn(*head, d).to(dt) if case["z"] else None
        # an open gate's decays lie between 0.9 and 0.999
        s["decay"] = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * rand(d)) / _C))
        if op == "linear_step":
            s["state"] = randn(case["slots"], d)
        else:
            s["h0"] = randn(len(lens), d) if lens is not None else None
        if op == "linear_train":
            s["dy"] = randn(*head, d).to(dt)
            s["dht"] = randn(len(lens), d) if lens is not None else None
            s["leaves"] = [s[k].requires_grad_() for k in ("x", "i", "r", "decay", "z", "h0") if s[k] is not None]
    elif op == "delta_step":
        rows, hq, hv, k, v = (case[n] for n in ("rows", "Hq", "Hv", "K", "V"))
        q, key = randn(rows, hq, k), randn(rows, hq, k)
        s["q"] = (q / torch.sqrt((q * q).sum(-1, keepdim=True))).to(dt)
        s["k"] = (key / torch.sqrt((key * key).sum(-1, keepdim=True))).to(dt)
        s["v"] = randn(rows, hv, v).to(dt)
        s["g"] = -torch.log1p(torch.exp(-(4.0 + 1.5 * randn(rows, hv))))
        s["beta"] = 1.0 / (1.0 + torch.exp(-randn(rows, hv)))
        s["state"] = 0.1 * randn(case["slots"], hv, k, v)
    else:
        m, d = case["M"], case["D"]
        s["x"] = (2.0 * randn(m, d)).to(dt)
        s["weight"] = 1.0 + 0.1 * randn(d)
        s["gate"] = randn(m, d).to(dt) if case["gate"] else None
        s["residual"] = (2.0 * randn(m, d)).to(dt) if case["residual"] else None
        s["next"] = 1.0 + 0.1 * randn(d) if case["next"] else None
        s["scale"] = 0.5 if case["residual"] else 1.0
        if op == "norm_train":
            s["dr"] = randn(m, d).to(dt)
            s["dy"] = randn(m, d).to(dt) if case["next"] else None
            s["leaves"] = [s[k].requires_grad_() for k in ("x", "weight", "gate", "residual", "next") if s[k] is not None]
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------------


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return v.clamp_min(0.0) + torch.log1p(torch.exp(-v.abs()))


def _dsilu(v):
    g = _sigmoid(v)
    return g * (1.0 + v * (1.0 - g))


def _f(t):
    return None if t is None else t.detach().float()


def _prefix(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1, by doubling the reach."""
    reach = 1
    while reach < b.shape[1]:
        b = torch.cat([b[:, :reach], b[:, reach:] + a[:, reach:] * b[:, :-reach]], 1)
        a = torch.cat([a[:, :reach], a[:, reach:] * a[:, :-reach]], 1)
        reach *= 2
    return b


def _gates(s):
    """The step's parts: x, sigmoid(i), sigmoid(r), log a, a, sqrt(1 - a^2)."""
    x, si, sr = _f(s["x"]), _sigmoid(_f(s["i"])), _sigmoid(_f(s["r"]))
    log_a = -_C * _softplus(_f(s["decay"])) * sr
    return x, si, sr, log_a, torch.exp(log_a), torch.sqrt(-torch.expm1(2.0 * log_a))


def _starts(s):
    """Which token opens a sequence [B, T, 1], and which sequence a token is of."""
    b, t = s["x"].shape[:2]
    at = torch.arange(t, device=s["x"].device)
    if s.get("cu") is None:
        return (at == 0)[None, :, None].expand(b, t, 1), torch.arange(b, device=at.device)[:, None].expand(b, t)
    seq = torch.searchsorted(s["cu"], at.to(torch.int32), right=True) - 1
    return (s["cu"][seq] == at)[None, :, None], seq[None]


def _plain_linear(s):
    x, si, sr, log_a, a, m = _gates(s)
    first, seq = _starts(s)
    bx = m * si * x
    if s["h0"] is not None:
        bx = torch.where(first, bx + a * _f(s["h0"])[seq], bx)
    cut = torch.where(first, 0.0, a)
    h = _prefix(cut, bx)
    if s.get("cu") is None:
        final = h[:, -1].clone()
    else:
        empty = (s["cu"][1:] == s["cu"][:-1])[:, None]
        final = torch.where(empty, _f(s["h0"]), h[0, (s["cu"][1:].long() - 1).clamp_min(0)])
    z = _f(s["z"])
    y = (h if z is None else h * z * _sigmoid(z)).to(s["x"].dtype)
    if s["op"] == "linear":
        return y, final
    dy = _f(s["dy"])
    din = dy if z is None else dy * z * _sigmoid(z)
    if s["dht"] is not None:
        ends = s["cu"][1:].long() - 1
        keep = s["cu"][1:] > s["cu"][:-1]
        din = din.clone()
        din[0, ends[keep]] += s["dht"][keep]
    nxt = torch.cat([cut[:, 1:], torch.zeros_like(cut[:, :1])], 1)
    e = _prefix(nxt.flip(1), din.flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    before = torch.where(first, 0.0 if s["h0"] is None else _f(s["h0"])[seq], before)
    u = si * x
    du = e * m
    dlog = e * a * before - e * u * a * a / m
    dt = s["x"].dtype
    out = [y, du * si, du * x * si * (1.0 - si), dlog * log_a * (1.0 - sr)]
    out = [v.to(dt) for v in out]
    decay = _f(s["decay"])
    out.append((-_C * _sigmoid(decay) * (dlog * sr).sum((0, 1), dtype=torch.float64)).float())
    if z is not None:
        out.append((dy * h * _dsilu(z)).to(dt))
    if s["h0"] is not None:
        dh0 = s["dht"].clone()
        heads = s["cu"][:-1].long()
        dh0[keep] = (a * e)[0, heads[keep]]
        out.append(dh0)
    return tuple(out)


def _plain_linear_step(s):
    slots = s["slots"].long()
    x, si, _, _, a, m = _gates(s)
    h = a * s["state"][slots] + m * si * x
    s["state"][slots] = h
    z = _f(s["z"])
    return (h if z is None else h * z * _sigmoid(z)).to(s["x"].dtype), s["state"]


def _plain_delta_step(s):
    slots = s["slots"].long()
    per = s["v"].shape[1] // s["q"].shape[1]
    q, k = (_f(s[n]).repeat_interleave(per, 1) for n in ("q", "k"))
    old = s["state"][slots] * torch.exp(s["g"])[..., None, None]
    delta = s["beta"][..., None] * (_f(s["v"]) - (old * k[..., None]).sum(-2))
    new = old + k[..., None] * delta[..., None, :]
    s["state"][slots] = new
    o = (new * q[..., None]).sum(-2) * s["q"].shape[-1] ** -0.5
    return o.to(s["q"].dtype), s["state"]


def _plain_norm(s):
    x, w, gate, res, w2, scale = (*(_f(s[k]) for k in ("x", "weight", "gate", "residual", "next")), s["scale"])
    dt = s["x"].dtype
    rx = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    hat = x * rx
    g = 1.0 if gate is None else gate * _sigmoid(gate)
    r = scale * hat * w * g
    if res is not None:
        r = r + res
    out = [r.to(dt)]
    if w2 is not None:
        rr = torch.rsqrt((r * r).mean(-1, keepdim=True) + _EPS)
        out.insert(0, (r * rr * w2).to(dt))
    if s["op"] == "norm":
        return tuple(out)
    dr = _f(s["dr"])
    if w2 is not None:
        dy = _f(s["dy"])
        dhat = dy * w2
        dr = dr + rr * (dhat - r * rr * (dhat * r * rr).mean(-1, keepdim=True))
        dw2 = (dy * r * rr).sum(0, dtype=torch.float64).float()
    du = scale * dr
    dw = (du * hat * g).sum(0, dtype=torch.float64).float()
    gx = du * w * g
    out += [(rx * (gx - hat * (gx * hat).mean(-1, keepdim=True))).to(dt), dw]
    if gate is not None:
        out.append((du * hat * w * _dsilu(gate)).to(dt))
    if res is not None:
        out.append(dr.to(dt))
    if w2 is not None:
        out.append(dw2)
    return tuple(out)


_PLAIN = {"linear": _plain_linear, "linear_train": _plain_linear, "linear_step": _plain_linear_step, "delta_step": _plain_delta_step,
          "norm": _plain_norm, "norm_train": _plain_norm}


# ---- the package's operators ----------------------------------------------------------------------------------------


def _own(s):
    import gated_deltanet_chunked_delta_gb300 as gdr
    op = s["op"]
    if op in ("linear", "linear_train"):
        y, final = gdr.gated_linear_scan(s["x"], s["i"], s["r"], s["decay"], s["z"], decay_scale=_C, initial_state=s["h0"],
                                         output_final_state=op == "linear" or s["dht"] is not None, cu_seqlens=s.get("cu"))
        if op == "linear":
            return y, final
        outs, grads = ([y], [s["dy"]]) if s["dht"] is None else ([y, final], [s["dy"], s["dht"]])
        return (y.detach(), *torch.autograd.grad(outs, s["leaves"], grads))
    if op == "linear_step":
        return gdr.gated_linear_step(s["x"], s["i"], s["r"], s["decay"], s["state"], s["z"], decay_scale=_C, slots=s["slots"]), s["state"]
    if op == "delta_step":
        return gdr.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"]), s["state"]
    y, r = gdr.gated_residual_rms_norm(s["x"], s["weight"], s["gate"], s["residual"], s["next"], scale=s["scale"], eps=_EPS)
    outs = [r] if y is None else [y, r]
    if op == "norm":
        return tuple(outs)
    grads = [s["dr"]] if y is None else [s["dy"], s["dr"]]
    return (*(o.detach() for o in outs), *torch.autograd.grad(outs, s["leaves"], grads))


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------------------------------


def work(case):
    op, e = case["op"], 4 if case["dtype"] == "f32" else 2
    if op in ("linear", "linear_train"):
        n, d, z = case["B"] * case["T"] * case["D"], case["D"], int(case["z"])
        states = 4 * d * len(_lengths(case)) if case.get("lengths") else 0
        if op == "linear":  # x, both gates, y (and the output gate); states in and out
            return {"bytes": e * n * (4 + z) + 4 * d + (2 * states or 4 * d * case["B"]), "flops": n * (24 + 5 * z)}
        # forward x, gates, y; backward x, gates, dy, dx and the gates' gradients (the output gate twice and its gradient)
        return {"bytes": e * n * (11 + 3 * z) + 8 * d + 5 * states, "flops": n * (75 + 15 * z)}
    if op == "linear_step":
        n, z = case["rows"] * case["D"], int(case["z"])
        return {"bytes": n * (e * (4 + z) + 8) + 4 * case["D"], "flops": n * (24 + 5 * z)}
    if op == "delta_step":
        r, hq, hv, k, v = (case[n] for n in ("rows", "Hq", "Hv", "K", "V"))
        return {"bytes": r * (8 * hv * k * v + e * (2 * hq * k + 2 * hv * v) + 8 * hv), "flops": r * hv * 7 * k * v}
    n, d = case["M"] * case["D"], case["D"]
    gate, res, after = (int(case[k]) for k in ("gate", "residual", "next"))
    if op == "norm":
        return {"bytes": n * e * (2 + gate + res + after) + 4 * d * (1 + after), "flops": n * (5 + 6 * gate + 2 * res + 4 * after)}
    # forward x, gate, stream, r, y; backward x, gate, the gradients of r and y, those of x and gate; with a next norm the
    # stream again (for r) and its gradient (without one that is the gradient of r itself)
    return {"bytes": n * e * (5 + 3 * gate + res + 2 * after + 2 * res * after) + 12 * d * (1 + after),
            "flops": n * (22 + 20 * gate + 4 * res + 18 * after)}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------------


def _exact_linear(case, s):
    """Token by token, each sequence on its own; for a training step backwards again."""
    v = {k: t.detach().double() for k, t in s.items() if torch.is_tensor(t) and t.is_floating_point()}
    lens = _lengths(case)
    spans = [(b, 0, case["T"]) for b in range(case["B"])]
    if lens is not None:
        spans, at = [], 0
        for n in lens:
            spans.append((0, at, n))
            at += n
    si, sr = torch.sigmoid(v["i"]), torch.sigmoid(v["r"])
    soft = torch.logaddexp(v["decay"], torch.zeros_like(v["decay"]))
    log_a = -_C * soft * sr
    a = log_a.exp()
    m = (-torch.expm1(2 * log_a)).sqrt()
    add = m * si * v["x"]
    h, finals = torch.empty_like(add), []
    before = torch.empty_like(add)
    for i, (b, at, n) in enumerate(spans):
        now = v["h0"][i] if "h0" in v else torch.zeros_like(v["decay"])
        for t in range(at, at + n):
            before[b, t] = now
            now = a[b, t] * now + add[b, t]
            h[b, t] = now
        finals.append(now)
    sz = torch.sigmoid(v["z"]) if "z" in v else None
    y = h if sz is None else h * v["z"] * sz
    if case["op"] == "linear":
        return y, torch.stack(finals)
    din = v["dy"] if sz is None else v["dy"] * v["z"] * sz
    e, dh0 = torch.empty_like(add), []
    for i, (b, at, n) in enumerate(spans):
        now = v["dht"][i] if "dht" in v else torch.zeros_like(v["decay"])
        for t in range(at + n - 1, at - 1, -1):
            now = now + din[b, t]
            e[b, t] = now
            now = now * a[b, t]
        dh0.append(now)
    dlog = e * (before * a - si * v["x"] * a * a / m)
    out = [y, e * m * si, e * m * v["x"] * si * (1 - si), dlog * -_C * soft * sr * (1 - sr),
           (dlog * -_C * sr).sum((0, 1)) * torch.sigmoid(v["decay"])]
    if sz is not None:
        out.append(v["dy"] * h * (sz + v["z"] * sz * (1 - sz)))
    if "h0" in v:
        out.append(torch.stack(dh0))
    return tuple(out)


def _exact_linear_step(s):
    v = {k: t.double() for k, t in s.items() if torch.is_tensor(t) and t.is_floating_point()}
    state, ys = v["state"].clone(), []
    for row, slot in enumerate(s["slots"].tolist()):
        log_a = -_C * torch.logaddexp(v["decay"], torch.zeros_like(v["decay"])) * torch.sigmoid(v["r"][row])
        now = log_a.exp() * state[slot] + (-torch.expm1(2 * log_a)).sqrt() * torch.sigmoid(v["i"][row]) * v["x"][row]
        state[slot] = now
        ys.append(now if s["z"] is None else now * v["z"][row] * torch.sigmoid(v["z"][row]))
    return torch.stack(ys), state


def _exact_delta_step(s):
    """S <- e^g (I - beta k k^T) S + beta k v^T, o = K^-1/2 S^T q, head by head."""
    v = {k: t.double() for k, t in s.items() if torch.is_tensor(t) and t.is_floating_point()}
    state, o = v["state"].clone(), torch.empty_like(v["v"])
    hv, width = v["v"].shape[1], v["q"].shape[-1]
    eye = torch.eye(width, dtype=torch.float64, device=o.device)
    for h in range(hv):
        at = h // (hv // v["q"].shape[1])
        key, query = v["k"][:, at], v["q"][:, at]
        beta = v["beta"][:, h, None, None]
        keep = (eye - beta * key[:, :, None] * key[:, None, :]) * v["g"][:, h, None, None].exp()
        new = keep @ state[s["slots"].long(), h] + beta * key[:, :, None] * v["v"][:, h, None, :]
        state[s["slots"].long(), h] = new
        o[:, h] = (query[:, None, :] @ new)[:, 0] / width ** 0.5
    return o, state


def _exact_norm(s):
    v = {k: t.detach().double() for k, t in s.items() if torch.is_tensor(t) and t.is_floating_point()}
    x, w, d = v["x"], v["weight"], s["x"].shape[-1]
    rx = 1.0 / torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + _EPS)
    sg = torch.sigmoid(v["gate"]) if "gate" in v else None
    gain = w if sg is None else w * v["gate"] * sg
    r = s["scale"] * x * rx * gain + (v["residual"] if "residual" in v else 0.0)
    out = [r]
    if "next" in v:
        rr = 1.0 / torch.sqrt((r ** 2).sum(-1, keepdim=True) / d + _EPS)
        out = [r * rr * v["next"], r]
    if s["op"] == "norm":
        return tuple(out)
    dr = v["dr"]
    if "next" in v:
        dr = dr + rr * v["dy"] * v["next"] - r * rr ** 3 * (v["dy"] * v["next"] * r).sum(-1, keepdim=True) / d
    back = s["scale"] * dr * gain
    out.append(rx * back - x * rx ** 3 * (back * x).sum(-1, keepdim=True) / d)
    out.append((s["scale"] * dr * x * rx * gain / w).sum(0))
    if sg is not None:
        out.append(s["scale"] * dr * x * rx * w * (sg + v["gate"] * sg * (1 - sg)))
    if "residual" in v:
        out.append(dr)
    if "next" in v:
        out.append((v["dy"] * r * rr).sum(0))
    return tuple(out)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "linear_train"):
        return _exact_linear(case, s)
    if op == "linear_step":
        return _exact_linear_step(s)
    if op == "delta_step":
        return _exact_delta_step(s)
    return _exact_norm(s)
