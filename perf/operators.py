"""The operators of a recurrent token mixer's layer, next to the gated delta rule: the cases they are measured at.

Four operators, each as a user's program calls it:

* the short causal convolution along the tokens (depthwise, 2 to 4 taps, SiLU), over packed sequences with its
  gradient, and for one token a sequence with the cached last inputs;
* the selective state space scan (per channel: h_t = exp(dt_t A) h_{t-1} + dt_t B_t x_t, y_t = C_t h_t + D x_t,
  times SiLU of a gate), over prompts, with its gradient, and for one token a sequence with the cached state;
* the root-mean-square norm of a residual stream with the residual's addition, written in 8 bits with a scale for
  each 128 channels (serving) or in the input's type with its gradient (training);
* the product of such 8-bit activations with weights held in 8 bits, one scale for each 128 x 128 block.

``own`` selects between the plain form (elementary torch operations in 32 bits) and this package's kernels.
"""
import math

import torch

own = False  # set by whoever measures: False the plain forms, True the package's operators

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_E4M3 = torch.float8_e4m3fn
_FLOOR = 1e-30  # least absolute maximum of a block of 8-bit values
_EPS = 1e-6


def _lengths(case):
    return [int(v) for v in case["lengths"].split(",")] if case.get("lengths") else None


def listed():
    return [
        # The smallest call: one new token for each of 64 running requests, whose last three inputs sit in a cache of 96.
        {"name": "conv_step_64", "op": "conv_step", "rows": 64, "slots": 96, "D": 8192, "W": 4, "dtype": "bf16"},
        # A training step over packed documents of uneven lengths (one of a single token): output and all gradients.
        {"name": "conv_train_packed", "op": "conv", "D": 4096, "W": 4, "dtype": "bf16", "lengths": "2500,1,2871,717,2103"},
        # A long prompt of one request: 32 heads of 128 channels, the gate, and the state that decoding starts from.
        {"name": "scan_prompt_8192", "op": "scan", "B": 1, "T": 8192, "D": 4096, "N": 16, "G": 1, "dtype": "bf16"},
        # A training step of two sequences: output and all gradients.
        {"name": "scan_train_2x2048", "op": "scan_train", "B": 2, "T": 2048, "D": 4096, "N": 16, "G": 1, "dtype": "bf16"},
        # Prompts of uneven lengths packed together, each continuing from a cached state, in 32 bits, odd width.
        {"name": "scan_packed_f32", "op": "scan", "B": 1, "T": 3001, "D": 1031, "N": 16, "G": 1, "dtype": "f32",
         "lengths": "1021,1,640,1339"},
        # One new token for each of 128 running requests.
        {"name": "scan_step_128", "op": "scan_step", "rows": 128, "slots": 160, "D": 4096, "N": 16, "G": 1, "dtype": "bf16"},
        # The norm before a projection, over a batch of prompts.
        {"name": "norm_fp8_prompt", "op": "norm_fp8", "M": 16384, "D": 4096, "dtype": "bf16"},
        # The same for one new token of 32 requests: a call's latency.
        {"name": "norm_fp8_token", "op": "norm_fp8", "M": 32, "D": 2048, "dtype": "bf16"},
        # A training step's norm: output, residual stream and gradients.
        {"name": "norm_train", "op": "norm_train", "M": 8192, "D": 4096, "dtype": "bf16"},
        # The input projection over a batch of prompts: the largest call.
        {"name": "matmul_prompt", "op": "matmul", "M": 8192, "N": 8192, "K": 4096},
        # The same projection for one new token of 16 requests: the weights have to be read.
        {"name": "matmul_token_16", "op": "matmul", "M": 16, "N": 8192, "K": 4096},
        # A ragged middle: a batch and widths that no tile divides, a last block of K that is short.
        {"name": "matmul_ragged", "op": "matmul", "M": 1237, "N": 5000, "K": 2064},
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def _cut(rng, total, parts):
    cuts = sorted(rng.randint(0, total) for _ in range(parts - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    op = rng.choice(["conv_step", "conv", "scan", "scan_train", "scan_step", "norm_fp8", "norm_train", "matmul", "matmul"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv_step":
        rows = _log(rng, 1, 256)
        return {"op": op, "rows": rows, "slots": rows + rng.randint(0, 64), "D": _log(rng, 64, 8192), "W": rng.choice([2, 3, 4]), "dtype": dt}
    if op == "conv":
        d = _log(rng, 64, 8192)
        t = _log(rng, 1, min(16384, (1 << 25) // d))
        return {"op": op, "D": d, "W": rng.choice([2, 3, 4]), "dtype": dt, "lengths": _cut(rng, t, rng.randint(1, 8))}
    if op == "scan":
        n = rng.choice([8, 16, 16, 32])
        g = rng.choice([1, 1, 2, 4])
        d = g * max(1, _log(rng, 64, 4096) // g)
        t = _log(rng, 1, min(16384, (1 << 29) // (d * n)))
        packed = rng.random() < 0.5
        b = 1 if packed else rng.choice([1, 1, 2, 3])
        t = max(1, t // b)
        c = {"op": op, "B": b, "T": t, "D": d, "N": n, "G": g, "dtype": dt}
        if packed:
            c["lengths"] = _cut(rng, t, rng.randint(1, 8))
        return c
    if op == "scan_train":
        d = _log(rng, 64, 4096)
        return {"op": op, "B": rng.choice([1, 2]), "T": _log(rng, 1, min(4096, (1 << 23) // d)), "D": d, "N": 16, "G": 1, "dtype": dt}
    if op == "scan_step":
        rows = _log(rng, 1, 256)
        g = rng.choice([1, 1, 2])
        return {"op": op, "rows": rows, "slots": rows + rng.randint(0, 64), "D": g * _log(rng, 32, 2048), "N": rng.choice([8, 16, 32]), "G": g, "dtype": dt}
    if op in ("norm_fp8", "norm_train"):
        d = _log(rng, 128, 8192)
        return {"op": op, "M": _log(rng, 1, min(16384, (1 << 26) // d)), "D": d, "dtype": dt}
    return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 8192), "K": 16 * rng.choice([_log(rng, 8, 191), _log(rng, 193, 256)])}


def _quantise(x, rows):
    """x [R, K] in 32 bits as 8-bit values and their scales, one for each `rows` x 128 block."""
    r, k = x.shape
    nr, nk = -(-r // rows), -(-k // 128)
    big = x.new_zeros(nr * rows, nk * 128)
    big[:r, :k] = x
    top = big.abs().view(nr, rows, nk, 128).amax(dim=(1, 3)).clamp_min(_FLOOR)
    scale = top / 448.0
    spread = scale.repeat_interleave(rows, 0)[:r].repeat_interleave(128, 1)[:, :k]
    return (x / spread).clamp(-448.0, 448.0).to(_E4M3), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    op, dt = case["op"], _DT[case.get("dtype", "bf16")]
    s = {"op": op}
    lens = _lengths(case)
    if lens is not None:
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if op in ("conv", "conv_step"):
        d, w = case["D"], case["W"]
        s["weight"] = randn(d, w) * w ** -0.5
        s["bias"] = randn(d) * 0.1
        if op == "conv":
            t = sum(lens)
            s["x"], s["dy"] = randn(1, t, d).to(dt), randn(1, t, d).to(dt)
            s["leaves"] = [s["x"].requires_grad_(), s["weight"].requires_grad_(), s["bias"].requires_grad_()]
        else:
            s["x"] = randn(case["rows"], d).to(dt)
            s["state"] = randn(case["slots"], w - 1, d).to(dt)
            s["slots"] = torch.randperm(case["slots"], device="cuda", generator=gen)[: case["rows"]].to(torch.int32)
    elif op in ("scan", "scan_train", "scan_step"):
        d, n, g = case["D"], case["N"], case["G"]
        head = (case["rows"],) if op == "scan_step" else (case["B"], case["T"])
        s["x"], s["z"] = randn(*head, d).to(dt), randn(*head, d).to(dt)
        s["dt"] = (0.5 * randn(*head, d)).to(dt)
        s["B"], s["C"] = randn(*head, g, n).to(dt), randn(*head, g, n).to(dt)
        s["A"] = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32).repeat(d, 1) * torch.exp(0.2 * randn(d, n))
        s["D"] = 1.0 + 0.1 * randn(d)
        # steps between 1e-3 and 1e-1, spread over their logarithm, through the inverse of softplus
        step = torch.exp(torch.rand(d, device="cuda", generator=gen) * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        if op == "scan_step":
            s["state"] = randn(case["slots"], d, n)
            s["slots"] = torch.randperm(case["slots"], device="cuda", generator=gen)[: case["rows"]].to(torch.int32)
        elif op == "scan":
            s["h0"] = randn(len(lens) if lens is not None else case["B"], d, n) if lens is not None else None
        else:
            s["dy"] = randn(*head, d).to(dt)
            s["leaves"] = [s[k].requires_grad_() for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")]
    elif op in ("norm_fp8", "norm_train"):
        m, d = case["M"], case["D"]
        s["x"], s["residual"] = randn(m, d).to(dt), (2.0 * randn(m, d)).to(dt)
        s["weight"] = 1.0 + 0.1 * randn(d)
        if op == "norm_train":
            s["dy"], s["dres"] = randn(m, d).to(dt), randn(m, d).to(dt)
            s["leaves"] = [s[k].requires_grad_() for k in ("x", "weight", "residual")]
    else:
        m, n, k = case["M"], case["N"], case["K"]
        s["a"], scale = _quantise(randn(m, k), 1)
        s["a_scales"] = scale.t().contiguous()
        s["b"], s["b_scales"] = _quantise(randn(n, k) * k ** -0.5, 128)
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------------


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _dsilu(v):
    g = 1.0 / (1.0 + torch.exp(-v))
    return g * (1.0 + v * (1.0 - g))


def _softplus(v):
    return v.clamp_min(0.0) + torch.log1p(torch.exp(-v.abs()))


def _plain_conv(s):
    """y, dx, dweight, dbias of the convolution over the packed sequences, which start from zeros."""
    x, w, b, dy = s["x"].detach()[0].float(), s["weight"].detach(), s["bias"].detach(), s["dy"][0].float()
    t, taps = x.shape[0], w.shape[1]
    at = torch.arange(t, device=x.device)
    seq = torch.searchsorted(s["cu"], at.to(torch.int32), right=True) - 1
    first, last = s["cu"][seq].long(), s["cu"][seq + 1].long()
    back = torch.arange(taps - 1, -1, -1, device=x.device)  # tap j reads the input taps - 1 - j tokens back
    src = at[:, None] - back
    seen = torch.where((src >= first[:, None])[..., None], x[src.clamp_min(0)], 0.0)  # [T, taps, D]
    pre = (seen * w.t()).sum(1) + b
    dp = dy * _dsilu(pre)
    dst = at[:, None] + back
    dx = (torch.where((dst < last[:, None])[..., None], dp[dst.clamp_max(t - 1)], 0.0) * w.t()).sum(1)
    dw = (dp[:, None] * seen).sum(0).t().contiguous()
    dt = s["x"].dtype
    return _silu(pre).to(dt)[None], dx.to(dt)[None], dw, dp.sum(0)


def _plain_conv_step(s):
    slots = s["slots"].long()
    x = s["x"]
    seen = torch.cat([s["state"][slots], x[:, None]], 1)
    y = _silu((seen.float() * s["weight"].t()).sum(1) + s["bias"])
    s["state"][slots] = seen[:, 1:]
    return y.to(x.dtype), s["state"]


def _prefix(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1, by doubling the reach."""
    reach = 1
    while reach < b.shape[1]:
        b = torch.cat([b[:, :reach], b[:, reach:] + a[:, reach:] * b[:, :-reach]], 1)
        a = torch.cat([a[:, :reach], a[:, reach:] * a[:, :-reach]], 1)
        reach *= 2
    return b


def _per_channel(v, d):
    return v.repeat_interleave(d // v.shape[-2], -2)


def _starts(s, b, t):
    """Whether a token opens a sequence [B, T], and which."""
    at = torch.arange(t, device=s["x"].device)
    if s.get("cu") is None:
        return (at == 0)[None].expand(b, t), torch.arange(b, device=at.device)[:, None].expand(b, t)
    seq = torch.searchsorted(s["cu"], at.to(torch.int32), right=True) - 1
    return (s["cu"][seq] == at)[None], seq[None]


def _scan_parts(s):
    x, raw = s["x"].detach().float(), s["dt"].detach().float() + s["dt_bias"].detach()
    step = _softplus(raw)
    a = torch.exp(step[..., None] * s["A"].detach())
    bx = (step * x)[..., None] * _per_channel(s["B"].detach().float(), x.shape[-1])
    starts, seq = _starts(s, x.shape[0], x.shape[1])
    first = starts[..., None, None]
    if s.get("h0") is not None:
        bx = torch.where(first, bx + a * s["h0"][seq], bx)
    return x, raw, step, a, torch.where(first, 0.0, a), bx


def _plain_scan(s):
    x, _, _, _, cut, bx = _scan_parts(s)
    h = _prefix(cut, bx)
    y = (h * _per_channel(s["C"].float(), x.shape[-1])).sum(-1) + s["D"] * x
    if s.get("cu") is None:
        final = h[:, -1].clone()
    else:
        empty = (s["cu"][1:] == s["cu"][:-1])[:, None, None]
        final = torch.where(empty, s["h0"], h[0, (s["cu"][1:].long() - 1).clamp_min(0)])
    return (y * _silu(s["z"].float())).to(s["x"].dtype), final


def _plain_scan_train(s):
    x, raw, step, a, cut, bx = _scan_parts(s)
    d, g = x.shape[-1], s["B"].shape[-2]
    B, C = (_per_channel(s[k].detach().float(), d) for k in ("B", "C"))
    A, skip, z = s["A"].detach(), s["D"].detach(), s["z"].detach().float()
    h = _prefix(cut, bx)
    inner = (h * C).sum(-1) + skip * x
    dy = s["dy"].float()
    din = dy * _silu(z)
    dz = dy * inner * _dsilu(z)
    nxt = torch.cat([cut[:, 1:], torch.zeros_like(cut[:, :1])], 1)
    e = _prefix(nxt.flip(1), (din[..., None] * C).flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    de = e * before * cut  # gradient of the decay's exponent
    eb = (e * B).sum(-1)
    draw_ = (eb * x + (de * A).sum(-1)) / (1.0 + torch.exp(-raw))
    dx = eb * step + skip * din
    shape = x.shape[:2] + (g, d // g, A.shape[1])
    dB = (e * (step * x)[..., None]).reshape(shape).sum(3)
    dC = (h * din[..., None]).reshape(shape).sum(3)
    dA = (de * step[..., None]).sum((0, 1))
    dt = s["x"].dtype
    y = (inner * _silu(z)).to(dt)
    return (y, dx.to(dt), draw_.to(dt), dA, dB.to(dt), dC.to(dt), (din * x).sum((0, 1)), dz.to(dt), draw_.sum((0, 1)))


def _plain_scan_step(s):
    slots, x = s["slots"].long(), s["x"].float()
    step = _softplus(s["dt"].float() + s["dt_bias"])
    d = x.shape[-1]
    h = torch.exp(step[..., None] * s["A"]) * s["state"][slots] + (step * x)[..., None] * _per_channel(s["B"].float(), d)
    y = (h * _per_channel(s["C"].float(), d)).sum(-1) + s["D"] * x
    s["state"][slots] = h
    return (y * _silu(s["z"].float())).to(s["x"].dtype), s["state"]


def _plain_norm(s):
    res = (s["x"].detach().float() + s["residual"].detach().float()).to(s["x"].dtype)
    h = res.float()
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + _EPS)
    return res, h, rstd, h * rstd * s["weight"].detach()


def _plain_norm_fp8(s):
    res, _, _, y = _plain_norm(s)
    q, scale = _quantise(y, 1)
    return q, scale.t().contiguous(), res


def _plain_norm_train(s):
    res, h, rstd, y = _plain_norm(s)
    dy = s["dy"].float()
    hat, g = h * rstd, dy * s["weight"].detach()
    dh = (rstd * (g - hat * (g * hat).mean(-1, keepdim=True)) + s["dres"].float()).to(s["x"].dtype)
    return y.to(s["x"].dtype), res, dh, (dy * hat).sum(0), dh


def _plain_matmul(s):
    m, k = s["a"].shape
    n = s["b"].shape[0]
    a = s["a"].float() * s["a_scales"].t().repeat_interleave(128, 1)[:, :k]
    b = s["b"].float() * s["b_scales"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return (a @ b.t()).to(torch.bfloat16)


_PLAIN = {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan, "scan_train": _plain_scan_train,
          "scan_step": _plain_scan_step, "norm_fp8": _plain_norm_fp8, "norm_train": _plain_norm_train, "matmul": _plain_matmul}


# ---- the package's operators ----------------------------------------------------------------------------------------


def _own(s):
    import gated_deltanet_chunked_delta_gb300 as gdr
    op = s["op"]
    if op == "conv":
        y, _ = gdr.short_conv(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu"])
        return (y.detach(), *torch.autograd.grad(y, s["leaves"], s["dy"]))
    if op == "conv_step":
        return gdr.short_conv_step(s["x"], s["weight"], s["state"], s["bias"], slots=s["slots"]), s["state"]
    if op == "scan":
        return gdr.state_space_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                                    initial_state=s["h0"], output_final_state=True, cu_seqlens=s.get("cu"))
    if op == "scan_train":
        y, _ = gdr.state_space_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"])
        return (y.detach(), *torch.autograd.grad(y, s["leaves"], s["dy"]))
    if op == "scan_step":
        return gdr.state_space_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], s["D"], s["z"], s["dt_bias"],
                                    slots=s["slots"]), s["state"]
    if op == "norm_fp8":
        return gdr.residual_rms_norm_fp8(s["x"], s["weight"], s["residual"], eps=_EPS)
    if op == "norm_train":
        y, res = gdr.residual_rms_norm(s["x"], s["weight"], s["residual"], eps=_EPS)
        return (y.detach(), res.detach(), *torch.autograd.grad((y, res), s["leaves"], (s["dy"], s["dres"])))
    return gdr.block_matmul_fp8(s["a"], s["a_scales"], s["b"], s["b_scales"])


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------------------------------


def work(case):
    op, e = case["op"], 4 if case.get("dtype") == "f32" else 2
    if op == "conv":
        t, d, w = sum(_lengths(case)), case["D"], case["W"]
        # forward x, y; backward x, dy, dx (the gradients need the input again after the loss)
        return {"bytes": 5 * t * d * e + 4 * d * (w + 1) * 3, "flops": t * d * (6 * w + 20)}
    if op == "conv_step":
        r, d, w = case["rows"], case["D"], case["W"]
        return {"bytes": r * d * e * (2 + 2 * (w - 1)) + 4 * d * (w + 1), "flops": r * d * (2 * w + 6)}
    if op == "scan":
        t, d, n, g = case["B"] * case["T"], case["D"], case["N"], case["G"]
        seqs = len(_lengths(case)) if case.get("lengths") else case["B"]
        return {"bytes": e * t * (4 * d + 2 * g * n) + 4 * d * (n + 2) + 4 * d * n * seqs * (2 if case.get("lengths") else 1),
                "flops": t * d * (7 * n + 20)}
    if op == "scan_train":
        t, d, n, g = case["B"] * case["T"], case["D"], case["N"], case["G"]
        # forward x, dt, z, y, B, C; backward x, dt, z, dy, dx, ddt, dz and B, C, dB, dC
        return {"bytes": e * t * (11 * d + 6 * g * n) + 4 * d * (n + 2) * 3, "flops": t * d * (29 * n + 60)}
    if op == "scan_step":
        r, d, n, g = case["rows"], case["D"], case["N"], case["G"]
        return {"bytes": e * r * (4 * d + 2 * g * n) + 8 * r * d * n + 4 * d * (n + 2), "flops": r * d * (7 * n + 20)}
    if op == "norm_fp8":
        m, d = case["M"], case["D"]
        return {"bytes": m * d * (3 * e + 1) + 4 * m * -(-d // 128) + 4 * d, "flops": m * d * 8}
    if op == "norm_train":
        m, d = case["M"], case["D"]
        # forward x, residual, y, sum; backward dy, the sum, its gradient, the result (one for x and residual)
        return {"bytes": 8 * m * d * e + 12 * d, "flops": m * d * 16}
    m, n, k = case["M"], case["N"], case["K"]
    nk = -(-k // 128)
    return {"bytes": m * k + n * k + 2 * m * n + 4 * nk * (m + -(-n // 128)), "flops": 2 * m * n * k}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------------


def _exact_conv(case, s):
    x, w, b, dy = (s[k].detach().double() for k in ("x", "weight", "bias", "dy"))
    taps = w.shape[1]
    ys, dxs, dw, db, at = [], [], torch.zeros_like(w), torch.zeros_like(b), 0
    for n in _lengths(case):
        xs, ds = x[0, at:at + n], dy[0, at:at + n]
        at += n
        pad = torch.cat([xs.new_zeros(taps - 1, xs.shape[1]), xs])
        pre = b.expand_as(xs).clone()
        for j in range(taps):
            pre += pad[j:j + n] * w[:, j]
        sig = torch.sigmoid(pre)
        ys.append(pre * sig)
        dp = ds * (sig + pre * sig * (1 - sig))
        dpad = torch.zeros_like(pad)
        for j in range(taps):
            dpad[j:j + n] += dp * w[:, j]
            dw[:, j] += (dp * pad[j:j + n]).sum(0)
        db += dp.sum(0)
        dxs.append(dpad[taps - 1:])
    return torch.cat(ys)[None], torch.cat(dxs)[None], dw, db


def _exact_conv_step(s):
    y, state = [], s["state"].double()
    w, b, x = s["weight"].double(), s["bias"].double(), s["x"].double()
    for r, slot in enumerate(s["slots"].tolist()):
        pre = b + (state[slot] * w[:, :-1].t()).sum(0) + x[r] * w[:, -1]
        y.append(pre * torch.sigmoid(pre))
        state[slot] = torch.cat([state[slot, 1:], x[r:r + 1]])
    return torch.stack(y), state


def _exact_scan(case, s):
    """Token by token, each sequence on its own; with a gradient of the output, backwards again."""
    v = {k: t.detach().double() for k, t in s.items() if torch.is_tensor(t) and t.is_floating_point()}
    train = "dy" in v
    d = case["D"]
    lens = _lengths(case)
    spans = [(b, 0, case["T"]) for b in range(case["B"])]
    if lens is not None:
        spans, at = [], 0
        for n in lens:
            spans.append((0, at, n))
            at += n
    raw = v["dt"] + v["dt_bias"]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    sig = torch.sigmoid(v["z"])
    wide = lambda m: m.repeat_interleave(d // m.shape[0], 0)  # noqa: E731  [G, N] -> [D, N]
    inner = torch.zeros_like(v["x"])
    final, states = [], []
    for i, (b, at, n) in enumerate(spans):
        h = v["h0"][i] if "h0" in v else torch.zeros_like(v["A"])
        kept = [h]
        for t in range(at, at + n):
            h = torch.exp(step[b, t, :, None] * v["A"]) * h + (step[b, t] * v["x"][b, t])[:, None] * wide(v["B"][b, t])
            inner[b, t] = (h * wide(v["C"][b, t])).sum(1)
            if train:
                kept.append(h)
        final.append(h)
        states.append(kept)
    inner += v["D"] * v["x"]
    y = inner * v["z"] * sig
    if not train:
        return y, torch.stack(final)
    g = case["G"]
    out = {k: torch.zeros_like(v[k]) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")}
    out["z"] = v["dy"] * inner * sig * (1 + v["z"] * (1 - sig))
    din = v["dy"] * v["z"] * sig
    out["D"] = (din * v["x"]).sum((0, 1))
    out["x"] = din * v["D"]
    for (b, at, n), kept in zip(spans, states):
        e = torch.zeros_like(v["A"])
        for t in range(at + n - 1, at - 1, -1):
            e = e + din[b, t, :, None] * wide(v["C"][b, t])
            out["C"][b, t] = (kept[t - at + 1] * din[b, t, :, None]).view(g, d // g, -1).sum(1)
            out["B"][b, t] = (e * (step[b, t] * v["x"][b, t])[:, None]).view(g, d // g, -1).sum(1)
            a = torch.exp(step[b, t, :, None] * v["A"])
            up = e * kept[t - at] * a
            eb = (e * wide(v["B"][b, t])).sum(1)
            out["A"] += up * step[b, t, :, None]
            out["x"][b, t] += eb * step[b, t]
            out["dt"][b, t] = (eb * v["x"][b, t] + (up * v["A"]).sum(1)) * torch.sigmoid(raw[b, t])
            e = e * a
    out["dt_bias"] = out["dt"].sum((0, 1))
    return (y, *(out[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")))


def _exact_scan_step(s):
    v = {k: t.double() for k, t in s.items() if torch.is_tensor(t) and t.is_floating_point()}
    raw = v["dt"] + v["dt_bias"]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    per = v["x"].shape[1] // v["B"].shape[1]
    y, state = [], v["state"].clone()
    for r, slot in enumerate(s["slots"].tolist()):
        h = torch.exp(step[r, :, None] * v["A"]) * state[slot] + (step[r] * v["x"][r])[:, None] * v["B"][r].repeat_interleave(per, 0)
        state[slot] = h
        out = (h * v["C"][r].repeat_interleave(per, 0)).sum(1) + v["D"] * v["x"][r]
        y.append(out * v["z"][r] * torch.sigmoid(v["z"][r]))
    return torch.stack(y), state


def _exact_norm(s):
    x, res = s["x"].detach(), s["residual"].detach()
    total = x.double() + res.double()
    h = total.to(x.dtype).double()  # the norm is of the residual stream as it is stored
    r = 1.0 / torch.sqrt((h ** 2).sum(-1, keepdim=True) / h.shape[1] + _EPS)
    w = s["weight"].detach().double()
    if s["op"] == "norm_train":
        dy = s["dy"].double()
        dh = r * dy * w - h * r ** 3 * (dy * w * h).sum(-1, keepdim=True) / h.shape[1] + s["dres"].double()
        return h * r * w, total, dh, (dy * h * r).sum(0), dh
    y = h * r * w
    q, scales = torch.empty_like(y), []
    for k in range(0, y.shape[1], 128):
        top = y[:, k:k + 128].abs().amax(1).clamp_min(_FLOOR) / 448.0
        scales.append(top)
        q[:, k:k + 128] = y[:, k:k + 128] / top[:, None]
    return q, torch.stack(scales), total


def _exact_matmul(s):
    m, k = s["a"].shape
    n = s["b"].shape[0]
    out = torch.zeros(m, n, dtype=torch.float64, device=s["a"].device)
    rows = torch.arange(n, device=out.device) // 128
    for i, at in enumerate(range(0, k, 128)):
        part = s["a"][:, at:at + 128].double() @ s["b"][:, at:at + 128].double().t()
        out += part * s["a_scales"][i].double()[:, None] * s["b_scales"][rows, i].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "conv":
        return _exact_conv(case, s)
    if op == "conv_step":
        return _exact_conv_step(s)
    if op in ("scan", "scan_train"):
        return _exact_scan(case, s)
    if op == "scan_step":
        return _exact_scan_step(s)
    if op in ("norm_fp8", "norm_train"):
        return _exact_norm(s)
    return _exact_matmul(s)
