"""Plain 64-bit forms of the layer operators, token by token, for the tests.

Every function takes the tensors that the operator gets (any floating type)
and computes in float64 on the CPU; gradients come from torch.autograd over
these loops, and test_layer_plain.py holds them against differences.
"""
import torch


def f64(t, grad=False):
    if t is None:
        return None
    t = t.detach().to("cpu", torch.float64)
    return t.requires_grad_() if grad else t


def spans(B, T, lengths):
    """(batch row, first token, tokens) of every sequence."""
    if lengths is None:
        return [(b, 0, T) for b in range(B)]
    out, at = [], 0
    for n in lengths:
        out.append((0, at, n))
        at += n
    return out


def conv(x, weight, bias=None, silu=True, h0=None, lengths=None):
    B, T, D = x.shape
    W = weight.shape[1]
    rows = [[None] * T for _ in range(B)]
    finals = []
    for i, (b, at, n) in enumerate(spans(B, T, lengths)):
        before = h0[i] if h0 is not None else x.new_zeros(W - 1, D)
        seen = torch.cat([before, x[b, at:at + n]])
        for t in range(n):
            pre = (seen[t:t + W] * weight.t()).sum(0)
            if bias is not None:
                pre = pre + bias
            rows[b][at + t] = pre * torch.sigmoid(pre) if silu else pre
        finals.append(seen[n:])
    y = torch.stack([torch.stack(r) if r else x.new_zeros(0, D) for r in rows])
    return y, torch.stack(finals)


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, h0=None, lengths=None):
    nb, T, d = x.shape
    g, n = B.shape[2:]
    raw = dt if dt_bias is None else dt + dt_bias
    step = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    rows = [[None] * T for _ in range(nb)]
    finals = []
    for i, (b, at, m) in enumerate(spans(nb, T, lengths)):
        h = h0[i] if h0 is not None else x.new_zeros(d, n)
        for t in range(at, at + m):
            Bt, Ct = (v[b, t].repeat_interleave(d // g, 0) for v in (B, C))
            h = torch.exp(step[b, t, :, None] * A) * h + (step[b, t] * x[b, t])[:, None] * Bt
            u = (h * Ct).sum(1)
            if D is not None:
                u = u + D * x[b, t]
            rows[b][t] = u if z is None else u * z[b, t] * torch.sigmoid(z[b, t])
        finals.append(h)
    y = torch.stack([torch.stack(r) if r else x.new_zeros(0, d) for r in rows])
    return y, torch.stack(finals)


def norm(r, weight, eps=1e-6):
    return r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * weight


def matmul(a, a_scales, b, b_scales):
    """The product and the sum of its terms' magnitudes."""
    m, k = a.shape
    n = b.shape[0]
    af, bf = f64(a.float()), f64(b.float())
    af = af * f64(a_scales).t().repeat_interleave(128, 1)[:, :k]
    bf = bf * f64(b_scales).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return af @ bf.t(), af.abs() @ bf.abs().t()
