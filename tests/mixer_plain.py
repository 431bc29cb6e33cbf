"""Plain 64-bit forms of the gated linear recurrence, the delta rule's single token and the norm after a block, for the
tests: float64 on the CPU, gradients from torch.autograd (held against differences in test_mixer_plain.py)."""
import torch

from layer_plain import spans


def silu(v):
    return v * torch.sigmoid(v)


def linear(x, input_gate, decay_gate, decay, z=None, h0=None, lengths=None, scale=8.0):
    """y and the final states, token by token."""
    B, T, D = x.shape
    log_a = -scale * torch.nn.functional.softplus(decay, threshold=1e9) * torch.sigmoid(decay_gate)
    a = torch.exp(log_a)
    add = torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(input_gate) * x
    rows, finals = [[None] * T for _ in range(B)], []
    for i, (b, at, n) in enumerate(spans(B, T, lengths)):
        h = h0[i] if h0 is not None else x.new_zeros(D)
        for t in range(at, at + n):
            h = a[b, t] * h + add[b, t]
            rows[b][t] = h if z is None else h * silu(z[b, t])
        finals.append(h)
    y = torch.stack([torch.stack(r) if r else x.new_zeros(0, D) for r in rows])
    return y, torch.stack(finals)


def delta_step(q, k, v, g, beta, state, scale):
    """o and the new states of the rows; and the sums of the magnitudes of their terms."""
    per = v.shape[1] // q.shape[1]
    q, k = (t.repeat_interleave(per, 1) for t in (q, k))
    old = state * torch.exp(g)[..., None, None]
    w = beta[..., None] * (v - (old * k[..., None]).sum(-2))
    new = old + k[..., None] * w[..., None, :]
    mag_w = beta.abs()[..., None] * (v.abs() + (old * k[..., None]).abs().sum(-2))
    mag = old.abs() + k.abs()[..., None] * mag_w[..., None, :]
    return scale * (new * q[..., None]).sum(-2), new, scale * (mag * q.abs()[..., None]).sum(-2), mag


def block_norm(x, weight, gate=None, residual=None, next_weight=None, scale=1.0, eps=1e-6):
    u = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight
    if gate is not None:
        u = u * silu(gate)
    r = scale * u if residual is None else residual + scale * u
    y = None if next_weight is None else r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * next_weight
    return y, r
