"""The plain forms themselves: their gradients against central differences, and the reverse formulas that the kernels
evaluate against those gradients (both in float64, so the formulas agree to rounding: 1e-10)."""
import itertools

import pytest
import torch

import mixer_plain as M
from layer_plain import spans
from test_layer_plain import _check_differences, _rand

LENGTHS = (3, 0, 1, 5)


def test_linear_gradient_against_differences_and_formula():
    gen = torch.Generator().manual_seed(0)
    T, D, c = sum(LENGTHS), 3, 8.0
    x, i, r, z = (_rand(gen, 1, T, D).requires_grad_() for _ in range(4))
    decay, h0 = (_rand(gen, D) - 3).requires_grad_(), _rand(gen, 4, D).requires_grad_()
    dy, dht = _rand(gen, 1, T, D), _rand(gen, 4, D)
    leaves = [x, i, r, decay, z, h0]
    dx, di, dr, ddecay, dz, dh0 = _check_differences(lambda *a: M.linear(*a, LENGTHS), leaves, [dy, dht])
    with torch.no_grad():
        si, sr, soft = torch.sigmoid(i), torch.sigmoid(r), torch.log1p(torch.exp(decay))
        L = -c * soft * sr
        a, m = torch.exp(L), torch.sqrt(-torch.expm1(2 * L))
        total = torch.zeros(D, dtype=torch.float64)
        for s, (_, at, n) in enumerate(spans(1, T, LENGTHS)):
            hs = [h0[s]]
            for t in range(at, at + n):
                hs.append(a[0, t] * hs[-1] + m[0, t] * si[0, t] * x[0, t])
            e = dht[s]
            for t in range(at + n - 1, at - 1, -1):
                e = e + dy[0, t] * M.silu(z[0, t])
                u = si[0, t] * x[0, t]
                G = e * (L[0, t] * a[0, t] * hs[t - at] + u * a[0, t] ** 2 * (-L[0, t] / m[0, t]))
                assert torch.allclose(dx[0, t], e * m[0, t] * si[0, t], atol=1e-10)
                assert torch.allclose(di[0, t], e * m[0, t] * u * (1 - si[0, t]), atol=1e-10)
                assert torch.allclose(dr[0, t], G * (1 - sr[0, t]), atol=1e-10)
                sz = torch.sigmoid(z[0, t])
                assert torch.allclose(dz[0, t], dy[0, t] * hs[t - at + 1] * sz * (1 + z[0, t] * (1 - sz)), atol=1e-10)
                total += G
                e = a[0, t] * e
            assert torch.allclose(dh0[s], e, atol=1e-10)
        assert torch.allclose(ddecay, torch.sigmoid(decay) / soft * total, atol=1e-10)


def test_delta_step_is_the_rule():
    """S <- e^g (I - beta k k^T) S + beta k v^T."""
    gen = torch.Generator().manual_seed(1)
    q, k, v = _rand(gen, 2, 2, 5), _rand(gen, 2, 2, 5), _rand(gen, 2, 4, 3)
    g, beta, state = -_rand(gen, 2, 4).abs(), torch.sigmoid(_rand(gen, 2, 4)), _rand(gen, 2, 4, 5, 3)
    o, new, mag_o, mag = M.delta_step(q, k, v, g, beta, state, 0.4)
    for r, h in itertools.product(range(2), range(4)):
        kk, qq = k[r, h // 2], q[r, h // 2]
        want = torch.exp(g[r, h]) * (torch.eye(5, dtype=torch.float64) - beta[r, h] * torch.outer(kk, kk)) @ state[r, h]
        want = want + beta[r, h] * torch.outer(kk, v[r, h])
        assert torch.allclose(new[r, h], want, atol=1e-12) and torch.allclose(o[r, h], 0.4 * want.t() @ qq, atol=1e-12)
    assert (o.abs() <= mag_o + 1e-12).all() and (new.abs() <= mag + 1e-12).all()


@pytest.mark.parametrize("gated,added,after", list(itertools.product([True, False], repeat=3)))
def test_block_norm_gradient_against_differences_and_formula(gated, added, after):
    gen = torch.Generator().manual_seed(2)
    m, d, scale, eps = 3, 10, 0.7, 1e-6
    x, w = _rand(gen, m, d).requires_grad_(), _rand(gen, d).requires_grad_()
    gate, res, w2 = (_rand(gen, *s).requires_grad_() if on else None for on, s in ((gated, (m, d)), (added, (m, d)), (after, (d,))))
    dy, dr = _rand(gen, m, d), _rand(gen, m, d)
    leaves = [t for t in (x, w, gate, res, w2) if t is not None]

    def f(*a):
        a = list(a)
        full = [a.pop(0) if t is not None else None for t in (x, w, gate, res, w2)]
        y, r = M.block_norm(*full, scale, eps)
        return (r,) if y is None else (r, y)

    grads = dict(zip([n for n, t in zip(("x", "w", "gate", "res", "w2"), (x, w, gate, res, w2)) if t is not None],
                     _check_differences(f, leaves, [dr, dy][:1 + after])))
    with torch.no_grad():
        rx = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        n, sg = x * rx, M.silu(gate) if gated else torch.ones(m, d, dtype=torch.float64)
        c = n * w * sg
        r = scale * c + (res if added else 0)
        total, s2, k = dr, 0, 0
        if after:
            rr = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
            fy = dy * w2
            k = rr ** 3 * (fy * r).mean(-1, keepdim=True)
            assert torch.allclose(grads["w2"], (dy * r * rr).sum(0), atol=1e-10)
            total = dr + rr * fy
            s2 = (r * c).sum(-1, keepdim=True)
        mean = scale * ((total * c).sum(-1, keepdim=True) - k * s2) / d
        total = total - k * r
        if added:
            assert torch.allclose(grads["res"], total, atol=1e-10)
        du = scale * total
        assert torch.allclose(grads["x"], rx * (du * w * sg - n * mean), atol=1e-10)
        assert torch.allclose(grads["w"], (du * n * sg).sum(0), atol=1e-10)
        if gated:
            s = torch.sigmoid(gate)
            assert torch.allclose(grads["gate"], du * n * w * s * (1 + gate * (1 - s)), atol=1e-10)
