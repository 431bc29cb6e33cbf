"""The plain forms themselves: gradients of the token loops against central
differences, and the reverse formulas that the kernels evaluate against those
gradients (both in float64, so the formulas agree to rounding: 1e-10)."""
import torch

import layer_plain as P

LENGTHS = (3, 0, 1, 5)


def _rand(gen, *s):
    return torch.randn(*s, generator=gen, dtype=torch.float64)


def _check_differences(f, leaves, weights, step=1e-6):
    outs = f(*leaves)
    loss = sum((o * w).sum() for o, w in zip(outs, weights))
    grads = torch.autograd.grad(loss, leaves)
    for leaf, g in zip(leaves, grads):
        flat = leaf.detach().reshape(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 7)):
            vals = []
            for s in (step, -step):
                moved = flat.clone()
                moved[i] += s
                args = [moved.view(leaf.shape) if p is leaf else p for p in leaves]
                vals.append(sum((o * w).sum().detach() for o, w in zip(f(*args), weights)))
            diff = float(vals[0] - vals[1]) / (2 * step)
            # truncation step^2 and cancellation 2^-52 / step, with derivatives of order ten
            assert abs(diff - float(g.reshape(-1)[i])) <= 1e-7 * (1 + abs(diff))
    return grads


def test_conv_gradient_against_differences_and_formula():
    gen = torch.Generator().manual_seed(0)
    T, D, W = sum(LENGTHS), 3, 4
    x, w, b, h0 = (v.requires_grad_() for v in (_rand(gen, 1, T, D), _rand(gen, D, W), _rand(gen, D), _rand(gen, 4, W - 1, D)))
    dy, dht = _rand(gen, 1, T, D), _rand(gen, 4, W - 1, D)
    dx, dw, db, dh0 = _check_differences(lambda *a: P.conv(a[0], a[1], a[2], True, a[3], LENGTHS), [x, w, b, h0], [dy, dht])
    with torch.no_grad():  # dx_s = sum_j w_j dp_{s + W - 1 - j} (+ the final state's gradient), dw_j, db
        pre, _ = P.conv(x, w, b, False, h0, LENGTHS)
        s = torch.sigmoid(pre)
        dp = dy * s * (1 + pre * (1 - s))
        for i, (_, at, n) in enumerate(P.spans(1, T, LENGTHS)):
            for t in range(at, at + n):
                want = sum(w[:, j] * dp[0, t + W - 1 - j] for j in range(W) if t + W - 1 - j < at + n)
                k = W - 1 - (at + n - t)
                want = want + (dht[i, k] if k >= 0 else 0)
                assert torch.allclose(dx[0, t], want, atol=1e-10)
            for r in range(W - 1):
                want = sum((w[:, r - u] * dp[0, at + u] for u in range(min(n, r + 1))), torch.zeros(D, dtype=torch.float64))
                want = want + (dht[i, r - n] if r >= n else 0)
                assert torch.allclose(dh0[i, r], want, atol=1e-10)
        assert torch.allclose(db, dp.sum((0, 1)), atol=1e-10)


def test_scan_gradient_against_differences_and_formula():
    gen = torch.Generator().manual_seed(1)
    T, D, G, N = sum(LENGTHS), 4, 2, 8
    x, dt, z = (_rand(gen, 1, T, D).requires_grad_() for _ in range(3))
    B, C = (_rand(gen, 1, T, G, N).requires_grad_() for _ in range(2))
    A = (-torch.rand(D, N, generator=gen, dtype=torch.float64) * 2).requires_grad_()
    skip, bias, h0 = (v.requires_grad_() for v in (_rand(gen, D), _rand(gen, D), _rand(gen, 4, D, N)))
    dy, dht = _rand(gen, 1, T, D), _rand(gen, 4, D, N)
    leaves = [x, dt, A, B, C, skip, z, bias, h0]
    grads = _check_differences(lambda *a: P.scan(*a[:8], True, a[8], LENGTHS), leaves, [dy, dht])
    dx, ddt, dA, dB, dC, dD, dz, dbias, dh0 = grads
    with torch.no_grad():
        raw = dt + bias
        s = torch.logaddexp(raw, torch.zeros_like(raw))
        sg = torch.sigmoid(z)
        du = dy * z * sg
        gA, gB, gC = torch.zeros_like(A), torch.zeros_like(B), torch.zeros_like(C)
        for i, (_, at, n) in enumerate(P.spans(1, T, LENGTHS)):
            hs = [h0[i]]
            for t in range(at, at + n):
                hs.append(torch.exp(s[0, t, :, None] * A) * hs[-1] + (s[0, t] * x[0, t])[:, None] * B[0, t].repeat_interleave(D // G, 0))
            e = dht[i]
            for t in range(at + n - 1, at - 1, -1):
                Bt, Ct = (v[0, t].repeat_interleave(D // G, 0) for v in (B, C))
                h = hs[t - at + 1]
                e = e + du[0, t, :, None] * Ct
                eb = (e * Bt).sum(1)
                gC[0, t] = (h * du[0, t, :, None]).view(G, D // G, N).sum(1)
                gB[0, t] = (e * (s[0, t] * x[0, t])[:, None]).view(G, D // G, N).sum(1)
                e = e * torch.exp(s[0, t, :, None] * A)
                f = e * hs[t - at]
                gA += f * s[0, t, :, None]
                assert torch.allclose(dx[0, t], s[0, t] * eb + skip * du[0, t], atol=1e-10)
                assert torch.allclose(ddt[0, t], (x[0, t] * eb + (f * A).sum(1)) * torch.sigmoid(raw[0, t]), atol=1e-10)
                u = (h * Ct).sum(1) + skip * x[0, t]
                assert torch.allclose(dz[0, t], dy[0, t] * u * sg[0, t] * (1 + z[0, t] * (1 - sg[0, t])), atol=1e-10)
            assert torch.allclose(dh0[i], e, atol=1e-10)
        for got, want in ((dA, gA), (dB, gB), (dC, gC), (dD, (du * x).sum((0, 1))), (dbias, ddt.sum((0, 1)))):
            assert torch.allclose(got, want, atol=1e-10)


def test_norm_gradient_against_differences_and_formula():
    gen = torch.Generator().manual_seed(2)
    r, w = _rand(gen, 3, 10).requires_grad_(), _rand(gen, 10).requires_grad_()
    dy = _rand(gen, 3, 10)
    dr, dw = _check_differences(lambda a, b: (P.norm(a, b),), [r, w], [dy])
    with torch.no_grad():
        rstd = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-6)
        k = rstd ** 2 * (dy * w * r).mean(-1, keepdim=True)
        assert torch.allclose(dr, rstd * (dy * w - r * k), atol=1e-10)
        assert torch.allclose(dw, (dy * r * rstd).sum(0), atol=1e-10)
