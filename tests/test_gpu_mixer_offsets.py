"""Offsets past 32 bits in the linear scan and in the norm's gradient, on varying data: strides that reach past 2^31 elements,
and outputs and gradients of more than 2^31 elements, against the same work in smaller pieces, bit for bit."""
import pytest
import torch

from test_gpu_layer import gdr, gen_of, rand  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def fill(t, gen):
    """Random values, a part at a time."""
    for part in t.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda", dtype=torch.bfloat16))


def test_scan_of_far_strides(gdr):  # noqa: F811
    """Every token holds other values, so that one read at a wrapped offset shows."""
    gen, T, stride = gen_of(121), (1 << 18) + 130, 8192
    assert (T - 1) * stride > 1 << 31
    wide = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    parts = [wide.as_strided((1, T, 64), (T * stride, stride, 1), at) for at in (0, 64, 128, 256)]
    near = [rand(gen, 1, T, 64, dt=torch.bfloat16) for _ in parts]
    for far, n in zip(parts, near):
        far.copy_(n)
    decay, dy, dht = rand(gen, 64) - 3, rand(gen, 1, T, 64, dt=torch.bfloat16), rand(gen, 1, 64)

    def run(x, i, r, z):
        leaves = [t.detach().requires_grad_() for t in (x, i, r, decay, z)]
        y, ht = gdr.gated_linear_scan(*leaves, output_final_state=True)
        return (y.detach(), ht.detach(), *torch.autograd.grad([y, ht], leaves, [dy, dht]))

    for a, b in zip(run(*parts), run(*near)):
        assert torch.isfinite(b.float()).all() and torch.equal(a, b)


def test_scan_of_far_outputs(gdr):  # noqa: F811
    """More than 2^31 elements of output and of each gradient; the inputs are one sequence, states and gradients each row's own."""
    gen, B, T, D = gen_of(122), 1050, 2048, 1024
    assert B * T * D > (1 << 31) + (1 << 24)
    x, i, r = (rand(gen, 1, T, D, dt=torch.bfloat16).expand(B, T, D) for _ in range(3))
    decay, h0, dht = torch.full((D,), -6.0, device="cuda"), rand(gen, B, D), rand(gen, B, D)
    dy = torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda")
    fill(dy, gen)

    def run(at):
        leaves = [t.detach().requires_grad_() for t in (x[at], i[at], r[at], h0[at])]
        y, ht = gdr.gated_linear_scan(*leaves[:3], decay, initial_state=leaves[3], output_final_state=True)
        return (y.detach(), ht.detach(), *torch.autograd.grad([y, ht], leaves, [dy[at], dht[at]]))

    whole = run(slice(0, B))
    for n in range(0, B, 150):
        at = slice(n, n + 150)
        for a, b in zip(whole, run(at)):
            assert torch.equal(a[at], b)
    assert not torch.equal(whole[0][0], whole[0][-1])


def test_norm_gradient_of_far_rows(gdr):  # noqa: F811
    gen, rows, D = gen_of(123), (1 << 20) + 7, 2056
    assert rows * D > 1 << 31
    x, res, dr, dy = (torch.empty(rows, D, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    for t in (x, res, dr, dy):
        fill(t, gen)
    w, w2 = 1 + 0.1 * rand(gen, D), 1 + 0.1 * rand(gen, D)

    def run(at):
        leaves = [t.detach().requires_grad_() for t in (x[at], res[at], w, w2)]
        y, r = gdr.gated_residual_rms_norm(leaves[0], leaves[2], residual=leaves[1], next_weight=leaves[3], scale=0.5)
        return (y.detach(), r.detach(), *torch.autograd.grad([y, r], leaves, [dy[at], dr[at]]))

    whole, sums = run(slice(0, rows)), [0.0, 0.0]
    for n in range(0, rows, 1 << 18):
        at = slice(n, min(n + (1 << 18), rows))
        part = run(at)
        assert all(torch.equal(a[at], b) for a, b in zip(whole[:4], part))
        sums = [s + g.double() for s, g in zip(sums, part[4:])]
    # A channel's terms have a variance below 1, so a CTA's running sum (of 2300 rows, 456 CTAs; in the parts fewer) stays below
    # 6 sqrt(2300) = 288, and each row's addition rounds to 2^-24 of that; twice, for both sides.
    for g, s in zip(whole[4:], sums):
        assert ((g.double() - s).abs() <= 2 * rows * 288 * 2.0 ** -24).all() and float(s.abs().max()) > 300
