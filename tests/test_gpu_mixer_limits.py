"""Calls at the edges of what the linear recurrence, the delta rule's step and the norm after a block take: most rows and heads,
gradients that are expanded or turned, a graph used twice, scans of several tiles a CTA captured and replayed, rows without a
batch.  Each against the same work called in another way, bit for bit."""
import pytest
import torch

from test_gpu_layer import gdr, gen_of, rand  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_most_rows_of_the_linear_step(gdr):  # noqa: F811
    gen, rows, D = gen_of(131), 65535, 72
    x, i, r = (rand(gen, rows, D, dt=torch.bfloat16) for _ in range(3))
    decay, state = rand(gen, D) - 3, rand(gen, rows, D)
    small = state.clone()
    y = gdr.gated_linear_step(x, i, r, decay, state)
    for at in (slice(0, 40000), slice(40000, rows)):
        assert torch.equal(y[at], gdr.gated_linear_step(x[at], i[at], r[at], decay, small[at]))
    assert torch.equal(state, small)
    more = torch.zeros(rows + 1, D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gdr.GdrError):
        gdr.gated_linear_step(more, more, more, decay, torch.zeros(rows + 1, D, device="cuda"))


@pytest.mark.parametrize("rows,heads", [(65535, 1), (1, 65535)])
def test_most_rows_and_heads_of_the_delta_step(gdr, rows, heads):  # noqa: F811
    gen = gen_of(132)
    q, k, v = (rand(gen, rows, heads, 64, dt=torch.bfloat16) * 0.1 for _ in range(3))
    g, beta, state = -rand(gen, rows, heads).abs(), torch.sigmoid(rand(gen, rows, heads)), rand(gen, rows, heads, 64, 64)
    small = state.clone()
    o = gdr.gated_delta_step(q, k, v, g, beta, state)
    cut = 30001
    for at in (slice(0, cut), slice(cut, None)):
        pick = (lambda t: t[at]) if rows > 1 else (lambda t: t[:, at].contiguous())
        part = pick(small)
        assert torch.equal(pick(o), gdr.gated_delta_step(*(pick(t) for t in (q, k, v, g, beta)), part))
        assert torch.equal(pick(state), part)
    more = [torch.zeros(*((rows + 1, heads) if rows > 1 else (rows, heads + 1)), n, dtype=torch.bfloat16, device="cuda") for n in (64, 64, 64)]
    gates = torch.zeros(more[0].shape[:2], device="cuda")
    with pytest.raises(gdr.GdrError):
        gdr.gated_delta_step(*more, gates, gates, torch.zeros(*more[0].shape[:2], 64, 64, device="cuda"))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_gradients_of_any_layout(gdr, dt):  # noqa: F811
    """Expanded and turned gradients, and one graph used twice."""
    gen, B, T, D = gen_of(133), 3, 130, 40
    leaves = [rand(gen, B, T, D, dt=dt).requires_grad_() for _ in range(3)] + [(rand(gen, D) - 3).requires_grad_()]
    y, ht = gdr.gated_linear_scan(*leaves, output_final_state=True)
    x, w, w2 = rand(gen, B, T, D, dt=dt).requires_grad_(), (1 + rand(gen, D)).requires_grad_(), (1 + rand(gen, D)).requires_grad_()
    a, b = gdr.gated_residual_rms_norm(x, w, next_weight=w2)
    one = torch.ones((), device="cuda")
    turned, final = rand(gen, T, B, D, dt=dt).transpose(0, 1), rand(gen, D, B).t()
    flat = rand(gen, B, D, T, dt=dt).transpose(1, 2)
    for gy, gh in ((one.to(dt).expand(B, T, D), one.expand(B, D)), (turned, final), (flat, final)):
        got = torch.autograd.grad([y, ht], leaves, [gy, gh], retain_graph=True)
        want = torch.autograd.grad([y, ht], leaves, [gy.contiguous(), gh.contiguous()], retain_graph=True)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        got = torch.autograd.grad([a, b], [x, w, w2], [gy, gy], retain_graph=True)
        want = torch.autograd.grad([a, b], [x, w, w2], [gy.contiguous(), gy.contiguous()], retain_graph=True)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    (y.float().sum() + a.float().sum()).backward()
    assert all(torch.isfinite(t.grad.float()).all() and t.grad.any() for t in (*leaves, x, w, w2))


def test_captured_scans_of_several_tiles_a_cta(gdr):  # noqa: F811
    """Counters and records are cleared at each replay; more rows than the norm's CTAs take at once."""
    gen, B, T, D = gen_of(134), 2, 1500, 1032
    v = [rand(gen, B, T, D, dt=torch.bfloat16) for _ in range(3)] + [rand(gen, D) - 4, rand(gen, B, T, D, dt=torch.bfloat16)]
    w = 1 + 0.1 * rand(gen, D)
    leaves = [t.requires_grad_() for t in (*v, w)]
    dy = rand(gen, B, T, D, dt=torch.bfloat16)

    def step():
        y, _ = gdr.gated_linear_scan(*v)
        r = gdr.gated_residual_rms_norm(y, w, next_weight=w)[0]
        return [r.detach(), *torch.autograd.grad(r, leaves, dy)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(5):
        with torch.no_grad():
            v[0].copy_(rand(gen, B, T, D, dt=torch.bfloat16))
        graph.replay()
        graph.replay()
        got = [t.clone() for t in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_rows_of_any_rank(gdr):  # noqa: F811
    gen, D = gen_of(135), 96
    x, w, w2 = rand(gen, 2, 1, 3, 5, D), 1 + rand(gen, D), 1 + rand(gen, D)
    y, r = gdr.gated_residual_rms_norm(x.view(-1, D), w, next_weight=w2)
    for shape in ((2, 1, 3, 5, D), (30, 1, D), (1, 30, D)):
        for got, want in zip(gdr.gated_residual_rms_norm(x.view(shape), w, next_weight=w2), (y, r)):
            assert got.shape == shape and torch.equal(got.view(-1, D), want)
    one = [t.requires_grad_() for t in (x[0, 0, 0, 0].clone(), w, w2)]
    y1, r1 = gdr.gated_residual_rms_norm(one[0], one[1], next_weight=one[2])
    assert y1.shape == (D,) and torch.equal(y1, y[0]) and torch.equal(r1, r[0])
    g = torch.autograd.grad([y1, r1], one, [y1.detach(), r1.detach()])
    assert [t.shape for t in g] == [(D,)] * 3
