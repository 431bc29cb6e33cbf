"""The gated linear recurrence, the delta rule's single token and the norm after a block on the GPU against the plain
64-bit forms, at the sizes and masks where they can go wrong.

Tolerances, set before the first run.  u is half a step of the output's type (bf16 2^-8, fp32 2^-24).

* recurrence, held by ``err`` = max (|x - ref| - u |x|) / rms(ref): a step's decay is off by 2^-21 of it (ex2.approx
  2^-22, its argument's rounding, sigmoid), which a state adds up over the tokens it remembers, at most T; the rest
  (softplus, sigmoids, square root, silu, gradients' products) is 2^-17.  32 covers the largest element over the rms;
* delta step, per element with the sum S of the terms' magnitudes: sums of 12 sequential products, then trees, and four
  products after them: 2^-19 S;
* norm after a block, per element: a sum of D squares (16 sequential, then trees) 2^-19, silu 2^-20 (ex2.approx 2^-22,
  rcp.approx 2^-23, its argument's rounding), five products: 2^-18 of each term of r, 2^-17 of what y makes of them.
  Gradients by ``err``: 32 (2^-17 + M 2^-24), the latter for the sum over M rows.
"""
import itertools

import pytest
import torch

import mixer_plain as M
from layer_plain import f64
from test_gpu_layer import DT, U, bounds, close, gdr, gen_of, rand  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


# ---- gated linear recurrence ---------------------------------------------------

LINEAR = [  # B, T, D, lengths, h0, gate
    (1, 1, 1, None, False, False), (1, 1, 64, None, True, True), (3, 2, 33, None, True, False), (2, 15, 31, None, False, True),
    (1, 16, 66, None, True, True), (1, 17, 32, None, True, False), (2, 64, 40, None, True, True), (1, 65, 130, None, False, False),
    (1, 127, 64, None, True, True), (2, 128, 62, None, False, True), (1, 129, 37, None, True, False), (1, 400, 70, None, True, True),
    (2, 700, 34, None, True, True), (1, 1300, 6, None, False, False),
    (1, 171, 40, (0, 3, 1, 0, 64, 32, 71, 0), True, True), (1, 260, 33, (129, 1, 1, 129), True, False), (1, 5, 8, (0, 0, 5, 0), True, True),
    (1, 514, 66, (128, 128, 1, 257), False, True), (1, 450, 9, (64, 64, 16, 306), True, True), (1, 200, 64, (200,), True, False),
    (1, 130, 2, (1,) * 130, True, True), (1, 3, 64, (0,) * 40 + (3,) + (0,) * 40, True, True)]


def linear_inputs(case, dt, seed=51):
    B, T, D, lengths, has_h0, gate = case
    gen, t = gen_of(seed), DT[dt]
    n = len(lengths) if lengths else B
    v = dict(x=rand(gen, B, T, D, dt=t), input_gate=rand(gen, B, T, D, dt=t), decay_gate=rand(gen, B, T, D, dt=t),
             decay=rand(gen, D) - 3, z=rand(gen, B, T, D, dt=t) if gate else None, initial_state=rand(gen, n, D) if has_h0 else None)
    return v, rand(gen, B, T, D, dt=t), rand(gen, n, D)


def linear_plain(v, lengths, grad=True):
    p = {k: f64(t, grad) for k, t in v.items()}
    h0 = p.pop("initial_state")
    y, ht = M.linear(**p, h0=h0, lengths=lengths)
    return y, ht, {**p, "initial_state": h0}


def linear_tol(T):
    return 32 * (T * 2.0 ** -21 + 2.0 ** -17)


def linear_check(gdr, v, dy, dht, lengths):  # noqa: F811
    names = [k for k in v if v[k] is not None]
    for k in names:
        v[k].requires_grad_()
    y, ht = gdr.gated_linear_scan(**v, output_final_state=True, cu_seqlens=bounds(lengths))
    grads = torch.autograd.grad([y, ht], [v[k] for k in names], [dy, dht])
    ry, rht, p = linear_plain(v, lengths)
    rg = torch.autograd.grad([ry, rht], [p[k] for k in names], [f64(dy), f64(dht)])
    tol = linear_tol(y.shape[1])
    close(y, ry, tol, "y")
    close(ht, rht, tol, "final")
    for k, g, r in zip(names, grads, rg):
        assert g.dtype is v[k].dtype
        close(g, r, tol, k)
    with torch.no_grad():  # without a gradient the same bits
        y2, ht2 = gdr.gated_linear_scan(**v, output_final_state=True, cu_seqlens=bounds(lengths))
        assert torch.equal(y, y2) and torch.equal(ht, ht2)
        assert gdr.gated_linear_scan(**v, cu_seqlens=bounds(lengths))[1] is None


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", LINEAR, ids=str)
def test_linear(gdr, case, dt):  # noqa: F811
    v, dy, dht = linear_inputs(case, dt)
    linear_check(gdr, v, dy, dht, case[3])


def test_linear_decay_scales_and_extreme_gates(gdr):  # noqa: F811
    """Gates far open and far closed (a = 1 and m = 0 in 32 bits, a = 0), decays from none to all."""
    for scale in (0.5, 8.0, 300.0):
        v, dy, dht = linear_inputs((1, 90, 12, None, True, True), "f32", 52)
        v["decay"] = torch.tensor([-200.0, -90.0, -40.0, -20.0, -12.0, -8.0, -4.0, 0.0, 3.0, 10.0, 50.0, 300.0], device="cuda")
        for k in ("input_gate", "decay_gate", "z"):
            v[k][0, 10:20] = -120.0
            v[k][0, 30:40] = 120.0
            v[k][0, 50:60] *= 20.0
        names = [k for k in v]
        for k in names:
            v[k].requires_grad_()
        y, ht = gdr.gated_linear_scan(**v, decay_scale=scale, output_final_state=True)
        grads = torch.autograd.grad([y, ht], [v[k] for k in names], [dy, dht])
        p = {k: f64(t, True) for k, t in v.items()}
        h0 = p.pop("initial_state")
        ry, rht = M.linear(**p, h0=h0, scale=scale)
        p["initial_state"] = h0
        # the formula in the form that has no 0 / 0: log a is bounded away from zero by what 64 bits hold
        rg = torch.autograd.grad([ry, rht], [p[k] for k in names], [f64(dy), f64(dht)])
        close(y, ry, linear_tol(90), "y")
        close(ht, rht, linear_tol(90), "final")
        for k, g, r in zip(names, grads, rg):
            assert torch.isfinite(g).all(), k
            close(g, torch.nan_to_num(r), linear_tol(90), k)


def test_linear_results_do_not_change_between_runs(gdr):  # noqa: F811
    """However the chunks' CTAs come to run beside one another."""
    v, dy, dht = linear_inputs((2, 5000, 200, None, True, True), "bf16", 53)
    names = [k for k in v]
    for k in names:
        v[k].requires_grad_()

    def run():
        y, ht = gdr.gated_linear_scan(**v, output_final_state=True)
        return (y.detach(), ht.detach(), *torch.autograd.grad([y, ht], [v[k] for k in names], [dy, dht]))

    first = run()
    junk = torch.randn(4096, 4096, device="cuda")
    for _ in range(4):
        junk = (junk @ junk).clamp(-1, 1)
        assert all(torch.equal(a, b) for a, b in zip(first, run()))


def test_linear_one_output_in_the_loss(gdr):  # noqa: F811
    case = (2, 200, 16, None, True, True)
    v, dy, dht = linear_inputs(case, "f32", 54)
    for k in v:
        v[k].requires_grad_()
    for which, g in ((0, dy), (1, dht)):
        outs = gdr.gated_linear_scan(**v, output_final_state=True)
        got = torch.autograd.grad(outs[which], [v["x"], v["decay"], v["initial_state"]], g)
        y, ht, p = linear_plain(v, None)
        want = torch.autograd.grad((y, ht)[which], [p["x"], p["decay"], p["initial_state"]], f64(g))
        for a, b in zip(got, want):
            close(a, b, linear_tol(200), "grad")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_reads_slices(gdr, dt):  # noqa: F811
    """Slices of one projection, aligned and not, and tokens outside the batch: results as from contiguous inputs, gradients
    among them."""
    v, dy, _ = linear_inputs((2, 150, 32, None, True, True), dt, 55)
    names = ("x", "input_gate", "decay_gate", "z")

    def run(w):
        leaves = [w[k].requires_grad_() for k in names]
        y, _ = gdr.gated_linear_scan(**w)
        return (y.detach(), *torch.autograd.grad(y, leaves, dy))

    want = run({k: t.clone() for k, t in v.items()})
    for off in (0, 8, 2, 5):
        big = torch.zeros(2, 150, 32 * 4 + 16, dtype=DT[dt], device="cuda")
        s = dict(v)
        for n, k in enumerate(names):
            at = off + 32 * n
            big[:, :, at:at + 32] = v[k].detach()
            s[k] = big[:, :, at:at + 32].detach()
        for a, b in zip(want, run(s)):
            assert torch.equal(a, b)
    s = {k: (t.detach().transpose(0, 1).contiguous().transpose(0, 1) if k in names else t) for k, t in v.items()}
    assert all(torch.equal(a, b) for a, b in zip(want, run(s)))
    s = {k: (t.detach()[:1].expand(2, -1, -1) if k in names else t) for k, t in v.items()}  # one row for both
    y, _ = gdr.gated_linear_scan(**s)
    assert torch.equal(y, gdr.gated_linear_scan(**{k: (t.contiguous() if k in names else t) for k, t in s.items()})[0])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D,S,gate", [(1, 1, 1, True), (6, 37, 9, True), (3, 64, 3, False), (5, 1026, 64, True), (70, 8, 70, False)])
def test_linear_step(gdr, rows, D, S, gate, dt):  # noqa: F811
    v, _, _ = linear_inputs((rows, 1, D, None, False, gate), dt, 56)
    v.pop("initial_state")
    gen = gen_of(57)
    state = rand(gen, S, D)
    slots = torch.randperm(S, generator=gen, device="cuda")[:rows].to(torch.int32)
    if rows > 2:
        slots[2] = -3
    was = state.clone()
    one = {k: (t[:, 0] if t is not None and k != "decay" else t) for k, t in v.items()}
    y = gdr.gated_linear_step(**one, state=state, slots=slots)
    live = [r for r, s in enumerate(slots.tolist()) if s >= 0]
    at = slots[live].long()
    p = {k: (f64(t)[live] if t is not None and k != "decay" else f64(t)) for k, t in v.items()}
    ry, rh = M.linear(**p, h0=f64(was[at]))
    close(y[live], ry[:, 0], linear_tol(1), "y")
    close(state[at], rh, linear_tol(1), "state")
    idle = [s for s in range(S) if s not in at.tolist()]
    assert torch.equal(state[idle], was[idle])
    if rows > 2:
        assert not y[2].any()
    if S == rows:  # without slots, row r uses slot r
        a, b = was.clone(), was.clone()
        assert torch.equal(gdr.gated_linear_step(**one, state=a),
                           gdr.gated_linear_step(**one, state=b, slots=torch.arange(rows, dtype=torch.int32, device="cuda")))
        assert torch.equal(a, b)


def test_linear_steps_continue_a_prompt(gdr):  # noqa: F811
    v, _, _ = linear_inputs((2, 145, 24, None, True, True), "f32", 58)
    names = ("x", "input_gate", "decay_gate", "z")
    whole, end = gdr.gated_linear_scan(**v, output_final_state=True)
    cut = {k: (t[:, :140] if k in names else t) for k, t in v.items()}
    _, state = gdr.gated_linear_scan(**cut, output_final_state=True)
    v.pop("initial_state")
    for t in range(140, 145):
        y = gdr.gated_linear_step(**{k: (a[:, t] if k in names else a) for k, a in v.items()}, state=state)
        close(y, f64(whole[:, t]), 2 * linear_tol(145), "y")
    close(state, f64(end), 2 * linear_tol(145), "state")


# ---- one token through the delta rule ------------------------------------------

DELTA = [  # rows, Hq, Hv, K, V, slots
    (1, 1, 1, 64, 64, 1), (3, 2, 4, 128, 128, 5), (5, 4, 4, 128, 256, 5), (2, 1, 3, 192, 192, 7), (4, 2, 2, 64, 256, 4),
    (2, 3, 6, 192, 64, 2), (1, 16, 32, 128, 128, 2)]


def delta_inputs(case, dt, seed=61):
    rows, hq, hv, K, V, S = case
    gen, t = gen_of(seed), DT[dt]
    q, k = (torch.nn.functional.normalize(rand(gen, rows, hq, K), dim=-1).to(t) for _ in range(2))
    return dict(q=q, k=k, v=rand(gen, rows, hv, V, dt=t), g=-rand(gen, rows, hv).abs(), beta=torch.sigmoid(rand(gen, rows, hv))), rand(gen, S, hv, K, V)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", DELTA, ids=str)
def test_delta_step(gdr, case, dt):  # noqa: F811
    rows, S = case[0], case[5]
    v, state = delta_inputs(case, dt)
    slots = torch.randperm(S, generator=gen_of(62), device="cuda")[:rows].to(torch.int32)
    if rows > 2:
        slots[1] = -1
    for scale in (None, 0.3):
        was = state.clone()
        o = gdr.gated_delta_step(**v, state=state, scale=scale, slots=slots)
        live = [r for r, s in enumerate(slots.tolist()) if s >= 0]
        at = slots[live].long()
        p = {k: f64(t)[live] for k, t in v.items()}
        ro, rs, mag_o, mag_s = M.delta_step(**p, state=f64(was[at]), scale=scale or case[3] ** -0.5)
        assert o.dtype is DT[dt]
        assert ((f64(o[live]) - ro).abs() <= U[DT[dt]] * ro.abs() + 2.0 ** -19 * mag_o).all()
        assert ((f64(state[at]) - rs).abs() <= 2.0 ** -24 * rs.abs() + 2.0 ** -19 * mag_s).all()
        idle = [s for s in range(S) if s not in at.tolist()]
        assert torch.equal(state[idle], was[idle])
        if rows > 2:
            assert not o[1].any()
    if S == rows:
        a, b = state.clone(), state.clone()
        assert torch.equal(gdr.gated_delta_step(**v, state=a),
                           gdr.gated_delta_step(**v, state=b, slots=torch.arange(rows, dtype=torch.int32, device="cuda")))
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_delta_step_reads_slices(gdr, dt):  # noqa: F811
    rows, hq, hv, K, V = 3, 2, 4, 128, 64
    v, state = delta_inputs((rows, hq, hv, K, V, 3), dt)
    want_state = state.clone()
    want = gdr.gated_delta_step(**v, state=want_state)
    for off in (0, 8, 3):
        big = torch.zeros(rows, 2 * hq * K + hv * V + 16, dtype=DT[dt], device="cuda")
        at, s = off, dict(v)
        for k, (h, w) in (("q", (hq, K)), ("k", (hq, K)), ("v", (hv, V))):
            big[:, at:at + h * w] = v[k].flatten(1)
            s[k] = big[:, at:at + h * w].unflatten(1, (h, w))
            at += h * w
        now = state.clone()
        assert torch.equal(gdr.gated_delta_step(**s, state=now), want) and torch.equal(now, want_state)


@pytest.mark.parametrize("K,V", [(128, 128), (64, 192)])
def test_delta_steps_continue_a_prompt(gdr, K, V):  # noqa: F811
    """The chunked prefill of 70 tokens and 5 steps against the prefill of 75, both held to the prefill's own tolerance
    (2e-3 of the rms for fp32 inputs, tests/parity.py)."""
    from parity import TOL
    gen, B, T, hq, hv = gen_of(63), 2, 75, 2, 4
    q, k = (torch.nn.functional.normalize(rand(gen, B, T, hq, K), dim=-1) for _ in range(2))
    v, g, beta = rand(gen, B, T, hv, V), -rand(gen, B, T, hv).abs(), torch.sigmoid(rand(gen, B, T, hv))
    h0 = rand(gen, B, hv, K, V)
    with torch.no_grad():
        whole, end = gdr.chunk_gated_delta_rule(q, k, v, g, beta, initial_state=h0, output_final_state=True)
        head = [t[:, :70].contiguous() for t in (q, k, v, g, beta)]
        _, state = gdr.chunk_gated_delta_rule(*head, initial_state=h0, output_final_state=True)
        for t in range(70, 75):
            o = gdr.gated_delta_step(*(a[:, t] for a in (q, k, v)), g[:, t].contiguous(), beta[:, t].contiguous(), state)
            close(o, f64(whole[:, t]), 2 * TOL["f32"], "o")
    close(state, f64(end), 2 * TOL["f32"], "state")


# ---- norm after a block ----------------------------------------------------------

BLOCK = [(1, 1), (3, 5), (2, 8), (7, 37), (40, 64), (33, 128), (19, 200), (5, 256), (6, 500), (3, 512), (2, 520), (3, 1001), (4, 4096),
         (2, 5003), (2, 8192), (2, 8200), (2, 16384), (1, 16383), (700, 264), (3000, 128)]
PARTS = list(itertools.product([True, False], repeat=3))


def block_check(gdr, rows, D, parts, dt, eps, scale=0.7):  # noqa: F811
    gated, added, after = parts
    gen, t = gen_of(71), DT[dt]
    x, w = 2 * rand(gen, rows, D), 1 + 0.1 * rand(gen, D)
    x = x.to(t)
    gate, res = (rand(gen, rows, D, dt=t) if on else None for on in (gated, added))
    w2 = 1 + 0.1 * rand(gen, D) if after else None
    dy, dr = (rand(gen, rows, D, dt=t) for _ in range(2))
    leaves = [v.requires_grad_() for v in (x, w, gate, res, w2) if v is not None]
    y, r = gdr.gated_residual_rms_norm(x, w, gate, res, w2, scale=scale, eps=eps)
    assert (y is None) == (not after) and r.dtype is t
    outs, gs = ([y, r], [dy, dr]) if after else ([r], [dr])
    grads = torch.autograd.grad(outs, leaves, gs)
    plain = [f64(v, True) for v in (x, w, gate, res, w2)]
    ry, rr = M.block_norm(*plain, scale, eps)
    pl = [v for v in plain if v is not None]
    rg = torch.autograd.grad([ry, rr] if after else [rr], pl, [f64(g) for g in gs])
    with torch.no_grad():
        _, u = M.block_norm(plain[0], plain[1], plain[2], None, None, scale, eps)
        mag = u.abs() + (plain[3].abs() if added else 0)
        assert ((f64(r) - rr).abs() <= U[t] * rr.abs() + 2.0 ** -18 * mag + 1e-37).all()
        if after:
            inv = 1 / torch.sqrt((rr * rr).mean(-1, keepdim=True) + eps)
            assert ((f64(y) - ry).abs() <= (U[t] + 2.0 ** -17) * ry.abs() + 2.0 ** -17 * inv * plain[4].abs() * mag + 1e-37).all()
        y2, r2 = gdr.gated_residual_rms_norm(x, w, gate, res, w2, scale=scale, eps=eps)
        assert torch.equal(r, r2) and (not after or torch.equal(y, y2))
    tol = 32 * (2.0 ** -17 + rows * 2.0 ** -24)
    for g, v, leaf in zip(grads, rg, leaves):
        assert g.dtype is leaf.dtype and g.shape == leaf.shape
        close(g, v, tol, str(tuple(leaf.shape)))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", BLOCK)
def test_block_norm(gdr, rows, D, dt):  # noqa: F811
    # rows of few channels: the norm's gradient is what is left of two equal terms unless eps weighs in
    block_check(gdr, rows, D, (True, True, True), dt, 0.3 if D <= 8 else 1e-6)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("parts", PARTS, ids=str)
@pytest.mark.parametrize("rows,D", [(37, 128), (3, 999), (5, 2048)])
def test_block_norm_parts(gdr, rows, D, parts, dt):  # noqa: F811
    block_check(gdr, rows, D, parts, dt, 1e-5, scale=-1.3)


def test_block_norm_one_output_in_the_loss(gdr):  # noqa: F811
    gen = gen_of(72)
    x, gate, res, g = (rand(gen, 9, 300) for _ in range(4))
    w, w2 = 1 + 0.1 * rand(gen, 300), 1 + 0.1 * rand(gen, 300)
    leaves = [t.requires_grad_() for t in (x, w, gate, res, w2)]
    plain = [f64(t, True) for t in leaves]
    for which in (0, 1):
        got = torch.autograd.grad(gdr.gated_residual_rms_norm(*leaves)[which], leaves[:4], g)
        want = torch.autograd.grad(M.block_norm(*plain)[which], plain[:4], f64(g))
        for a, b in zip(got, want):
            close(a, b, 32 * (2.0 ** -17 + 9 * 2.0 ** -24), "grad")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [128, 96, 640])
def test_block_norm_reads_slices(gdr, D, dt):  # noqa: F811
    """Rows of one stride inside a wider tensor, aligned and not, and heads of a mixer's output."""
    gen = gen_of(73)
    wide = rand(gen, 2, 11, 3 * D + 24, dt=DT[dt])
    w, w2 = 1 + 0.1 * rand(gen, D), 1 + 0.1 * rand(gen, D)
    dy, dr = rand(gen, 2, 11, D, dt=DT[dt]), rand(gen, 2, 11, D, dt=DT[dt])

    def run(parts):
        parts = [t.detach().requires_grad_() for t in parts]
        y, r = gdr.gated_residual_rms_norm(parts[0], w, parts[1], parts[2], w2, scale=0.5)
        return (y.detach(), r.detach(), *torch.autograd.grad([y, r], parts, [dy, dr]))

    for off in (0, 8, 3):
        parts = [wide[..., off + i * D:off + (i + 1) * D] for i in range(3)]
        want = run([t.contiguous() for t in parts])
        # the same sums; other threads hold other channels where rows are read element by element
        tol = 0 if off != 3 else 32 * 2.0 ** -17
        for a, b in zip(want, run(parts)):
            if tol:
                close(b, f64(a), tol + (2.0 ** -7 if dt == "bf16" else 0), "slices")
            else:
                assert torch.equal(a, b)
    heads = rand(gen, 2, 11, 4, D, dt=DT[dt])
    _, r = gdr.gated_residual_rms_norm(heads, w)
    assert torch.equal(r.view(-1, D), gdr.gated_residual_rms_norm(heads.view(-1, D), w)[1])
    # heads of a slice of a projection: a stride for tokens and one for heads
    dy, dr = rand(gen, 2, 11, 4, D, dt=DT[dt]), rand(gen, 2, 11, 4, D, dt=DT[dt])
    wide = rand(gen, 2, 11, 8 * D + 8, dt=DT[dt])
    slices = [heads, *(wide[..., off:off + 4 * D].unflatten(-1, (4, D)) for off in (0, 4 * D + 8))]
    for order in ((0, 1, 2), (1, 2, 0), (2, 0, 1)):
        parts = [slices[i] for i in order]
        assert all(torch.equal(a, b) for a, b in zip(run([t.contiguous() for t in parts]), run(parts)))
    turned = heads.transpose(1, 2)  # three strides
    with pytest.raises(gdr.GdrError):
        gdr.gated_residual_rms_norm(turned, w)
    assert torch.equal(gdr.gated_residual_rms_norm(turned[0], w)[1], gdr.gated_residual_rms_norm(turned[0].contiguous(), w)[1])
