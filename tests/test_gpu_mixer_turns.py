"""The linear scan with several tiles a CTA and the norm's gradient with several rows a CTA, on varying data against 64-bit
forms: stages and buffers by turns, rows copied ahead, tiles that are dealt out and tiles that are taken from the counter,
weights' gradients summed over many rows, at every width of access.

Tolerances, set before the first run.  u is half a step of the output's type.

* recurrence, by ``err`` as in test_gpu_mixer.py: a step's decay is off by 2^-21, the rest by 2^-17.  Here the slow channels
  have s = 8 softplus(-5) = 0.054 and half-open gates, so that a state's terms are on average 37 tokens old, taken as
  64; the largest of some 10^6 elements over the rms (products of up to three normal variables) is covered by 128.
  The gradient of the decay is held, channel by channel, to the sum of G = dr / (1 - sigmoid(r)) of the kernel's own fp32 dr:
  a term's error is 2^-19 and that of 1 - sigmoid (2^-21 absolute), the sum's 2^-24 for each of the additions on its way
  (runs, warps, rows of partial sums, a tree).
* norm: gradients of elements by ``err``, 128 x 2^-17; the weights', channel by channel with the sum of the terms' magnitudes:
  a term is off by 2^-16 of its parts, the sum by 2^-24 for each addition on its way, fewer than 128.
"""
import itertools

import pytest
import torch

import mixer_plain as M
from layer_plain import spans
from test_gpu_layer import DT, U, bounds, gdr, gen_of, rand  # noqa: F401  (the fixture)

gpu = pytest.mark.gpu


def linear(x, input_gate, decay_gate, decay, z=None, h0=None, lengths=None, scale=8.0):
    """mixer_plain.linear for long sequences: batch rows together, every token taken out of its tensor once."""
    B, T, D = x.shape
    log_a = -scale * torch.nn.functional.softplus(decay, threshold=1e9) * torch.sigmoid(decay_gate)
    a = torch.exp(log_a).unbind(1)
    add = (torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(input_gate) * x).unbind(1)
    rows, finals = [], []
    for i, (_, at, n) in enumerate(spans(1, T, lengths)):
        h = x.new_zeros(B, D) if h0 is None else h0 if lengths is None else h0[i:i + 1]
        for t in range(at, at + n):
            h = a[t] * h + add[t]
            rows.append(h)
        finals.append(h)
    y = torch.stack(rows, 1)
    return y if z is None else y * M.silu(z), torch.cat(finals)


@pytest.mark.parametrize("B,T,lengths", [(2, 13, None), (1, 17, (5, 0, 1, 11, 0))])
def test_the_long_form_is_the_plain_one(B, T, lengths):
    gen = torch.Generator().manual_seed(3)
    n = len(lengths) if lengths else B
    v = [torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((B, T, 4),) * 3 + ((4,), (B, T, 4), (n, 4))]
    for a, b in zip(linear(*v, lengths), M.linear(*v, lengths)):
        assert torch.allclose(a, b, rtol=1e-13, atol=1e-13)


def d64(t, grad=False):
    return None if t is None else t.detach().double().requires_grad_(grad)


def held(got, want, tol, what):
    """max (|x - ref| - u |x|) / rms(ref), on the GPU."""
    got, want = got.detach(), want.detach()
    x = got.double()
    e = float(((x - want).abs() - U[got.dtype] * x.abs()).max() / want.square().mean().sqrt())
    assert e <= tol, (what, e, tol)


SCANS = [  # B, T, D, lengths, h0, gate: tiles of 64 channels x 96 tokens, in the backward 48, against 152 CTAs of full chunks
    (2, 2000, 1024, None, True, False),    # 672 and 1344 tiles; vectors
    (3, 1500, 1031, None, False, True),    # 816 and 1632; bf16 halves of words, fp32 words
    (1, 2500, 1026, (700, 1, 0, 799, 1000), True, True),  # 459 and 901, packed; words
    (1, 3100, 1024, (96, 48, 960, 1996), True, False),    # packed, sequences that end with chunks
    (1, 2100, 1031, (1,) * 60 + (2040,), False, True),
    (700, 7, 130, None, True, True),       # 2100 tiles of one chunk: dealt out
    (300, 44, 136, None, True, False),     # the same of six and eleven warps
    (90, 90, 320, None, False, True),      # 450 tiles of one chunk forward, 900 of two backward
    (1, 44, 30000, (10, 0, 30, 4), True, True),  # 469 packed tiles of one chunk
]


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", SCANS, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}{'-packed' if c[3] else ''}")
def test_scans_of_several_tiles_a_cta(gdr, case, dt):  # noqa: F811
    B, T, D, lengths, has_h0, gate = case
    gen, t = gen_of(111), DT[dt]
    n = len(lengths) if lengths else B
    decay = torch.full((D,), -5.0, device="cuda")  # whole tiles of slow channels, then slow and fast ones by turns
    decay[D // 2::2] = rand(gen, D - D // 2)[::2] - 1
    v = dict(x=rand(gen, B, T, D, dt=t), input_gate=rand(gen, B, T, D, dt=t), decay_gate=rand(gen, B, T, D, dt=t), decay=decay,
             z=rand(gen, B, T, D, dt=t) if gate else None, initial_state=rand(gen, n, D) if has_h0 else None)
    dy, dht = rand(gen, B, T, D, dt=t), rand(gen, n, D)
    names = [k for k in v if v[k] is not None]
    for k in names:
        v[k].requires_grad_()
    y, ht = gdr.gated_linear_scan(**v, output_final_state=True, cu_seqlens=bounds(lengths))
    grads = dict(zip(names, torch.autograd.grad([y, ht], [v[k] for k in names], [dy, dht])))
    gdr.check_status()
    p = {k: d64(w, True) for k, w in v.items() if w is not None}
    h0 = p.pop("initial_state", None)
    ry, rht = linear(**p, h0=h0, lengths=lengths)
    if h0 is not None:
        p["initial_state"] = h0
    want = dict(zip(names, torch.autograd.grad([ry, rht], [p[k] for k in names], [d64(dy), d64(dht)])))
    tol = 128 * (64 * 2.0 ** -21 + 2.0 ** -17)
    held(y, ry, tol, "y")
    held(ht, rht, tol, "final")
    for k in names:
        if k != "decay":
            held(grads[k], want[k], tol, k)
    if dt == "f32":
        d, rest = d64(decay), 1 - torch.sigmoid(p["decay_gate"].detach())
        ratio = torch.sigmoid(d) / torch.nn.functional.softplus(d)
        G = grads["decay_gate"].double() / rest
        adds = 4 + 12 + B * -(-T // 44) / 32 + 8
        bound = ratio * (G.abs() * (2.0 ** -19 + 2.0 ** -21 / rest + adds * 2.0 ** -24)).sum((0, 1))
        assert ((grads["decay"].double() - ratio * G.sum((0, 1))).abs() <= bound).all()
    with torch.no_grad():  # without a gradient the same bits
        y2, ht2 = gdr.gated_linear_scan(**v, output_final_state=True, cu_seqlens=bounds(lengths))
        assert torch.equal(y, y2) and torch.equal(ht, ht2)


# More rows than 152 SMs take at once, and a last round that is not full.
ROWS = [(40000, 128), (39000, 72), (20000, 200), (9001, 101), (7000, 264), (6000, 512), (5000, 390), (3001, 1024), (2500, 1001), (1501, 4096),
        (700, 5003), (800, 8192), (700, 8200), (500, 16384), (400, 9001)]
EPS = 1e-5


def norm_check(gdr, x, w, gate, res, w2, dy, dr, scale):  # noqa: F811
    """Gradients through both outputs or (dy or dr None) one."""
    leaves = [v.requires_grad_() for v in (x, w, gate, res, w2) if v is not None]
    y, r = gdr.gated_residual_rms_norm(x, w, gate, res, w2, scale=scale, eps=EPS)
    pairs = [(o, g) for o, g in ((y, dy), (r, dr)) if o is not None and g is not None]
    grads = iter(torch.autograd.grad([o for o, _ in pairs], leaves, [g for _, g in pairs], allow_unused=True))
    dx, dw, dgate, dres, dw2 = (None if v is None else next(grads) for v in (x, w, gate, res, w2))
    px, pw, pg, ps, pn = plain = [d64(v, True) for v in (x, w, gate, res, w2)]
    ry, rr = M.block_norm(*plain, scale, EPS)
    for o, ref in ((y, ry), (r, rr)):
        if o is not None:
            held(o, ref, 128 * 2.0 ** -17, "out")
    given = [(o, g) for o, g in ((ry, dy), (rr, dr)) if o is not None and g is not None]
    back = iter(torch.autograd.grad([o for o, _ in given], [v for v in plain if v is not None], [d64(g) for _, g in given], allow_unused=True))
    rdx, rdw, rdgate, rdres, rdw2 = (None if v is None else next(back) for v in plain)
    for name, g, ref in (("x", dx, rdx), ("gate", dgate, rdgate), ("residual", dres, rdres)):
        if g is not None:
            held(g, ref, 128 * 2.0 ** -17, name)
    with torch.no_grad():
        hat = px / torch.sqrt(px.square().mean(-1, keepdim=True) + EPS)
        on = hat if gate is None else hat * M.silu(pg)
        mag_r = (scale * on * pw).abs() + (0 if res is None else ps.abs())
        mag = torch.zeros_like(px) if dr is None else d64(dr).abs()
        if w2 is not None and dy is not None:
            inv = 1 / torch.sqrt(rr.square().mean(-1, keepdim=True) + EPS)
            f = (d64(dy) * pn).abs()
            mag = mag + inv * f + inv ** 3 * (f * mag_r).mean(-1, keepdim=True) * mag_r
            bound = (d64(dy).abs() * mag_r * inv).flatten(0, -2).sum(0) * (2.0 ** -16 + 128 * 2.0 ** -24)
            assert ((dw2.double() - rdw2).abs() <= bound).all()
        bound = (abs(scale) * mag * on.abs()).flatten(0, -2).sum(0) * (2.0 ** -16 + 128 * 2.0 ** -24)
        assert ((dw.double() - rdw).abs() <= bound).all()


def norm_inputs(rows, D, parts, t, seed=112):
    gen, (gated, added, after) = gen_of(seed), parts
    some = lambda on: rand(gen, rows, D, dt=t) if on else None  # noqa: E731
    return ((2 * rand(gen, rows, D)).to(t), 1 + 0.1 * rand(gen, D), some(gated), some(added), 1 + 0.1 * rand(gen, D) if after else None,
            some(after), some(True))


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", ROWS)
def test_norm_gradients_of_several_rows_a_cta(gdr, rows, D, dt):  # noqa: F811
    norm_check(gdr, *norm_inputs(rows, D, (True, True, True), DT[dt]), 0.7)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("parts", list(itertools.product([True, False], repeat=3)), ids=str)
@pytest.mark.parametrize("rows,D", [(20000, 128), (9001, 101), (3000, 1000), (1000, 4096), (500, 8208)])
def test_parts_of_several_rows_a_cta(gdr, rows, D, parts, dt):  # noqa: F811
    norm_check(gdr, *norm_inputs(rows, D, parts, DT[dt]), -1.3)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("rows,D", [(20000, 128), (7000, 264), (1000, 4096), (2500, 1001)])
def test_one_output_of_several_rows_a_cta(gdr, rows, D, which, dt):  # noqa: F811
    x, w, gate, res, w2, dy, dr = norm_inputs(rows, D, (True, True, True), DT[dt])
    norm_check(gdr, x, w, gate, res, w2, dy if which == 0 else None, dr if which == 1 else None, 0.7)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,heads,D,off", [(3001, 7, 128, 8), (2501, 4, 200, 8), (2501, 4, 200, 3), (900, 8, 264, 0), (701, 5, 1024, 8), (701, 5, 999, 1),
                                                (301, 5, 4096, 8)])
def test_heads_of_slices_of_several_rows_a_cta(gdr, tokens, heads, D, off, dt):  # noqa: F811
    """Heads read in place from a projection: a stride for tokens and one for heads; the same bits as from copies where both are read in
    vectors, and the 64-bit form."""
    gen, t = gen_of(113), DT[dt]
    wide = rand(gen, tokens, 3 * heads * D + 16, dt=t)
    x, gate, res = (wide[:, off + i * heads * D:off + (i + 1) * heads * D].unflatten(-1, (heads, D)) for i in range(3))
    w, w2 = 1 + 0.1 * rand(gen, D), 1 + 0.1 * rand(gen, D)
    dy, dr = (rand(gen, tokens, heads, D, dt=t) for _ in range(2))
    norm_check(gdr, x, w, gate, res, w2, dy, dr, 0.7)
    if D % 8 == 0 and off % 8 == 0:
        def run(*parts):
            leaves = [v.detach().requires_grad_() for v in (*parts, w, w2)]
            y, r = gdr.gated_residual_rms_norm(leaves[0], leaves[3], leaves[1], leaves[2], leaves[4], scale=0.7)
            return (y.detach(), r.detach(), *torch.autograd.grad([y, r], leaves, [dy, dr]))
        assert all(torch.equal(a, b) for a, b in zip(run(x, gate, res), run(*(v.contiguous() for v in (x, gate, res)))))
