"""The norm of rows shorter than a piece of eight channels, where pieces reach over several rows and the tensor's ends.

Per-element bound: half a step of the output's type, and 2^-19 of the terms' magnitudes (at most sixteen fp32
operations of 2^-24 each on any of them)."""
import pytest
import torch

import layer_plain as P
from test_gpu_layer import DT, U, gdr, gen_of, rand  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("added", [True, False])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 6, 7, 9])
@pytest.mark.parametrize("M", [1, 2, 11])
def test_norm_of_short_rows(gdr, M, D, added, dt):  # noqa: F811
    gen, t = gen_of(100 * M + D), DT[dt]
    x, w = rand(gen, M, D, dt=t), 1 + 0.1 * rand(gen, D)
    res = rand(gen, M, D, dt=t) if added else None
    dy, ds = rand(gen, M, D, dt=t), rand(gen, M, D, dt=t)
    leaves = [v.requires_grad_() for v in (x, w, res) if v is not None]
    y, r = gdr.residual_rms_norm(x, w, res)
    grads = torch.autograd.grad([y, r], leaves, [dy, ds])
    with torch.no_grad():
        q, scales, r8 = gdr.residual_rms_norm_fp8(x, w, res)
        assert torch.equal(r, (x.float() + res.float()).to(t) if added else x) and torch.equal(r, r8)
    pr, pw = P.f64(r, True), P.f64(w, True)
    ref = P.norm(pr, pw)
    rdr, rdw = torch.autograd.grad([ref, pr], [pr, pw], [P.f64(dy), P.f64(ds)])
    with torch.no_grad():
        rstd = 1 / torch.sqrt((pr * pr).mean(1, keepdim=True) + 1e-6)
        wdy, hat = (P.f64(dy) * pw).abs(), (pr * rstd).abs()
        c, u = 2.0 ** -19, U[t]
        assert ((P.f64(y) - ref).abs() <= (u + c) * ref.abs()).all()
        terms = rstd * (wdy + hat * (wdy * hat).mean(1, keepdim=True)) + P.f64(ds).abs()
        for g in [grads[0]] + ([grads[2]] if added else []):
            assert ((P.f64(g) - rdr).abs() <= u * rdr.abs() + c * terms).all()
        assert ((P.f64(grads[1]) - rdw).abs() <= c * (P.f64(dy).abs() * hat).sum(0)).all()
        top = ref.abs().amax(1).clamp_min(1e-30) / 448
        assert ((P.f64(scales[0]) - top).abs() <= c * top).all()
        off = (P.f64(q.float()) * P.f64(scales[0])[:, None] - ref).abs()
        assert (off <= torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * top[:, None]) * (1 + c) + c * ref.abs()).all()
