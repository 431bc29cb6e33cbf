"""The layer operators at sizes whose plans run what small sizes do not: long runs of the convolution, several rows a CTA
in the norm's backward, more scan CTAs than SMs, and segmented scans of every state size, aligned and not.  What a plan
comes to at 152 SMs stands beside the sizes.

References are 64-bit forms on the GPU (the scan's on the CPU).  Values that are sums over n tokens or rows of terms with
random signs, added one after another over at most ``depth`` of them, are off by at most (depth 2^-24 + 2^-19) of the sum
of magnitudes, sqrt(n) times the value's size and 4 for the largest of them."""
import pytest
import torch

import test_gpu_layer as G
from test_gpu_layer import DT, U, bounds, gdr, gen_of, rand  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

C = 2.0 ** -19


def summed(got, ref, n, depth, what):
    e = float((got.double() - ref).abs().max() / ref.square().mean().sqrt())
    assert e <= 4 * (depth * 2.0 ** -24 + C) * n ** 0.5, (what, e)


# ---- short convolution: runs of 32 tokens (forward), 64 (backward) -----------------------------------------------------

CONV = [  # B, T, D, W, lengths: channels a thread, columns of CTAs, blocks along the tokens
    (1, 7400, 2048, 4, None),                          # 4, 16, 29
    (1, 7400, 2048, 3, (33, 0, 2999, 1, 255, 4112)),   # 4, 16, 29
    (4, 1900, 2040, 2, None),                          # 4, 16, 8 a batch row
    (1, 3700, 2046, 4, (1, 2, 3, 3661, 33)),           # 2, 32, 15
    (1, 3700, 2046, 3, None),                          # 2, 32, 15
    (1, 1900, 1999, 4, (700, 1, 1, 1198)),             # 1, 63, 8
    (2, 1900, 999, 2, None),                           # 1, 32, 8 a batch row
]


def conv64(x, w, b, h0, lengths, silu):
    """The definition over whole sequences: windows of W inputs."""
    taps, out, at = w.shape[1], [], 0
    spans = [(i, 0, x.shape[1]) for i in range(x.shape[0])]
    if lengths is not None:
        spans = []
        for n in lengths:
            spans.append((0, at, n))
            at += n
    for i, (row, at, n) in enumerate(spans):
        if not n:
            continue
        pre = (torch.cat([h0[i], x[row, at:at + n]]).unfold(0, taps, 1) * w).sum(-1) + b
        out.append(pre * torch.sigmoid(pre) if silu else pre)
    return torch.cat(out).view(x.shape)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_in_long_runs(gdr, case, dt):  # noqa: F811
    B, T, D, W, lengths = case
    gen, t = gen_of(70), DT[dt]
    x, dy = rand(gen, B, T, D, dt=t), rand(gen, B, T, D, dt=t)
    w, b, h0 = rand(gen, D, W), rand(gen, D), rand(gen, len(lengths) if lengths else B, W - 1, D, dt=t)
    leaves = [v.requires_grad_() for v in (x, w, b, h0)]
    y, _ = gdr.short_conv(x, w, b, initial_state=h0, cu_seqlens=bounds(lengths))
    grads = torch.autograd.grad(y, leaves, dy)
    wide = [v.detach().double().requires_grad_() for v in leaves]
    ref = conv64(*wide, lengths, True)
    rg = torch.autograd.grad(ref, wide, dy.double())
    with torch.no_grad():
        mag = conv64(*(v.abs() for v in wide), lengths, False)
        assert ((y.double() - ref).abs() <= U[t] * ref.abs() + C * mag).all()
        for g, r, what in ((grads[0], rg[0], "dx"), (grads[3], rg[3], "dinit")):
            off = ((g.double() - r).abs() - U[t] * 1.01 * g.double().abs()).max() / r.square().mean().sqrt()
            assert float(off) <= 32 * C, what
        for g, r, what in ((grads[1], rg[1], "dw"), (grads[2], rg[2], "dbias")):
            summed(g, r, B * T, 64 + 4 + 32, what)


# ---- norm: several rows a CTA in the backward --------------------------------------------------------------------------

NORM = [  # M, D: CTAs
    (5000, 264), (5000, 263),    # 2432
    (2000, 2048), (1900, 2043),  # 912
    (700, 8192),                 # 152
    (700, 16384), (700, 16381),  # 152
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("added", [True, False])
@pytest.mark.parametrize("M,D", NORM)
def test_norm_backward_with_rows_in_turn(gdr, M, D, added, dt):  # noqa: F811
    gen, t = gen_of(71), DT[dt]
    x, w = rand(gen, M, D, dt=t), 1 + 0.1 * rand(gen, D)
    res = rand(gen, M, D, dt=t) if added else None
    dy, ds = rand(gen, M, D, dt=t), rand(gen, M, D, dt=t)
    leaves = [v.requires_grad_() for v in (x, w, res) if v is not None]
    y, r = gdr.residual_rms_norm(x, w, res)
    grads = torch.autograd.grad([y, r], leaves, [dy, ds])
    with torch.no_grad():
        h, g, w64 = r.double(), dy.double(), w.double()
        rstd = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6)
        hat = h * rstd
        assert ((y.double() - hat * w64).abs() <= (U[t] + C) * (hat * w64).abs()).all()
        back = rstd * (g * w64 - hat * (g * w64 * hat).mean(1, keepdim=True)) + ds.double()
        terms = rstd * ((g * w64).abs() + hat.abs() * (g * w64 * hat).abs().mean(1, keepdim=True)) + ds.double().abs()
        for d in [grads[0]] + ([grads[2]] if added else []):
            assert ((d.double() - back).abs() <= U[t] * back.abs() + C * terms).all()
        summed(grads[1], (g * hat).sum(0), M, 5 + 76 + 5, "dw")


# ---- scan --------------------------------------------------------------------------------------------------------------

BATCHED = [  # more CTAs than SMs, one segment (the forward with one group of helpers)
    (80, 70, 40, 1, 16), (80, 70, 37, 1, 16),  # 160 CTAs
    (80, 40, 72, 1, 8), (80, 40, 67, 1, 8),    # 160
    (40, 40, 64, 1, 32), (40, 40, 61, 1, 32),  # 160
    (20, 40, 64, 1, 64), (20, 40, 59, 1, 64),  # 160
    (40, 40, 64, 2, 16), (52, 40, 63, 3, 16),  # 80 + 80 (two groups), 156 (three)
]
SEGMENTED = [  # cut into segments, forward and backward
    (1, 1100, 40, 1, 16), (1, 1100, 37, 1, 16), (1, 1100, 72, 1, 8), (1, 1100, 67, 1, 8),
    (1, 1100, 40, 1, 32), (1, 1100, 37, 1, 32), (1, 1100, 24, 1, 64), (1, 1100, 21, 1, 64), (2, 900, 48, 2, 16),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", BATCHED, ids=str)
def test_scan_of_more_ctas_than_sms(gdr, case, dt):  # noqa: F811
    G.scan_check(gdr, (*case, None, True, True, True, True, True), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("case", SEGMENTED, ids=str)
def test_scan_in_segments(gdr, case, packed, dt):  # noqa: F811
    lengths = (321, 0, 1, 478, 300) if packed and case[0] == 1 else None
    if packed and lengths is None:
        pytest.skip("packed sequences have one batch row")
    G.scan_check(gdr, (*case, lengths, True, True, True, True, True), dt)


def test_the_cases_are_cut_as_said(gdr):  # noqa: F811
    import ctypes

    from gated_deltanet_chunked_delta_gb300 import layer as L
    for case in BATCHED + SEGMENTED:
        B, T, D, g, N = case
        for dtype in (0, 1):
            a = L._SsmArgs(B=B, T=T, D=D, G=g, N=N, n_seqs=B, dtype=dtype)
            cut = L._calls().gdr_ssm_fwd_workspace_size(ctypes.byref(a)) > 0
            assert cut == (case in SEGMENTED), case
