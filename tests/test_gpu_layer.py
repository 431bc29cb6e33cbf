"""The layer operators on the GPU against the plain 64-bit forms, at the sizes
and masks where they can go wrong.

Tolerances, set before the first run.  u is half a step of the output's type
(bf16 2^-8, fp32 2^-24; e4m3 2^-4).  Per-element bounds are u |ref| + c S with
S the sum of the terms' magnitudes:

* convolution: five fused fp32 operations (2^-24 each) and silu (ex2.approx
  2^-22, rcp.approx 2^-23, its argument's rounding |pre| 2^-23): c = 2^-19;
* norm: a sum of D squares in trees of at most 32 sequential adds: 2^-19 of y;
* product: four MMAs a block whose fp32 accumulators keep at least 22 bits, then
  one rounding a block: c = 2^-20.

The scan's relative error grows by 2^-21 a token (ex2.approx, two roundings) and
2^-17 in all (softplus, sums over N, silu).  Scan outputs and every gradient are
held by ``err`` = max (|x - ref| - u |x|) / rms(ref); 32 covers the largest
element over the rms and the terms' magnitudes over their sum.
"""
import pytest
import torch

import layer_plain as P
from parity import err

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_chunked_delta_gb300 as gdr
    gdr.load(build_if_missing=True)
    yield gdr
    torch.cuda.synchronize()
    gdr.check_status()


def rand(gen, *s, dt=torch.float32):
    return torch.randn(*s, generator=gen, device="cuda").to(dt)


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def bounds(lengths):
    if lengths is None:
        return None
    return torch.tensor([0] + list(lengths), dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)


def close(x, ref, tol, key):
    if ref.numel() == 0:
        assert x.numel() == 0
        return
    e = err(x.detach(), ref.detach().numpy(), key)
    assert e <= tol, (key, e, tol)


# ---- short convolution ------------------------------------------------------

CONV = [  # B, T, D, W, lengths, h0, bias, silu
    (1, 1, 8, 4, None, False, True, True), (2, 130, 64, 4, None, True, True, True), (3, 37, 264, 3, None, False, False, True),
    (1, 300, 37, 2, None, True, True, False), (2, 5, 1, 4, None, True, False, True),
    (1, 140, 48, 4, (0, 3, 1, 0, 64, 2, 70, 0), True, True, True), (1, 521, 16, 4, (129, 1, 1, 1, 262, 127), True, True, True),
    (1, 77, 30, 3, (76, 1), False, True, True), (1, 4, 8, 4, (0, 0, 4, 0, 0), True, True, True),
    (1, 2050, 256, 4, (1024, 1026), True, True, True)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv(gdr, case, dt):
    B, T, D, W, lengths, has_h0, has_bias, silu = case
    gen, t = gen_of(3), DT[dt]
    n = len(lengths) if lengths else B
    x, dy = rand(gen, B, T, D, dt=t), rand(gen, B, T, D, dt=t)
    w, b = rand(gen, D, W), rand(gen, D) if has_bias else None
    h0 = rand(gen, n, W - 1, D, dt=t) if has_h0 else None
    dht = rand(gen, n, W - 1, D, dt=t)
    leaves = [v.requires_grad_() for v in (x, w, b, h0) if v is not None]
    y, ht = gdr.short_conv(x, w, b, activation="silu" if silu else None, initial_state=h0, output_final_state=True,
                           cu_seqlens=bounds(lengths))
    grads = torch.autograd.grad([y, ht], leaves, [dy, dht])
    plain = [P.f64(v, True) for v in (x, w, b, h0)]
    ry, rht = P.conv(*plain[:3], silu, plain[3], lengths)
    with torch.no_grad():
        mag, _ = P.conv(*(None if v is None else v.abs() for v in plain[:3]), False, None if h0 is None else plain[3].abs(), lengths)
        assert ((P.f64(y) - ry).abs() <= U[t] * ry.abs() + 2.0 ** -19 * mag + 1e-30).all()
        assert torch.equal(P.f64(ht), rht)
    rg = torch.autograd.grad([ry, rht], [v for v in plain if v is not None], [P.f64(dy), P.f64(dht)])
    for g, r, v in zip(grads, rg, leaves):
        close(g, r, 32 * (2.0 ** -19 + T * B * 2.0 ** -24), str(tuple(v.shape)))
    # without a gradient the same kernel gives the same bits; a call from a saved state continues the sequence
    with torch.no_grad():
        y2, _ = gdr.short_conv(x, w, b, activation="silu" if silu else None, initial_state=h0, cu_seqlens=bounds(lengths))
        assert torch.equal(y, y2)
        if lengths is None and T > 1:
            cut = T // 2
            a1, s1 = gdr.short_conv(x[:, :cut], w, b, "silu" if silu else None, h0, True)
            a2, s2 = gdr.short_conv(x[:, cut:], w, b, "silu" if silu else None, s1, True)
            assert torch.equal(torch.cat([a1, a2], 1), y) and torch.equal(s2, ht)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D,W,S", [(1, 8, 4, 1), (5, 37, 3, 9), (64, 256, 4, 64), (3, 1032, 2, 4)])
def test_conv_step(gdr, rows, D, W, S, dt):
    gen, t = gen_of(4), DT[dt]
    x, w, b = rand(gen, rows, D, dt=t), rand(gen, D, W), rand(gen, D)
    state = rand(gen, S, W - 1, D, dt=t)
    slots = torch.randperm(S, generator=gen, device="cuda")[:rows].to(torch.int32)
    if rows > 2:
        slots[1] = -1
    was = state.clone()
    y = gdr.short_conv_step(x, w, state, b, slots=slots)
    expect = P.f64(was)
    for r, s in enumerate(slots.tolist()):
        if s < 0:
            assert not y[r].any()
            continue
        ry, rs = P.conv(P.f64(x[r])[None, None], P.f64(w), P.f64(b), True, P.f64(was[s])[None])
        mag, _ = P.conv(P.f64(x[r]).abs()[None, None], P.f64(w).abs(), P.f64(b).abs(), False, P.f64(was[s]).abs()[None])
        assert ((P.f64(y[r]) - ry[0, 0]).abs() <= U[t] * ry[0, 0].abs() + 2.0 ** -19 * mag[0, 0]).all()
        expect[s] = rs[0]
    assert torch.equal(P.f64(state), expect)


def test_conv_reads_slices(gdr):
    gen = gen_of(5)
    big = rand(gen, 2, 50, 200, dt=torch.bfloat16)
    w = rand(gen, 64, 4)
    for off in (0, 8, 3):  # aligned and not
        x = big[:, :, off:off + 64]
        assert torch.equal(gdr.short_conv(x, w)[0], gdr.short_conv(x.contiguous(), w)[0])
        tr = x.transpose(0, 1).contiguous().transpose(0, 1)  # tokens outside the batch
        assert torch.equal(gdr.short_conv(tr, w)[0], gdr.short_conv(x.contiguous(), w)[0])


# ---- scan --------------------------------------------------------------------

SCAN = [  # B, T, D, G, N, lengths, h0, gate, skip, bias, softplus
    (1, 1, 8, 1, 16, None, False, True, True, True, True), (2, 67, 40, 1, 16, None, True, True, True, True, True),
    (1, 200, 37, 1, 16, None, True, True, True, True, True), (2, 33, 24, 3, 8, None, False, True, True, True, True),
    (1, 48, 16, 2, 32, None, True, False, True, False, True), (1, 31, 8, 1, 64, None, True, True, False, True, True),
    (1, 300, 96, 2, 16, None, True, True, True, True, True), (1, 40, 32, 1, 16, None, True, False, False, False, False),
    (1, 171, 40, 1, 16, (0, 3, 1, 0, 64, 32, 71, 0), True, True, True, True, True),
    (1, 260, 33, 1, 8, (129, 1, 1, 129), True, True, True, True, True), (1, 5, 8, 1, 16, (0, 0, 5, 0), True, True, True, True, True),
    (1, 450, 8, 1, 16, (31, 33, 190, 196), True, True, True, True, True)]


def scan_inputs(case, dt, seed=7):
    B, T, D, G, N, lengths, has_h0, gate, skip, bias, softplus = case
    gen, t = gen_of(seed), DT[dt]
    n = len(lengths) if lengths else B
    x, z = rand(gen, B, T, D, dt=t), rand(gen, B, T, D, dt=t) if gate else None
    step = rand(gen, B, T, D)
    step = (step - 1.5 if softplus else 0.2 * step.abs()).to(t)
    A = -0.2 - 1.5 * torch.rand(D, N, generator=gen, device="cuda")
    Bm, Cm = rand(gen, B, T, G, N, dt=t), rand(gen, B, T, G, N, dt=t)
    return dict(x=x, dt=step, A=A, B=Bm, C=Cm, D=rand(gen, D) if skip else None, z=z, dt_bias=0.3 * rand(gen, D) if bias else None,
                initial_state=rand(gen, n, D, N) if has_h0 else None), rand(gen, B, T, D, dt=t), rand(gen, n, D, N)


def scan_check(gdr, case, dt):
    lengths, softplus = case[5], case[10]
    v, dy, dht = scan_inputs(case, dt)
    names = [k for k in v if v[k] is not None]
    for k in names:
        v[k].requires_grad_()
    y, ht = gdr.state_space_scan(**v, dt_softplus=softplus, output_final_state=True, cu_seqlens=bounds(lengths))
    grads = torch.autograd.grad([y, ht], [v[k] for k in names], [dy, dht])
    p = {k: P.f64(v[k], True) for k in v}
    h0 = p.pop("initial_state")
    ry, rht = P.scan(**p, softplus=softplus, h0=h0, lengths=lengths)
    p["initial_state"] = h0
    rg = torch.autograd.grad([ry, rht], [p[k] for k in names], [P.f64(dy), P.f64(dht)])
    T = case[1]
    tol = 32 * (T * 2.0 ** -21 + 2.0 ** -17)
    close(y, ry, tol, "y")
    close(ht, rht, tol, "final")
    for k, g, r in zip(names, grads, rg):
        close(g, r, tol, k)
    with torch.no_grad():
        y2, ht2 = gdr.state_space_scan(**v, dt_softplus=softplus, output_final_state=True, cu_seqlens=bounds(lengths))
        assert torch.equal(y, y2) and torch.equal(ht, ht2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan(gdr, case, dt):
    scan_check(gdr, case, dt)


def test_scan_gradients_do_not_change_between_runs(gdr):
    v, dy, _ = scan_inputs((1, 900, 72, 1, 16, None, False, True, True, True, True), "bf16")
    names = [k for k in v if v[k] is not None]
    for k in names:
        v[k].requires_grad_()
    runs = [torch.autograd.grad(gdr.state_space_scan(**v)[0], [v[k] for k in names], dy) for _ in range(2)]
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_scan_only_final_state_in_the_loss(gdr):
    case = (2, 50, 16, 1, 16, None, True, True, True, True, True)
    v, _, dht = scan_inputs(case, "f32")
    for k in v:
        v[k].requires_grad_()
    _, ht = gdr.state_space_scan(**v, output_final_state=True)
    got = torch.autograd.grad(ht, [v["x"], v["initial_state"]], dht)
    p = {k: P.f64(v[k], True) for k in v}
    h0 = p.pop("initial_state")
    want = torch.autograd.grad(P.scan(**p, h0=h0)[1], [p["x"], h0], P.f64(dht))
    for g, r in zip(got, want):
        close(g, r, 32 * (50 * 2.0 ** -21 + 2.0 ** -17), "grad")


def test_scan_reads_slices(gdr):
    v, _, _ = scan_inputs((2, 40, 32, 2, 16, None, True, True, True, True, True), "bf16")
    want = gdr.state_space_scan(**v)[0]
    for off in (0, 8, 5):
        big = torch.zeros(2, 40, 32 * 3 + 64 * 2 + 16, dtype=torch.bfloat16, device="cuda")
        at, s = off, dict(v)
        for k in ("x", "dt", "z"):
            big[:, :, at:at + 32] = v[k]
            s[k] = big[:, :, at:at + 32]
            at += 32
        for k in ("B", "C"):
            big[:, :, at:at + 32] = v[k].flatten(2)
            s[k] = big[:, :, at:at + 32].unflatten(2, (2, 16))
            at += 32
        assert torch.equal(gdr.state_space_scan(**s)[0], want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D,G,N,S", [(1, 8, 1, 16, 1), (6, 37, 1, 16, 9), (3, 24, 2, 8, 3), (4, 20, 1, 32, 7), (2, 9, 1, 64, 2)])
def test_scan_step(gdr, rows, D, G, N, S, dt):
    v, _, _ = scan_inputs((rows, 1, D, G, N, None, False, True, True, True, True), dt)
    v.pop("initial_state")
    gen = gen_of(9)
    state = rand(gen, S, D, N)
    slots = torch.randperm(S, generator=gen, device="cuda")[:rows].to(torch.int32)
    if rows > 2:
        slots[2] = -3
    was = state.clone()
    one = {k: (t[:, 0] if k in ("x", "dt", "B", "C", "z") else t) for k, t in v.items()}
    y = gdr.state_space_step(**one, state=state, slots=slots)
    expect = P.f64(was)
    live = [r for r, s in enumerate(slots.tolist()) if s >= 0]
    at = slots[live].long()
    p = {k: P.f64(t) for k, t in v.items()}
    for k in ("x", "dt", "B", "C", "z"):
        p[k] = p[k][live]
    ry, rh = P.scan(**p, h0=P.f64(was[at]))
    close(y[live], ry[:, 0], 32 * (2.0 ** -21 + 2.0 ** -17), "y")
    expect[at.cpu()] = rh
    close(state, expect, 32 * (2.0 ** -21 + 2.0 ** -17), "state")
    idle = [s for s in range(S) if s not in at.tolist()]
    assert torch.equal(state[idle], was[idle])
    if rows > 2:
        assert not y[2].any()


def test_steps_continue_a_prompt(gdr):
    """A prompt and then tokens one by one give what the whole sequence gives."""
    v, _, _ = scan_inputs((2, 45, 24, 1, 16, None, True, True, True, True, True), "f32")
    whole, end = gdr.state_space_scan(**v, output_final_state=True)
    cut = {k: (t[:, :40] if k in ("x", "dt", "B", "C", "z") else t) for k, t in v.items()}
    _, state = gdr.state_space_scan(**cut, output_final_state=True)
    v.pop("initial_state")
    for t in range(40, 45):
        y = gdr.state_space_step(**{k: (a[:, t] if k in ("x", "dt", "B", "C", "z") else a) for k, a in v.items()}, state=state)
        close(y, P.f64(whole[:, t]), 64 * (45 * 2.0 ** -21 + 2.0 ** -17), "y")
    close(state, P.f64(end), 64 * (45 * 2.0 ** -21 + 2.0 ** -17), "state")


def test_scan_keeps_nan_where_it_is(gdr):
    v, _, _ = scan_inputs((1, 64, 16, 1, 16, (30, 34), False, True, True, True, True), "f32")
    v["x"][0, 10, 3] = float("nan")
    v["dt"][0, 40, 5] = float("inf")
    y, ht = gdr.state_space_scan(**v, output_final_state=True, cu_seqlens=bounds((30, 34)))
    bad = torch.isnan(y[0])
    assert bad[10:30, 3].all() and not bad[:10].any() and not bad[30:, 3].any()
    assert not bad[:, :3].any() and not bad[:40, 5].any()


# ---- norm --------------------------------------------------------------------

NORM = [(1, 8), (3, 37), (5, 128), (2, 1000), (7, 2048), (3, 4096), (2, 5003), (2, 16384), (700, 264), (2, 12345)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("added", [True, False])
@pytest.mark.parametrize("M,D", NORM)
def test_norm(gdr, M, D, added, dt):
    gen, t = gen_of(11), DT[dt]
    x, w = rand(gen, M, D, dt=t), 1 + 0.1 * rand(gen, D)
    res = rand(gen, M, D, dt=t) if added else None
    dy, ds = rand(gen, M, D, dt=t), rand(gen, M, D, dt=t)
    leaves = [v.requires_grad_() for v in (x, w, res) if v is not None]
    y, r = gdr.residual_rms_norm(x, w, res)
    with torch.no_grad():
        assert torch.equal(r, (x.float() + res.float()).to(t) if added else x)
    grads = torch.autograd.grad([y, r], leaves, [dy, ds], allow_unused=True)
    pr, pw = P.f64(r, True), P.f64(w, True)
    ref = P.norm(pr, pw)
    rdr, rdw = torch.autograd.grad([ref, pr], [pr, pw], [P.f64(dy), P.f64(ds)])
    with torch.no_grad():
        assert ((P.f64(y) - ref).abs() <= (U[t] + 2.0 ** -19) * ref.abs() + 1e-30).all()
    tol = 32 * (2.0 ** -19 + M * 2.0 ** -24)
    close(grads[0], rdr, tol, "dx")
    close(grads[1], rdw, tol, "dw")
    if added:
        close(grads[2], rdr, tol, "dres")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("added", [True, False])
@pytest.mark.parametrize("M,D", NORM)
def test_norm_fp8(gdr, M, D, added, dt):
    gen, t = gen_of(12), DT[dt]
    x, w = rand(gen, M, D, dt=t), 1 + 0.1 * rand(gen, D)
    res = rand(gen, M, D, dt=t) if added else None
    x[0, : D // 2] = 0
    if added:
        res[0, : D // 2] = 0
    q, scales, r = gdr.residual_rms_norm_fp8(x, w, res)
    assert q.dtype == torch.float8_e4m3fn and scales.shape == (-(-D // 128), M)
    assert torch.equal(r, (x.float() + res.float()).to(t) if added else x)
    ref = P.norm(P.f64(r), P.f64(w))
    wide = torch.zeros(M, scales.shape[0] * 128, dtype=torch.float64)
    wide[:, :D] = ref
    top = wide.abs().view(M, -1, 128).amax(2).clamp_min(1e-30) / 448
    assert ((P.f64(scales).t() - top).abs() <= 2.0 ** -18 * top).all()
    spread = top.repeat_interleave(128, 1)[:, :D]
    off = (P.f64(q.float()) * P.f64(scales).t().repeat_interleave(128, 1)[:, :D] - ref).abs()
    assert (off <= torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * spread) * (1 + 2.0 ** -17) + 2.0 ** -17 * ref.abs()).all()


def test_norm_of_strided_rows_and_of_no_rows(gdr):
    gen = gen_of(13)
    big = rand(gen, 9, 300, dt=torch.bfloat16)
    w = rand(gen, 128)
    for off in (0, 8, 1):
        x = big[:, off:off + 128]
        assert torch.equal(gdr.residual_rms_norm(x, w)[0], gdr.residual_rms_norm(x.contiguous(), w)[0])
    y, r = gdr.residual_rms_norm(big[:0, :128], w, big[:0, 128:256])
    assert y.shape == r.shape == (0, 128)
    q, s, _ = gdr.residual_rms_norm_fp8(big[:0, :128], w)
    assert q.shape == (0, 128) and s.shape == (1, 0)


def test_norm_of_rows_with_nan_inf_and_zeros(gdr):
    x = torch.ones(4, 256, device="cuda")
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    x[3] = 0
    w = torch.ones(256, device="cuda")
    y, _ = gdr.residual_rms_norm(x, w)
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1]).all() and torch.isnan(y[2, 9]) and not y[2, :9].any() and not y[3].any()
    q, s, _ = gdr.residual_rms_norm_fp8(x, w)
    assert torch.isnan(q[1].float()).all() and torch.isnan(s[:, 1]).all() and not q[3].float().any() and torch.isnan(s[0, 2])


# ---- block-scaled product ----------------------------------------------------


def operands(gen, M, N, K):
    a = (rand(gen, M, K) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    b = (rand(gen, N, K) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    sa = torch.rand(-(-K // 128), M, generator=gen, device="cuda") + 0.01
    sb = torch.rand(-(-N // 128), -(-K // 128), generator=gen, device="cuda") + 0.01
    return a, sa, b, sb


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 128, 128), (3, 200, 144), (16, 1000, 512), (17, 256, 2064), (33, 77, 4096), (64, 640, 1024),
                                   (65, 128, 256), (100, 129, 272), (128, 512, 2048), (129, 1031, 384), (300, 2048, 1024), (511, 4096, 128),
                                   (1000, 8200, 160), (2300, 5000, 128)])
def test_matmul(gdr, M, N, K, out):
    a, sa, b, sb = operands(gen_of(M + N + K), M, N, K)
    got = gdr.block_matmul_fp8(a, sa, b, sb, out_dtype=DT[out])
    torch.cuda.synchronize()
    gdr.check_status()
    ref, mag = P.matmul(a, sa, b, sb)
    off = (P.f64(got) - ref).abs()
    assert (off <= U[DT[out]] * ref.abs() + 2.0 ** -20 * mag).all(), float((off / mag).max())


def test_matmul_of_no_rows(gdr):
    a, sa, b, sb = operands(gen_of(1), 4, 64, 128)
    assert gdr.block_matmul_fp8(a[:0], sa[:, :0], b, sb).shape == (0, 64)


def test_matmul_does_not_read_past_its_operands(gdr):
    """Rows beside the operands hold NaN: a padded tile must not take them in."""
    M, N, K = 5, 130, 160
    a, sa, b, sb = operands(gen_of(2), M, N, K)
    want = gdr.block_matmul_fp8(a, sa, b, sb)
    big = torch.full((M + 128, K), float("nan"), device="cuda").to(torch.float8_e4m3fn)
    big[:M] = a
    wide = torch.full((N + 256, K), float("nan"), device="cuda").to(torch.float8_e4m3fn)
    wide[:N] = b
    assert torch.equal(gdr.block_matmul_fp8(big[:M], sa, wide[:N], sb), want)


def test_gradients_against_differences(gdr):
    """Along each gradient, with steps h of a hundredth of the parameter's norm and of half that: a central difference
    D(h) is off by c h^2 + O(h^4) (c is large for A, whose gradient lies in the few slowly decaying states), so
    (4 D(h / 2) - D(h)) / 3 is off by O(h^4); the forward's rounding (2^-17 against a change of the loss of about a
    hundredth) gives 1e-3: 2e-2 holds both."""
    v, dy, _ = scan_inputs((1, 100, 32, 1, 16, None, False, True, True, True, True), "f32")
    v.pop("initial_state")
    gen = gen_of(30)
    v["w"], v["b"], v["n"] = 0.5 * rand(gen, 32, 4), rand(gen, 32), 1 + 0.1 * rand(gen, 32)

    def loss(p):
        x, _ = gdr.short_conv(p["x"], p["w"], p["b"])
        y, _ = gdr.state_space_scan(x, *(p[k] for k in ("dt", "A", "B", "C", "D", "z", "dt_bias")))
        y, r = gdr.residual_rms_norm(y, p["n"], p["x"])
        return (y.double() * dy).sum() + (r.double() * dy).sum()

    leaves = {k: t.detach().requires_grad_() for k, t in v.items()}
    grads = dict(zip(leaves, torch.autograd.grad(loss(leaves), list(leaves.values()))))
    for k, g in grads.items():
        move = g * (0.01 * v[k].detach().norm() / g.norm())
        with torch.no_grad():
            d1, d2 = ((loss({**v, k: v[k] + f * move}) - loss({**v, k: v[k] - f * move})) / (2 * f) for f in (1.0, 0.5))
        diff, want = (4 * d2 - d1) / 3, (g.double() * move).sum()
        assert abs(diff - want) <= 2e-2 * abs(want), (k, float(diff), float(want))


# ---- across operators --------------------------------------------------------


def test_python_refusals(gdr):
    gen = gen_of(20)
    x, w = rand(gen, 1, 8, 16), rand(gen, 16, 4)
    bf = x.bfloat16()
    bad = [lambda: gdr.short_conv(x.half(), w), lambda: gdr.short_conv(x[0], w), lambda: gdr.short_conv(x, w.bfloat16()),
           lambda: gdr.short_conv(x, rand(gen, 16, 5)), lambda: gdr.short_conv(x, rand(gen, 15, 4)), lambda: gdr.short_conv(x.transpose(1, 2), w[:8]),
           lambda: gdr.short_conv(x, w, initial_state=bf[:, :3]), lambda: gdr.short_conv(x, w, cu_seqlens=torch.tensor([0, 8], device="cuda")),
           lambda: gdr.short_conv(x.expand(2, 8, 16), w, cu_seqlens=bounds((8,))),
           lambda: gdr.short_conv_step(x[0], w, rand(gen, 7, 3, 16)), lambda: gdr.short_conv_step(x[0], w.requires_grad_(), rand(gen, 8, 3, 16)),
           lambda: gdr.state_space_scan(x, bf, rand(gen, 16, 16), rand(gen, 1, 8, 1, 16), rand(gen, 1, 8, 1, 16)),
           lambda: gdr.state_space_scan(x, x, rand(gen, 16, 12), rand(gen, 1, 8, 1, 12), rand(gen, 1, 8, 1, 12)),
           lambda: gdr.state_space_scan(x, x, rand(gen, 16, 16), rand(gen, 1, 8, 3, 16), rand(gen, 1, 8, 3, 16)),
           lambda: gdr.residual_rms_norm(x, rand(gen, 15)), lambda: gdr.residual_rms_norm(x, rand(gen, 16), bf),
           lambda: gdr.residual_rms_norm_fp8(x, rand(gen, 16).requires_grad_()), lambda: gdr.residual_rms_norm(rand(gen, 2, 16385), rand(gen, 16385)),
           lambda: gdr.block_matmul_fp8(x[0], x[0], x[0], x[0])]
    for call in bad:
        with pytest.raises(gdr.GdrError):
            call()


def test_bad_bounds_and_slots_are_reported(gdr):
    """Bounds that do not rise from 0 to T, and a slot past the cache, stay inside the tensors and are reported."""
    gen = gen_of(21)
    torch.cuda.synchronize()
    gdr.check_status()
    v, _, _ = scan_inputs((1, 64, 16, 1, 16, (32, 32), True, True, True, True, True), "f32")
    w = rand(gen, 16, 4)
    for cu in ([0, 70, 64], [5, 20, 64], [0, 40, 30], [-9, 1 << 30, 7]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        leaves = [v[k].requires_grad_() for k in ("x", "A")]
        for call in (lambda: gdr.short_conv(v["x"], w, output_final_state=True, cu_seqlens=cu),
                     lambda: gdr.state_space_scan(**v, output_final_state=True, cu_seqlens=cu)):
            y, _ = call()
            torch.autograd.grad(y.sum(), leaves, allow_unused=True)
            with pytest.raises(gdr.GdrError):
                gdr.check_status()
            gdr.check_status()  # cleared
    x = rand(gen, 2, 16)
    slots = torch.tensor([1, 9], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        y = gdr.short_conv_step(x, w, rand(gen, 3, 3, 16), slots=slots)
        assert not y[1].any()
        with pytest.raises(gdr.GdrError):
            gdr.check_status()
        y = gdr.state_space_step(x, x, v["A"].detach(), rand(gen, 2, 1, 16), rand(gen, 2, 1, 16), rand(gen, 3, 16, 16), slots=slots)
        assert not y[1].any()
        with pytest.raises(gdr.GdrError):
            gdr.check_status()


def test_on_another_stream_and_in_a_graph(gdr):
    gen = gen_of(22)
    v, _, _ = scan_inputs((1, 300, 40, 1, 16, None, True, True, True, True, True), "bf16")
    a, sa, b, sb = operands(gen, 40, 512, 512)
    cw, nw = rand(gen, 40, 4), rand(gen, 40)

    def all_of_them():
        x, _ = gdr.short_conv(v["x"], cw)
        y, h = gdr.state_space_scan(**{**v, "x": x}, output_final_state=True)
        q, s, r = gdr.residual_rms_norm_fp8(y, nw, v["x"])
        return x, y, h, q, s, r, gdr.block_matmul_fp8(a, sa, b, sb)

    with torch.no_grad():
        want = all_of_them()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = all_of_them()
        side.synchronize()
        for x, y in zip(want, got):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = all_of_them()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, held):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
