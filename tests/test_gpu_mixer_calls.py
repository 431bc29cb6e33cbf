"""Calls around the gated linear recurrence, the delta rule's single token and the norm after a block: sequences and rows
that must not reach one another, captured and replayed calls, other streams, stepped caches that were saved, bounds and
slots that are wrong, offsets past 32 bits, and the operators run together as a layer."""
import pytest
import torch

import mixer_plain as M
from layer_plain import f64
from test_gpu_layer import DT, bounds, close, gdr, gen_of, rand  # noqa: F401  (the fixture)
from test_gpu_mixer import delta_inputs, linear_inputs, linear_tol

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
TOKENS = ("x", "input_gate", "decay_gate", "z")


def run_linear(gdr, v, dy, dht, lengths):  # noqa: F811
    leaves = {k: t.detach().clone().requires_grad_() for k, t in v.items() if t is not None}
    y, ht = gdr.gated_linear_scan(**{**v, **leaves}, output_final_state=True, cu_seqlens=bounds(lengths))
    return y.detach(), ht.detach(), dict(zip(leaves, torch.autograd.grad([y, ht], list(leaves.values()), [dy, dht])))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [(30, 34), (1501, 1499), (128, 128), (64, 7)], ids=str)
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("where", ["x", "input_gate", "decay_gate", "z", "dy", "h0", "dht"])
@pytest.mark.parametrize("bad", [0, 1])
def test_a_foul_sequence_changes_nothing_of_the_other(gdr, bad, where, value, lengths, dt):  # noqa: F811
    v, dy, dht = linear_inputs((1, sum(lengths), 35, lengths, True, True), dt, 81)
    clean = run_linear(gdr, v, dy, dht, lengths)
    at = slice(lengths[0] - 3, lengths[0]) if bad == 0 else slice(lengths[0], lengths[0] + 3)
    w, fdy, fdht = {k: t.clone() for k, t in v.items()}, dy.clone(), dht.clone()
    if where == "h0":
        w["initial_state"][bad] = value
    elif where == "dht":
        fdht[bad] = value
    else:
        (fdy if where == "dy" else w[where])[0, at] = value
    foul = run_linear(gdr, w, fdy, fdht, lengths)
    keep = 1 - bad
    kept = slice(0, lengths[0]) if keep == 0 else slice(lengths[0], sum(lengths))
    for a, b in ((clean[0][:, kept], foul[0][:, kept]), (clean[1][keep], foul[1][keep]),
                 (clean[2]["initial_state"][keep], foul[2]["initial_state"][keep]),
                 *((clean[2][k][:, kept], foul[2][k][:, kept]) for k in TOKENS)):
        assert torch.isfinite(b.float()).all() and torch.equal(a, b)
    if not (value == INF and where in ("input_gate", "decay_gate")):  # an infinite gate is a closed or an open one
        assert not all(torch.isfinite(t.float()).all() for t in (foul[0], foul[1], *foul[2].values()))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_thousands_of_short_sequences(gdr, dt):  # noqa: F811
    """More sequences than a warp's lanes, and than their square; many of them empty, some at one place by the hundred."""
    gen = torch.Generator().manual_seed(98)
    lengths = torch.randint(0, 4, (1500,), generator=gen).tolist() + [0] * 400 + [70] + [1] * 90 + [0] * 33
    v, dy, dht = linear_inputs((1, sum(lengths), 5, lengths, True, True), dt, 99)
    y, ht, g = run_linear(gdr, v, dy, dht, lengths)
    p = {k: f64(t, True) for k, t in v.items()}
    h0 = p.pop("initial_state")
    ry, rht = M.linear(**p, h0=h0, lengths=lengths)
    p["initial_state"] = h0
    want = torch.autograd.grad([ry, rht], [p[k] for k in g], [f64(dy), f64(dht)])
    close(y, ry, linear_tol(70), "y")
    close(ht, rht, linear_tol(70), "final")
    for k, w in zip(g, want):
        close(g[k], w, linear_tol(len(lengths) if k == "decay" else 70), k)


def test_nan_stays_in_its_channel_and_row(gdr):  # noqa: F811
    v, dy, dht = linear_inputs((2, 300, 70, None, False, True), "bf16", 82)
    v["decay_gate"][1, 137, 41] = NAN
    y, ht, g = run_linear(gdr, v, dy, dht, None)
    bad = torch.isnan(y)
    assert bad[1, 137:, 41].all() and int(bad.sum()) == 300 - 137
    assert torch.isnan(ht[1, 41]) and int(torch.isnan(ht).sum()) == 1
    assert torch.isnan(g["x"][1, :138, 41]).any() and not torch.isnan(g["x"][0]).any() and not torch.isnan(g["x"][1, :, :41]).any()
    x, w = rand(gen_of(83), 40, 128), torch.ones(128, device="cuda")
    x[7, 3] = NAN
    r = gdr.gated_residual_rms_norm(x, w)[1]
    assert torch.isnan(r[7]).all() and int(torch.isnan(r).sum()) == 128
    d, state = delta_inputs((3, 1, 2, 64, 64, 3), "f32")
    d["k"][1] = NAN
    o = gdr.gated_delta_step(**d, state=state)
    assert torch.isnan(o[1]).all() and torch.isnan(state[1]).all() and torch.isfinite(o[[0, 2]]).all() and torch.isfinite(state[[0, 2]]).all()


def test_nothing_behind_the_outputs_is_written(gdr):  # noqa: F811
    """Idle slots, and the memory around a state that is a slice of a larger one."""
    v, _, _ = linear_inputs((3, 1, 65, None, False, False), "f32", 84)
    one = {k: t[:, 0] for k, t in v.items() if t is not None and k != "decay"}
    pool = torch.full((7, 65), 5.0, device="cuda")
    gdr.gated_linear_step(**one, decay=v["decay"], state=pool[2:5])
    assert (pool[:2] == 5).all() and (pool[5:] == 5).all() and not (pool[2:5] == 5).any()
    d, _ = delta_inputs((2, 1, 2, 64, 64, 2), "bf16")
    pool = torch.full((6, 2, 64, 64), 5.0, device="cuda")
    gdr.gated_delta_step(**d, state=pool[1:4], slots=torch.tensor([2, 0], dtype=torch.int32, device="cuda"))
    assert (pool[0] == 5).all() and (pool[2] == 5).all() and (pool[4:] == 5).all()


def test_wrong_bounds_and_slots_are_reported(gdr):  # noqa: F811
    v, dy, _ = linear_inputs((1, 300, 40, None, False, True), "bf16", 85)
    for cu in ([0, 200, 100, 300], [0, 400], [5, 300], [0, -7, 300], [0, 100]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        x = v["x"].detach().clone().requires_grad_()
        y, ht = gdr.gated_linear_scan(**{**v, "x": x}, output_final_state=True, cu_seqlens=cu)
        with pytest.raises(gdr.GdrError, match="DEVICE"):
            gdr.check_status()
        torch.autograd.grad(y, x, dy)
        with pytest.raises(gdr.GdrError, match="DEVICE"):
            gdr.check_status()
    one = {k: (t[0, :4] if k != "decay" else t) for k, t in v.items() if t is not None}
    state = torch.zeros(4, 40, device="cuda")
    slots = torch.tensor([0, 4, -1, 1 << 30], dtype=torch.int32, device="cuda")
    y = gdr.gated_linear_step(**one, state=state, slots=slots)
    assert y[0].any() and not y[1:].any() and not state[1:].any()
    with pytest.raises(gdr.GdrError, match="DEVICE"):
        gdr.check_status()
    d, _ = delta_inputs((4, 1, 2, 64, 64, 4), "bf16")
    state = torch.zeros(4, 2, 64, 64, device="cuda")
    o = gdr.gated_delta_step(**d, state=state, slots=slots)
    assert o[0].any() and not o[1:].any() and not state[1:].any()
    with pytest.raises(gdr.GdrError, match="DEVICE"):
        gdr.check_status()
    gdr.check_status()


def test_calls_without_tokens(gdr):  # noqa: F811
    v, dy, dht = linear_inputs((2, 0, 12, None, True, True), "bf16", 86)
    y, ht, g = run_linear(gdr, v, dy, dht, None)
    assert y.shape == (2, 0, 12) and torch.equal(ht, v["initial_state"]) and torch.equal(g["initial_state"], dht) and not g["decay"].any()
    v, dy, dht = linear_inputs((1, 0, 12, (0, 0), False, False), "f32", 86)
    y, ht, g = run_linear(gdr, v, dy, dht, (0, 0))
    assert not ht.any() and not g["decay"].any()
    x, w = torch.zeros(0, 64, device="cuda", requires_grad=True), torch.ones(64, device="cuda", requires_grad=True)
    y, r = gdr.gated_residual_rms_norm(x, w, next_weight=w)
    gx, gw = torch.autograd.grad([y, r], [x, w], [x.detach(), x.detach()])
    assert gx.shape == (0, 64) and not gw.any()
    assert gdr.gated_linear_step(*(torch.zeros(0, 8, device="cuda"),) * 3, torch.zeros(8, device="cuda"), torch.zeros(0, 8, device="cuda")).shape == (0, 8)
    q = torch.zeros(0, 2, 64, device="cuda")
    assert gdr.gated_delta_step(q, q, q, q[:, :, 0].contiguous(), q[:, :, 0].contiguous(), torch.zeros(1, 2, 64, 64, device="cuda")).shape == (0, 2, 64)


def test_steps_raise_the_version_of_their_state(gdr):  # noqa: F811
    v, dy, dht = linear_inputs((2, 9, 16, None, True, False), "f32", 87)
    x = v["x"].detach().clone().requires_grad_()
    y, _ = gdr.gated_linear_scan(**{**v, "x": x})
    one = {k: v[k][:, 0] for k in TOKENS if v[k] is not None}
    gdr.gated_linear_step(**one, decay=v["decay"], state=v["initial_state"])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y, x, dy)
    d, state = delta_inputs((2, 1, 1, 64, 64, 2), "f32")
    before = state._version
    gdr.gated_delta_step(**d, state=state)
    assert state._version == before + 1
    with torch.inference_mode():
        gdr.gated_delta_step(**d, state=state)
        gdr.gated_linear_step(**one, decay=v["decay"], state=v["initial_state"])


def test_python_refusals(gdr):  # noqa: F811
    v, _, _ = linear_inputs((2, 9, 16, None, True, True), "f32", 88)
    call = gdr.gated_linear_scan
    for bad in (dict(x=v["x"].half()), dict(input_gate=v["x"].bfloat16()), dict(decay_gate=v["x"][:, :8]), dict(z=v["x"].transpose(1, 2)),
                dict(decay=v["decay"].double()), dict(decay=v["decay"][:8]), dict(decay_scale=0), dict(decay_scale=NAN), dict(decay_scale=-2.0),
                dict(initial_state=v["initial_state"][:1]), dict(cu_seqlens=bounds((9,))), dict(x=v["x"][0]),
                dict(x=v["x"].transpose(1, 2).contiguous().transpose(1, 2)), dict(decay=v["decay"].cpu()), dict(input_gate=v["x"].cpu())):
        with pytest.raises(gdr.GdrError):
            call(**{**v, **bad})
    one = {k: v[k][:, 0] for k in TOKENS}
    state = torch.zeros(2, 16, device="cuda")
    for bad in (dict(state=state[:1]), dict(state=state.double()), dict(state=state[0]), dict(slots=torch.zeros(2, dtype=torch.int64, device="cuda")),
                dict(x=one["x"].clone().requires_grad_()), dict(state=state.clone().requires_grad_()), dict(decay_scale=-1.0)):
        with pytest.raises(gdr.GdrError):
            gdr.gated_linear_step(**{**one, "decay": v["decay"], "state": state, **bad})
    d, st = delta_inputs((2, 2, 4, 64, 64, 3), "f32")
    for bad in (dict(q=d["q"][0]), dict(k=d["k"][:, :1]), dict(k=d["k"].bfloat16()), dict(v=d["v"][:, :3]), dict(g=d["g"].double()), dict(beta=d["beta"][:, :2]),
                dict(state=st[:1]), dict(state=st[:, :2]), dict(state=st.transpose(2, 3)), dict(v=d["v"].transpose(1, 2).contiguous().transpose(1, 2)),
                dict(q=d["q"].clone().requires_grad_()), dict(q=d["q"][..., :32], k=d["k"][..., :32]),
                dict(state=torch.zeros(3 * 4 * 64 * 64 + 1, device="cuda")[1:].view(3, 4, 64, 64))):
        with pytest.raises(gdr.GdrError):
            gdr.gated_delta_step(**{**d, "state": st, **bad})
    x, w = torch.zeros(4, 32, device="cuda"), torch.ones(32, device="cuda")
    for args in ((x, w[:8]), (x, w.double()), (x.half(), w), (x, w, x.bfloat16()), (x, w, x[:2]), (x, w, None, x[:, :8]), (x, w, None, None, w[:3]),
                 (x.t(), w), (torch.zeros(1, 16385, device="cuda"), torch.ones(16385, device="cuda")), (torch.zeros(3, 4, 5, 8, device="cuda").transpose(1, 2), w[:8].contiguous())):
        with pytest.raises(gdr.GdrError):
            gdr.gated_residual_rms_norm(*args)
    y, r = gdr.gated_residual_rms_norm(x.requires_grad_(), w)
    g = torch.autograd.grad(r, x, torch.ones_like(r), retain_graph=True)
    with pytest.raises(gdr.GdrError):
        torch.autograd.grad(r, x, torch.ones_like(r), create_graph=True)


def test_captured_calls_replay(gdr):  # noqa: F811
    """Two graphs of one pool, each a training step and a token, replayed in turn on new inputs; then eager ones again."""
    v, dy, dht = linear_inputs((1, 900, 66, (300, 0, 600), True, True), "bf16", 89)
    cu = bounds((300, 0, 600))
    d, state = delta_inputs((3, 2, 4, 128, 128, 3), "bf16")
    gen = gen_of(90)
    x, gate, res, w, w2 = (rand(gen, 50, 200), rand(gen, 50, 200), rand(gen, 50, 200), rand(gen, 200), rand(gen, 200))
    leaves = [t.requires_grad_() for t in (*v.values(), x, gate, res, w, w2)]

    def step():
        y, ht = gdr.gated_linear_scan(**v, output_final_state=True, cu_seqlens=cu)
        a, b = gdr.gated_residual_rms_norm(x, w, gate, res, w2, scale=0.5)
        grads = torch.autograd.grad([y, ht, a, b], leaves, [dy, dht, x.detach(), res.detach()])
        o = gdr.gated_delta_step(**d, state=state)
        return [t.detach() for t in (y, ht, a, b, *grads, o, state.clone())]

    start = state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs, pool = [], [], torch.cuda.graph_pool_handle()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(step())
        graphs.append(g)
    for turn in range(4):
        with torch.no_grad():
            v["x"].copy_(torch.randn_like(v["x"]))
            x.copy_(torch.randn_like(x))
            d["v"].copy_(torch.randn_like(d["v"]))
        state.copy_(start)
        graphs[turn % 2].replay()
        got = [t.clone() for t in outs[turn % 2]]
        state.copy_(start)
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_another_stream(gdr):  # noqa: F811
    v, dy, dht = linear_inputs((1, 1500, 66, None, True, True), "bf16", 91)
    want = run_linear(gdr, v, dy, dht, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            got = run_linear(gdr, v, dy, dht, None)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want[0], got[0]) and all(torch.equal(want[2][k], got[2][k]) for k in want[2])


def test_two_calls_at_once(gdr):  # noqa: F811
    """Long scans on two streams, whose chunks' CTAs share the SMs."""
    v, dy, dht = linear_inputs((1, 20000, 256, None, True, False), "bf16", 92)
    w, ey, eht = linear_inputs((1, 20000, 250, None, True, False), "bf16", 93)
    want = run_linear(gdr, v, dy, dht, None), run_linear(gdr, w, ey, eht, None)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(3):
        for i, (s, args) in enumerate(zip(streams, ((v, dy, dht), (w, ey, eht)))):
            with torch.cuda.stream(s):
                got[i] = run_linear(gdr, *args, None)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(a[2][k], b[2][k]) for k in a[2])


def test_offsets_past_32_bits(gdr):  # noqa: F811
    """The last slot of caches of more than 2^31 bytes and elements, and rows of more than 2^31 elements."""
    d, _ = delta_inputs((1, 1, 2, 128, 128, 1), "bf16")
    slots = (1 << 31) // (2 * 128 * 128) + 3  # elements past 2^31
    state = torch.zeros(slots, 2, 128, 128, device="cuda")
    o = gdr.gated_delta_step(**d, state=state, slots=torch.tensor([slots - 1], dtype=torch.int32, device="cuda"))
    small = torch.zeros(1, 2, 128, 128, device="cuda")
    assert torch.equal(o, gdr.gated_delta_step(**d, state=small)) and torch.equal(state[-1], small[0]) and not state[0].any() and not state[-2].any()
    del state
    v, _, _ = linear_inputs((1, 1, 64, None, False, False), "f32", 94)
    one = {k: v[k][:, 0] for k in TOKENS if v[k] is not None}
    state = torch.zeros((1 << 25) + 5, 64, device="cuda")
    y = gdr.gated_linear_step(**one, decay=v["decay"], state=state, slots=torch.tensor([state.shape[0] - 1], dtype=torch.int32, device="cuda"))
    small = torch.zeros(1, 64, device="cuda")
    assert torch.equal(y, gdr.gated_linear_step(**one, decay=v["decay"], state=small)) and torch.equal(state[-1], small[0]) and not state[:4].any()
    del state
    rows, D = (1 << 20) + 7, 2056  # 2.16e9 elements
    x, w = torch.ones(rows, D, dtype=torch.bfloat16, device="cuda"), torch.ones(D, device="cuda")
    x[-1] = rand(gen_of(95), D, dt=torch.bfloat16)
    r = gdr.gated_residual_rms_norm(x, w)[1]
    assert torch.equal(r[-1:], gdr.gated_residual_rms_norm(x[-1:].clone(), w)[1])
    del r
    wide = x.view(-1)[: (rows * D) // 64 * 64].view(1, -1, 64)  # the same memory as 33.8 million tokens
    tail, gates = 130, torch.zeros(1, 130, 64, dtype=torch.bfloat16, device="cuda")
    T = (1 << 18) + 130
    long = wide.as_strided((1, T, 64), (wide.numel(), 8192, 1))  # strides that pass 2^31 elements
    assert (T - 1) * 8192 > 1 << 31
    zero = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda").expand(1, T, 64)
    decay = torch.full((64,), -1.0, device="cuda")
    y, h = gdr.gated_linear_scan(long, zero, zero, decay, output_final_state=True)
    with torch.no_grad():
        end = long[:, -tail:].contiguous()
        _, h0 = gdr.gated_linear_scan(long[:, :-tail], zero[:, :-tail], zero[:, :-tail], decay, output_final_state=True)
        y2, h2 = gdr.gated_linear_scan(end, gates, gates, decay, initial_state=h0, output_final_state=True)
    close(h, f64(h2), linear_tol(300), "state")
    close(y[:, -tail:], f64(y2), linear_tol(300) + 2.0 ** -7, "y")


def test_a_layer_of_them(gdr):  # noqa: F811
    """A recurrent layer: the norm before it, gates from a projection, short convolution, recurrence with its output gate,
    gated norm of each head, projection, and the norm after it with the stream and the next layer's norm.  A prompt and then
    tokens give what the whole sequence gives; its gradients are those of the 64-bit layer."""
    gen, B, T, D, heads = gen_of(96), 2, 70, 96, 4
    P = dict(norm=1 + 0.1 * rand(gen, D), w_in=rand(gen, 5 * D, D) * D ** -0.5, conv=rand(gen, D, 4) * 0.5, decay=rand(gen, D) - 3,
             head=1 + 0.1 * rand(gen, D // heads), w_out=rand(gen, D, D) * D ** -0.5, post=1 + 0.1 * rand(gen, D), after=1 + 0.1 * rand(gen, D))
    h = rand(gen, B, T, D)

    def mix(p, h, conv, scan):
        a, stream = gdr.residual_rms_norm(h, p["norm"])
        x, i, r, z, g = (a @ p["w_in"].t()).split(D, dim=-1)
        x = scan(conv(x), i, r, z)
        x = gdr.gated_residual_rms_norm(x.unflatten(-1, (heads, -1)), p["head"], g.unflatten(-1, (heads, -1)))[1].flatten(-2)
        return gdr.gated_residual_rms_norm(x @ p["w_out"].t(), p["post"], None, stream, p["after"], scale=0.5)

    conv_end, scan_end = [], []

    def prompt(p):
        def conv(x):
            y, s = gdr.short_conv(x, p["conv"], output_final_state=True)
            conv_end.append(s)
            return y

        def scan(x, i, r, z):
            y, s = gdr.gated_linear_scan(x, i, r, p["decay"], z, output_final_state=True)
            scan_end.append(s)
            return y
        return conv, scan

    with torch.no_grad():
        whole = mix(P, h, *prompt(P))
        mix(P, h[:, :64].contiguous(), *prompt(P))
        cs, ss = conv_end[-1], scan_end[-1]
        for t in range(64, T):
            y, r = mix(P, h[:, t], lambda x: gdr.short_conv_step(x, P["conv"], cs),
                       lambda x, i, r, z: gdr.gated_linear_step(x, i, r, P["decay"], ss, z))
            close(y, f64(whole[0][:, t]), 1e-4, "y")
            close(r, f64(whole[1][:, t]), 1e-4, "r")
    leaves = {k: t.detach().clone().requires_grad_() for k, t in P.items()}
    y, r = mix(leaves, h, *prompt(leaves))
    dy, dr = rand(gen, B, T, D), rand(gen, B, T, D)
    got = torch.autograd.grad([y, r], list(leaves.values()), [dy, dr])
    q = {k: f64(t, True) for k, t in P.items()}
    import layer_plain as L
    hh = f64(h)
    x, i, rg, z, g = (L.norm(hh, q["norm"]) @ q["w_in"].t()).split(D, dim=-1)
    x, _ = M.linear(L.conv(x, q["conv"])[0], i, rg, q["decay"], z)
    x = M.block_norm(x.unflatten(-1, (heads, -1)), q["head"], g.unflatten(-1, (heads, -1)))[1].flatten(-2)
    yy, rr = M.block_norm(x @ q["w_out"].t(), q["post"], None, hh, q["after"], 0.5)
    want = torch.autograd.grad([yy, rr], list(q.values()), [f64(dy), f64(dr)])
    close(y, yy, 2e-3, "y")  # torch's fp32 products between the operators
    for k, a, b in zip(P, got, want):
        close(a, b, 2e-3, k)
