"""What one packed sequence holds, NaN and infinities included, changes nothing of another: each test runs a call with
and without the foreign values and wants the other sequence's results bit for bit."""
import pytest
import torch

from test_gpu_layer import DT, bounds, gdr, gen_of, rand, scan_inputs  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
PER_TOKEN = ("x", "dt", "B", "C", "z")


def run_scan(gdr, v, dy, dht, lengths, softplus):  # noqa: F811
    leaves = {k: t.detach().clone().requires_grad_() for k, t in v.items() if t is not None}
    y, ht = gdr.state_space_scan(**{**v, **leaves}, dt_softplus=softplus, output_final_state=True, cu_seqlens=bounds(lengths))
    return y.detach(), ht.detach(), dict(zip(leaves, torch.autograd.grad([y, ht], list(leaves.values()), [dy, dht])))


def same(a, b, what):
    assert torch.isfinite(a.float()).all(), what
    assert torch.equal(a, b), what


def scan_case(gdr, lengths, D, G, N, dt, foul, softplus=True, bias=True):  # noqa: F811
    """``foul`` changes the inputs of one of two sequences and says which."""
    T = sum(lengths)
    v, dy, dht = scan_inputs((1, T, D, G, N, lengths, True, True, True, bias, softplus), dt)
    clean = run_scan(gdr, v, dy, dht, lengths, softplus)
    w = {k: None if t is None else t.clone() for k, t in v.items()}
    bad = foul(w)
    fouled = run_scan(gdr, w, dy, dht, lengths, softplus)
    assert not torch.isfinite(fouled[0]).all()  # it was foul indeed
    keep = 1 - bad
    at = slice(0, lengths[0]) if keep == 0 else slice(lengths[0], T)
    same(fouled[0][:, at], clean[0][:, at], "y")
    same(fouled[1][keep], clean[1][keep], "final")
    for k in PER_TOKEN:
        same(fouled[2][k][:, at], clean[2][k][:, at], k)
    same(fouled[2]["initial_state"][keep], clean[2]["initial_state"][keep], "initial_state")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,G,N", [(40, 1, 16), (33, 1, 8), (16, 2, 32)])
@pytest.mark.parametrize("bad", [0, 1])
def test_scan_nan_steps_stay_in_their_sequence(gdr, bad, D, G, N, dt):  # noqa: F811
    """Long enough to be cut into segments, the sequences' border inside one of them."""
    lengths = (1501, 1499)

    def foul(v):
        v["dt"][0, 1495 if bad == 0 else 1510, 5] = NAN
        return bad
    scan_case(gdr, lengths, D, G, N, dt, foul)


@pytest.mark.parametrize("bad", [0, 1])
def test_scan_overflowing_steps_stay_in_their_sequence(gdr, bad):  # noqa: F811
    """Without the softplus, steps of one sequence that make every decay a growth (e^{A sum s} overflows).  No bias: it
    would turn some of the other sequence's steps negative too."""
    lengths = (1501, 1499)

    def foul(v):
        v["dt"][0, slice(0, 1501) if bad == 0 else slice(1501, 3000)] = -2.0
        return bad
    scan_case(gdr, lengths, 24, 1, 16, "f32", foul, softplus=False, bias=False)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [(30, 34), (1501, 1499)], ids=str)
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("bad", [0, 1])
def test_scan_foul_tokens_beside_the_border(gdr, bad, value, lengths, dt):  # noqa: F811
    """Inputs, gates, B and C of the tokens next to the border, in the tile that both sequences share."""
    def foul(v):
        at = slice(lengths[0] - 3, lengths[0]) if bad == 0 else slice(lengths[0], lengths[0] + 3)
        for k in PER_TOKEN:
            v[k][0, at] = value
        return bad
    scan_case(gdr, lengths, 40, 1, 16, dt, foul)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [(30, 34), (3, 2), (128, 129)], ids=str)
@pytest.mark.parametrize("D,W", [(64, 4), (37, 3), (30, 2)])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("bad", [0, 1])
def test_conv_foul_tokens_beside_the_border(gdr, bad, value, silu, D, W, lengths, dt):  # noqa: F811
    gen, T = gen_of(31), sum(lengths)
    x, dy, w, b = rand(gen, 1, T, D, dt=DT[dt]), rand(gen, 1, T, D, dt=DT[dt]), rand(gen, D, W), rand(gen, D)
    h0, dht = rand(gen, 2, W - 1, D, dt=DT[dt]), rand(gen, 2, W - 1, D, dt=DT[dt])

    def run(x, dy):
        x, h = x.clone().requires_grad_(), h0.clone().requires_grad_()
        y, ht = gdr.short_conv(x, w, b, "silu" if silu else None, h, True, bounds(lengths))
        return (y.detach(), ht.detach(), *torch.autograd.grad([y, ht], [x, h], [dy, dht]))

    at = slice(lengths[0] - 2, lengths[0]) if bad == 0 else slice(lengths[0], lengths[0] + 2)
    clean = run(x, dy)
    for foul_dy in (False, True):
        fx, fdy = x.clone(), dy.clone()
        (fdy if foul_dy else fx)[0, at] = value
        fouled = run(fx, fdy)
        assert not torch.isfinite(fouled[2 if foul_dy else 0]).all()
        keep = 1 - bad
        kept = slice(0, lengths[0]) if keep == 0 else slice(lengths[0], T)
        for i, what in ((0, "y"), (2, "dx")):
            same(fouled[i][:, kept], clean[i][:, kept], what)
        for i, what in ((1, "final"), (3, "dinit")):
            same(fouled[i][keep], clean[i][keep], what)
