"""The linear recurrence over thousands of tokens is about as precise as elementary torch operations in 32 bits, and a closed
gate keeps its state bit for bit.

The bound, set before the first run: the norm of each result's error against 64 bits is at most twice that of the plain form, or
2^-22.  Both round a decay to about half a step, which a state adds up at random over the tokens that it remembers (up to 2000 at
the cases' decays of 0.9 to 0.999 behind half-open gates), and here one rounding a token comes on top.

Such a norm hardly sees a small error that all decays have alike, so that has a bound of its own.  ex2.approx, for one, is off by 0.5e-8
to 3e-8 on average, by ranges of its argument, and lies 1.5e-8 low over them.  A state of 1 without inputs decays by the product of T decays; the
mean over 4096 channels of its logarithm's error, over T, is the decays' mean error, known to 2^-24 / sqrt(4096 T) = 4e-11 for T = 600.  At most
7.5e-9, half of that offset, is allowed.
"""
import importlib.util
import os

import pytest
import torch

from test_gpu_layer import gdr  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")
NAMES = {"linear": ("y", "final"), "linear_train": ("y", "dx", "di", "dr", "ddecay", "dz", "dh0")}


@pytest.fixture(scope="module")
def ops():
    spec = importlib.util.spec_from_file_location("more_layer_operators_cases", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("seed", [1, 2])
@pytest.mark.parametrize("case", [
    {"op": "linear", "B": 2, "T": 4096, "D": 512, "z": False, "dtype": "f32"},
    {"op": "linear_train", "B": 2, "T": 4096, "D": 512, "z": False, "dtype": "f32"},
    {"op": "linear_train", "B": 1, "T": 5000, "D": 131, "z": True, "dtype": "f32", "lengths": "1500,3500"}],
    ids=lambda c: f"{c['op']}-{c['T']}x{c['D']}")
def test_errors_are_those_of_32_bits(gdr, ops, case, seed):  # noqa: F811
    exact = ops.exact(case, seed)
    ops.own = True
    got = ops.run(ops.prepare(case, seed))
    ops.own = False
    plain = ops.run(ops.prepare(case, seed))
    found = {}
    for k, (e, g, p) in enumerate(zip(exact, got, plain)):
        size = e.norm()
        found[NAMES[case["op"]][k]] = float((g.detach().double() - e).norm() / size), float((p.detach().double() - e).norm() / size)
    print({k: "%.2e against %.2e" % v for k, v in found.items()})
    assert all(mine <= max(2 * theirs, 2.0 ** -22) for mine, theirs in found.values()), found


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths", [None, (1000, 0, 1100)])
def test_a_closed_gate_keeps_its_state(gdr, lengths, dt):  # noqa: F811
    """sigmoid(decay_gate) = 0 is a decay of exactly 1 and an input of 0: states come out, and gradients go back, bit for bit."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    B, T, D = (2, 2100, 70) if lengths is None else (1, 2100, 70)
    n = B if lengths is None else len(lengths)
    x, i = (torch.randn(B, T, D, device="cuda", generator=gen).to(dt) for _ in range(2))
    shut = torch.full_like(x, -1000.0)
    decay = torch.linspace(-20, 20, D, device="cuda")
    cu = None if lengths is None else torch.tensor([0, 1000, 1000, 2100], dtype=torch.int32, device="cuda")
    h0 = torch.randn(n, D, device="cuda", generator=gen).requires_grad_()
    y, ht = gdr.gated_linear_scan(x, i, shut, decay, initial_state=h0, output_final_state=True, cu_seqlens=cu)
    assert torch.equal(ht, h0)
    for b in range(B):
        for s, (at, end) in enumerate(((0, T),) if lengths is None else ((0, 1000), (1000, 1000), (1000, 2100))):
            assert torch.equal(y[b, at:end], h0[b if lengths is None else s].to(dt).expand(end - at, D))
    dht = torch.randn(n, D, device="cuda", generator=gen)
    assert torch.equal(torch.autograd.grad(ht, h0, dht)[0], dht)
    state = h0.detach().clone()
    rows = x[0, :n]
    gdr.gated_linear_step(rows, rows, shut[0, :n], decay, state)
    assert torch.equal(state, h0)


def test_decays_have_no_offset(gdr):  # noqa: F811
    gen, T, D = torch.Generator(device="cuda").manual_seed(4), 600, 4096
    r = torch.randn(1, T, D, device="cuda", generator=gen)
    decay = -7.0 + 2.0 * torch.rand(D, device="cuda", generator=gen)  # s from 0.007 to 0.054: states of 1 end between 0.1 and 1e-7
    exact = (-8.0 * torch.nn.functional.softplus(decay.double()) * torch.sigmoid(r.double())).sum((0, 1))
    assert float(exact.min()) > -25
    zeros, one = torch.zeros_like(r), torch.ones(1, D, device="cuda")
    h0 = one.clone().requires_grad_()
    _, ht = gdr.gated_linear_scan(zeros, zeros, r, decay, initial_state=h0, output_final_state=True)
    dh0, = torch.autograd.grad(ht, h0, one)
    state = one.clone()
    for t in range(T):
        gdr.gated_linear_step(zeros[:, t], zeros[:, t], r[:, t], decay, state)
    for name, got in (("forward", ht), ("backward", dh0), ("step", state)):
        mean = float((got.detach().double().log() - exact).mean()) / T
        print(name, "%.2e" % mean)
        assert abs(mean) <= 7.5e-9, (name, mean)
