"""The scan over thousands of tokens is no less precise than elementary torch operations in 32 bits: the norm of each
result's error against 64 bits, at steps between 1e-3 and 1e-1, is at most 1.5 times that of the plain form (whose own
error moves by a few tenths with the inputs), or 2^-22."""
import importlib.util
import os

import pytest
import torch

from test_gpu_layer import gdr  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
NAMES = {"scan": ("y", "final"), "scan_train": ("y", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")}


@pytest.fixture(scope="module")
def ops():
    spec = importlib.util.spec_from_file_location("layer_operators_cases", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("seed", [1, 2])
@pytest.mark.parametrize("case", [
    {"op": "scan_train", "B": 2, "T": 2048, "D": 256, "N": 16, "G": 1, "dtype": "f32"},
    {"op": "scan_train", "B": 1, "T": 4096, "D": 96, "N": 16, "G": 1, "dtype": "f32"},
    {"op": "scan", "B": 1, "T": 4096, "D": 96, "N": 16, "G": 1, "dtype": "f32", "lengths": "1500,2596"}],
    ids=lambda c: f"{c['op']}-{c['T']}x{c['D']}")
def test_errors_are_those_of_32_bits(gdr, ops, case, seed):  # noqa: F811
    exact = ops.exact(case, seed)
    ops.own = True
    got = ops.run(ops.prepare(case, seed))
    ops.own = False
    plain = ops.run(ops.prepare(case, seed))
    found = {}
    for name, e, g, p in zip(NAMES[case["op"]], exact, got, plain):
        size = e.norm()
        found[name] = float((g.detach().double() - e).norm() / size), float((p.detach().double() - e).norm() / size)
    print({k: "%.2e against %.2e" % v for k, v in found.items()})
    assert all(mine <= max(1.5 * theirs, 2.0 ** -22) for mine, theirs in found.values()), found


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_tokens_without_a_step_change_nothing(gdr, dt):  # noqa: F811
    """s = 0 is a decay of exactly 1, whatever A: states come out, and gradients go back, bit for bit."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, D, N = 333, 40, 16
    x, BC = (torch.randn(2, T, D, device="cuda", generator=gen).to(dt), torch.randn(2, T, 1, N, device="cuda", generator=gen).to(dt))
    A = -torch.logspace(-6, 6, D * N, device="cuda").view(D, N)
    A[0] = 0
    h0 = torch.randn(2, D, N, device="cuda", generator=gen).requires_grad_()
    _, ht = gdr.state_space_scan(x, torch.zeros_like(x), A, BC, BC, dt_softplus=False, initial_state=h0, output_final_state=True)
    dht = torch.randn(2, D, N, device="cuda", generator=gen)
    assert torch.equal(ht, h0) and torch.equal(torch.autograd.grad(ht, h0, dht)[0], dht)
    state = h0.detach().clone()
    gdr.state_space_step(x[:, 0], torch.zeros_like(x[:, 0]), A, BC[:, 0], BC[:, 0], state, dt_softplus=False)
    assert torch.equal(state, h0)
