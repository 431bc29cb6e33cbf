"""What the gated linear recurrence, the delta rule's single token and the norm after a block refuse, without a GPU:
through the C ABI (codes, nothing launched) and through the Python calls."""
import ctypes

import pytest
import torch
from torch.autograd import forward_ad

import gated_deltanet_chunked_delta_gb300 as gdr
from gated_deltanet_chunked_delta_gb300 import layer as L

ARG, SHAPE, DTYPE, ALIGN, WORKSPACE = 1, 2, 3, 4, 5
P = 0x10000  # an aligned address that is never read: every call below is refused


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_chunked_delta_gb300 import build
    build.build()
    return L._calls()


def _call(f, args):
    return f(ctypes.byref(args), None)


def _linear(**kw):
    rows = {n + s: 64 for n in "xirz" for s in ("_row", "_batch")}
    a = dict(x=P, input_gate=P, decay_gate=P, z=P, decay=P, B=1, T=300, D=64, n_seqs=1, decay_scale=8.0, dtype=0, y=P, states=P,
             dy=P, dx=P, di=P, dr=P, dz=P, ddecay=P, workspace=P, workspace_bytes=1 << 40, **rows)
    return L._LinearArgs(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(input_gate=None), ARG), (dict(decay_gate=None), ARG), (dict(decay=None), ARG), (dict(B=0), SHAPE),
    (dict(T=-1), SHAPE), (dict(D=0), SHAPE), (dict(T=1 << 30), SHAPE), (dict(D=1 << 24), SHAPE), (dict(B=65536, n_seqs=65536), SHAPE),
    (dict(dtype=3), DTYPE), (dict(n_seqs=2), SHAPE), (dict(cu_seqlens=P, n_seqs=0), SHAPE), (dict(cu_seqlens=P, B=2, n_seqs=2), SHAPE),
    (dict(cu_seqlens=P, n_seqs=(1 << 24) + 1), SHAPE), (dict(cu_seqlens=P + 2), ALIGN), (dict(decay_scale=0.0), ARG),
    (dict(decay_scale=-1.0), ARG), (dict(decay_scale=float("inf")), ARG), (dict(decay_scale=float("nan")), ARG), (dict(x=P + 1), ALIGN),
    (dict(z=P + 1), ALIGN), (dict(decay=P + 2), ALIGN), (dict(h0=P + 2), ALIGN), (dict(states=P + 1), ALIGN),
    (dict(x=P + 2, dtype=1), ALIGN)])
def test_linear_refusals(lib, kw, code):
    assert _call(lib.gdr_linear_fwd, _linear(**kw)) == code
    assert _call(lib.gdr_linear_bwd, _linear(**kw)) == code
    assert lib.gdr_last_error()


@pytest.mark.parametrize("kw,code", [(dict(y=None), ARG), (dict(y=P + 1), ALIGN), (dict(ht=P + 2), ALIGN)])
def test_linear_forward_refusals(lib, kw, code):
    assert _call(lib.gdr_linear_fwd, _linear(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), ARG), (dict(states=None), ARG), (dict(dx=None), ARG), (dict(di=None), ARG), (dict(dr=None), ARG), (dict(dz=None), ARG),
    (dict(ddecay=None), ARG), (dict(dht=P + 2), ALIGN), (dict(dh0=P + 1), ALIGN), (dict(workspace=None), WORKSPACE),
    (dict(workspace=P + 8), ALIGN), (dict(workspace_bytes=16), WORKSPACE)])
def test_linear_backward_refusals(lib, kw, code):
    assert _call(lib.gdr_linear_bwd, _linear(**kw)) == code


def test_linear_workspace_sizes(lib):
    for f, a in ((lib.gdr_linear_fwd_workspace_size, lib.gdr_linear_fwd), (lib.gdr_linear_bwd_workspace_size, lib.gdr_linear_bwd)):
        need = f(1, 5000, 100)
        assert need >= 16 * 100 * 5000 // 96 and need % 16 == 0
        for kw, code in ((dict(workspace=None), WORKSPACE), (dict(workspace=P + 8), ALIGN), (dict(workspace_bytes=need - 1), WORKSPACE)):
            assert _call(a, _linear(**{**dict(T=5000, D=100), **kw})) == code
        assert f(0, 5, 5) == f(1, -1, 5) == f(1, 5, 0) == 0
        assert f(1, 1 << 20, 1 << 12) >= 16 * (1 << 12) * (1 << 20) // 96
    assert lib.gdr_linear_fwd_workspace_size(1, 1, 100) == 0  # one chunk needs none


def _step(cls, **kw):
    if cls is L._LinearStepArgs:
        a = dict(x=P, input_gate=P, decay_gate=P, decay=P, state=P, rows=4, D=16, n_slots=4, decay_scale=8.0, dtype=0, y=P)
    else:
        a = dict(q=P, k=P, v=P, g=P, beta=P, state=P, rows=4, Hq=2, Hv=4, n_slots=4, K=128, V=128, scale=1.0, dtype=0, o=P)
    return cls(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(input_gate=None), ARG), (dict(decay_gate=None), ARG), (dict(decay=None), ARG), (dict(state=None), ARG),
    (dict(y=None), ARG), (dict(rows=-1), SHAPE), (dict(rows=65536, n_slots=1 << 20), SHAPE), (dict(n_slots=3), SHAPE),
    (dict(n_slots=-1, slots=P), SHAPE), (dict(D=0), SHAPE), (dict(dtype=5), DTYPE), (dict(decay_scale=0.0), ARG), (dict(x=P + 1), ALIGN),
    (dict(state=P + 2), ALIGN), (dict(slots=P + 1), ALIGN)])
def test_linear_step_refusals(lib, kw, code):
    assert _call(lib.gdr_linear_step, _step(L._LinearStepArgs, **kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(g=None), ARG), (dict(beta=None), ARG), (dict(state=None), ARG),
    (dict(o=None), ARG), (dict(rows=-1), SHAPE), (dict(rows=65536, n_slots=1 << 20), SHAPE), (dict(n_slots=3), SHAPE),
    (dict(n_slots=-1, slots=P), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=3), SHAPE), (dict(Hv=0), SHAPE), (dict(Hv=1 << 17), SHAPE),
    (dict(K=32), SHAPE), (dict(K=256), SHAPE), (dict(V=32), SHAPE), (dict(V=512), SHAPE), (dict(dtype=2), DTYPE), (dict(q=P + 1), ALIGN),
    (dict(state=P + 8), ALIGN), (dict(g=P + 2), ALIGN)])
def test_delta_step_refusals(lib, kw, code):
    assert _call(lib.gdr_delta_step, _step(L._DeltaStepArgs, **kw)) == code


def _block(**kw):
    a = dict(x=P, gate=P, residual=P, weight=P, next_weight=P, M=4, D=64, inner=1, x_outer=64, gate_outer=64, residual_outer=64, scale=1.0, eps=1e-6,
             dtype=0, r=P, y=P, stats=P, dr=P, dy=P, dx=P, dgate=P, dresidual=P, dweight=P, dnext_weight=P, workspace=P,
             workspace_bytes=1 << 40)
    return L._BlockNormArgs(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(weight=None), ARG), (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(D=0), SHAPE), (dict(D=16385), SHAPE),
    (dict(inner=0), SHAPE), (dict(inner=3), SHAPE), (dict(inner=1 << 31), SHAPE), (dict(dtype=9), DTYPE), (dict(x=P + 1), ALIGN), (dict(gate=P + 1), ALIGN), (dict(residual=P + 1), ALIGN), (dict(weight=P + 2), ALIGN),
    (dict(next_weight=P + 1), ALIGN), (dict(stats=P + 4), ALIGN)])
def test_block_norm_refusals(lib, kw, code):
    assert _call(lib.gdr_block_norm_fwd, _block(**kw)) == code
    assert _call(lib.gdr_block_norm_bwd, _block(**kw)) == code


@pytest.mark.parametrize("kw,code", [(dict(r=None), ARG), (dict(y=None), ARG), (dict(r=P + 1), ALIGN)])
def test_block_norm_forward_refusals(lib, kw, code):
    assert _call(lib.gdr_block_norm_fwd, _block(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(stats=None), ARG), (dict(dx=None), ARG), (dict(dgate=None), ARG), (dict(dresidual=None), ARG), (dict(dweight=None), ARG),
    (dict(dnext_weight=None), ARG), (dict(workspace=None), WORKSPACE), (dict(workspace=P + 4), ALIGN), (dict(workspace_bytes=64), WORKSPACE)])
def test_block_norm_backward_refusals(lib, kw, code):
    assert _call(lib.gdr_block_norm_bwd, _block(**kw)) == code


NAMES = ("linear_fwd", "linear_bwd", "linear_step", "delta_step", "block_norm_fwd", "block_norm_bwd")


def test_null_arguments(lib):
    for name in NAMES:
        assert getattr(lib, "gdr_" + name)(None, None) == ARG


def test_calls_without_tokens_return_without_a_launch(lib):
    assert _call(lib.gdr_linear_fwd, _linear(T=0, x=None, input_gate=None, decay_gate=None, z=None, y=None, workspace=None)) == 0
    assert _call(lib.gdr_linear_step, _step(L._LinearStepArgs, rows=0, x=None, input_gate=None, decay_gate=None, y=None)) == 0
    assert _call(lib.gdr_delta_step, _step(L._DeltaStepArgs, rows=0, q=None, k=None, v=None, g=None, beta=None, o=None)) == 0
    assert _call(lib.gdr_block_norm_fwd, _block(M=0, x=None, r=None, y=None)) == 0


x3, x2, vec = torch.zeros(1, 8, 16), torch.zeros(8, 16), torch.zeros(16)
heads, gates = torch.zeros(8, 2, 64), torch.zeros(8, 2)
CALLS = {
    "gated_linear_scan": (gdr.gated_linear_scan, [x3, x3, x3, vec, x3]),
    "gated_linear_step": (gdr.gated_linear_step, [x2, x2, x2, vec, x2, x2]),
    "gated_delta_step": (gdr.gated_delta_step, [heads, heads, heads, gates, gates, torch.zeros(8, 2, 64, 64)]),
    "gated_residual_rms_norm": (gdr.gated_residual_rms_norm, [x2, vec, x2, x2, vec]),
}


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_tangents_and_cpu_tensors_are_refused(name, grad):
    call, args = CALLS[name]
    with pytest.raises(gdr.GdrError, match="GPU"):
        call(*args)
    with forward_ad.dual_level():
        for i, t in enumerate(args):
            t = t.clone().requires_grad_(grad)
            with pytest.raises(gdr.GdrError, match="forward-mode"):
                call(*args[:i], forward_ad.make_dual(t, torch.ones_like(t)), *args[i + 1:])
