"""What the layer operators refuse, without a GPU: through the C ABI (codes,
nothing launched) and through the Python calls."""
import ctypes

import pytest
import torch

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


def _conv(**kw):
    a = dict(x=P, weight=P, bias=P, y=P, B=1, T=8, D=16, n_seqs=1, x_row=16, x_batch=128, W=4, dtype=0, silu=1,
             dy=P, dx=P, dweight=P, dbias=P, workspace=P, workspace_bytes=1 << 30)
    return L._ConvArgs(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(weight=None), ARG), (dict(B=0), SHAPE), (dict(T=-1), SHAPE), (dict(D=0), SHAPE),
    (dict(W=1), SHAPE), (dict(W=5), SHAPE), (dict(T=1 << 30), SHAPE), (dict(dtype=7), DTYPE), (dict(n_seqs=2), SHAPE),
    (dict(cu_seqlens=P, n_seqs=0), SHAPE), (dict(cu_seqlens=P, B=2), SHAPE), (dict(x=P + 1), ALIGN), (dict(weight=P + 2), ALIGN)])
def test_conv_refusals(lib, kw, code):
    assert _call(lib.gdr_conv_fwd, _conv(**kw)) == code
    assert _call(lib.gdr_conv_bwd, _conv(**kw)) == code
    assert lib.gdr_last_error()


@pytest.mark.parametrize("kw,code", [(dict(y=None), ARG), (dict(y=P + 1), ALIGN)])
def test_conv_forward_refusals(lib, kw, code):
    assert _call(lib.gdr_conv_fwd, _conv(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), ARG), (dict(dx=None), ARG), (dict(dweight=None), ARG), (dict(workspace=None), WORKSPACE),
    (dict(workspace=P + 4), ALIGN), (dict(workspace_bytes=15), WORKSPACE)])
def test_conv_backward_refusals(lib, kw, code):
    assert _call(lib.gdr_conv_bwd, _conv(**kw)) == code


def _ssm(**kw):
    rows = {n + s: 64 for n in ("x", "dt", "z", "b", "c") for s in ("_row", "_batch")}
    a = dict(x=P, dt=P, z=P, Bm=P, Cm=P, A=P, skip=P, dt_bias=P, B=1, T=64, D=64, G=1, n_seqs=1, N=16, dtype=0, softplus=1,
             y=P, states=P, dy=P, dx=P, ddt=P, dz=P, dB=P, dC=P, dA=P, dskip=P, ddt_bias=P, workspace=P,
             workspace_bytes=1 << 40, **rows)
    return L._SsmArgs(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(dt=None), ARG), (dict(Bm=None), ARG), (dict(A=None), ARG), (dict(G=0), SHAPE), (dict(G=3), SHAPE),
    (dict(N=12), SHAPE), (dict(N=128), SHAPE), (dict(dtype=2), DTYPE), (dict(n_seqs=3), SHAPE), (dict(B=70000), SHAPE),
    (dict(cu_seqlens=P, n_seqs=0), SHAPE), (dict(A=P + 4), ALIGN), (dict(x=P + 1), ALIGN), (dict(h0=P + 8), ALIGN)])
def test_scan_refusals(lib, kw, code):
    assert _call(lib.gdr_ssm_fwd, _ssm(**kw)) == code
    assert _call(lib.gdr_ssm_bwd, _ssm(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), ARG), (dict(states=None), ARG), (dict(dz=None), ARG), (dict(dskip=None), ARG), (dict(ddt_bias=None), ARG),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=16), WORKSPACE), (dict(workspace=P + 8), ALIGN)])
def test_scan_backward_refusals(lib, kw, code):
    assert _call(lib.gdr_ssm_bwd, _ssm(**kw)) == code


def test_scan_workspace_sizes(lib):
    one = _ssm(T=1, workspace=None, workspace_bytes=0)
    assert lib.gdr_ssm_fwd_workspace_size(ctypes.byref(one)) == 0  # one segment needs none
    assert lib.gdr_ssm_bwd_workspace_size(ctypes.byref(one)) > 0
    long = _ssm(T=1 << 16)
    need = lib.gdr_ssm_fwd_workspace_size(ctypes.byref(long))
    assert need > 0
    assert _call(lib.gdr_ssm_fwd, _ssm(T=1 << 16, workspace_bytes=need - 1)) == WORKSPACE
    assert lib.gdr_ssm_fwd_workspace_size(ctypes.byref(_ssm(N=12))) == 0


def _step(cls, **kw):
    a = dict(x=P, state=P, rows=4, D=16, n_slots=4, y=P, x_row=16, dtype=0)
    more = dict(weight=P, W=4, silu=1) if cls is L._ConvStepArgs else dict(dt=P, Bm=P, Cm=P, A=P, G=1, N=16, softplus=1, dt_row=16, b_row=16, c_row=16)
    return cls(**{**a, **more, **kw})


@pytest.mark.parametrize("cls,name", [(L._ConvStepArgs, "gdr_conv_step"), (L._SsmStepArgs, "gdr_ssm_step")])
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(state=None), ARG), (dict(y=None), ARG), (dict(rows=-1), SHAPE), (dict(rows=70000, n_slots=70000), SHAPE),
    (dict(n_slots=3), SHAPE), (dict(n_slots=-1, slots=P), SHAPE), (dict(D=0), SHAPE), (dict(dtype=5), DTYPE), (dict(x=P + 1), ALIGN)])
def test_step_refusals(lib, cls, name, kw, code):
    assert _call(getattr(lib, name), _step(cls, **kw)) == code


def _norm(**kw):
    return L._NormArgs(**{**dict(x=P, residual=P, weight=P, M=4, D=64, x_row=64, r_row=64, eps=1e-6, dtype=0, sum=P, y=P), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(weight=None), ARG), (dict(sum=None), ARG), (dict(y=None), ARG), (dict(q=P), ARG),
    (dict(y=None, q=P), ARG), (dict(M=-1), SHAPE), (dict(D=0), SHAPE), (dict(D=16385), SHAPE), (dict(dtype=9), DTYPE), (dict(x=P + 1), ALIGN)])
def test_norm_refusals(lib, kw, code):
    assert _call(lib.gdr_norm_fwd, _norm(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(r=None), ARG), (dict(dy=None), ARG), (dict(dr=None), ARG), (dict(dweight=None), ARG), (dict(D=20000), SHAPE),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=8), WORKSPACE)])
def test_norm_backward_refusals(lib, kw, code):
    a = dict(r=P, dy=P, weight=P, M=4, D=64, eps=1e-6, dtype=0, dr=P, dweight=P, workspace=P, workspace_bytes=1 << 30)
    assert _call(lib.gdr_norm_bwd, L._NormBwdArgs(**{**a, **kw})) == code


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), ARG), (dict(b=None), ARG), (dict(a_scales=None), ARG), (dict(b_scales=None), ARG), (dict(out=None), ARG),
    (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(K=24), SHAPE), (dict(out_dtype=3), DTYPE), (dict(a=P + 8), ALIGN)])
def test_matmul_refusals(lib, kw, code):
    a = dict(a=P, b=P, a_scales=P, b_scales=P, M=4, N=8, K=32, out_dtype=0, out=P)
    assert _call(lib.gdr_fp8_matmul, L._Fp8Args(**{**a, **kw})) == code


def test_null_arguments(lib):
    for name in ("conv_fwd", "conv_bwd", "conv_step", "ssm_fwd", "ssm_bwd", "ssm_step", "norm_fwd", "norm_bwd", "fp8_matmul"):
        assert getattr(lib, "gdr_" + name)(None, None) == ARG


def test_calls_without_tokens_return_without_a_launch(lib):
    assert _call(lib.gdr_conv_fwd, _conv(T=0, x=None, y=None)) == 0
    assert _call(lib.gdr_conv_step, _step(L._ConvStepArgs, rows=0, x=None, y=None)) == 0
    assert _call(lib.gdr_ssm_step, _step(L._SsmStepArgs, rows=0, x=None, y=None, dt=None, Bm=None, Cm=None)) == 0
    assert _call(lib.gdr_norm_fwd, _norm(M=0)) == 0
    a = L._Fp8Args(b=P, b_scales=P, M=0, N=8, K=32)
    assert _call(lib.gdr_fp8_matmul, a) == 0


def test_python_calls_refuse_cpu_tensors_and_bad_arguments(lib):
    x = torch.zeros(1, 8, 16)
    w = torch.zeros(16, 4)
    for call in (lambda: gdr.short_conv(x, w), lambda: gdr.short_conv_step(x[0], w, torch.zeros(8, 3, 16)),
                 lambda: gdr.state_space_scan(x, x, torch.zeros(16, 16), torch.zeros(1, 8, 1, 16), torch.zeros(1, 8, 1, 16)),
                 lambda: gdr.state_space_step(x[0], x[0], torch.zeros(16, 16), torch.zeros(8, 1, 16), torch.zeros(8, 1, 16), torch.zeros(8, 16, 16)),
                 lambda: gdr.residual_rms_norm(x, torch.zeros(16)), lambda: gdr.residual_rms_norm_fp8(x, torch.zeros(16)),
                 lambda: gdr.block_matmul_fp8(x[0], x[0], x[0], x[0])):
        with pytest.raises(gdr.GdrError):
            call()
    with pytest.raises(gdr.GdrError):
        gdr.short_conv(x, w, activation="relu")
