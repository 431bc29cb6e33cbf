"""The operators around a recurrent mixer (C ABI in ``include/gdr.h``, "Layer
operators"): argument checks and marshalling; every step runs in the library's
CUDA kernels.

* ``short_conv`` / ``short_conv_step``: depthwise causal convolution along the
  tokens (2 to 4 taps), over sequences and for one token of each;
* ``state_space_scan`` / ``state_space_step``: the selective state space scan;
* ``residual_rms_norm`` / ``residual_rms_norm_fp8``: root-mean-square norm of a
  residual stream, in the input's type or in 8 bits with scales;
* ``block_matmul_fp8``: product of 8-bit operands with a scale for each block
  of 128.

Activations are bf16 or fp32 ``[B, T, ...]`` (one token: ``[rows, ...]``) with
a contiguous innermost part; the strides between tokens and batch rows are
free, so that slices of a projection's output go in as they are.  Parameters
and recurrent states are fp32 (the convolution's state holds inputs, in their
type); the scan's A and states begin on 16-byte boundaries.  Packed sequences:
``cu_seqlens`` int32 on the GPU with ``B = 1``; its values are checked on the
device (``check_status``).  Work is enqueued on the current stream of the
inputs' device; nothing synchronises.  Reverse mode only: inputs with
forward-mode tangents are refused.
"""
from __future__ import annotations

import ctypes
import struct
from ctypes import c_float, c_int, c_longlong, c_size_t, c_void_p

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from .binding import GDR_BF16, GDR_F32, GdrError, load

__all__ = ["short_conv", "short_conv_step", "state_space_scan", "state_space_step", "residual_rms_norm",
           "residual_rms_norm_fp8", "block_matmul_fp8"]

STATE_STRIDE = 16  # GDR_SSM_STRIDE: tokens between the states kept for the backward
STATE_SIZES = (8, 16, 32, 64)

_DTYPES = {torch.bfloat16: GDR_BF16, torch.float32: GDR_F32}
_F32, _I32 = torch.float32, torch.int32
_empty = torch.empty


class _Args:
    """An argument struct of the C ABI: its ctypes class, and ``pack``, which lays all of its fields out at once
    (a call for one token is bound by the host; filling a ctypes structure takes twice as long)."""

    def __init__(self, name, spec):
        kinds = {"p": (c_void_p, "P"), "l": (c_longlong, "q"), "i": (c_int, "i"), "f": (c_float, "f"), "z": (c_size_t, "N")}
        fields = [(n, kinds[k]) for k, names in spec for n in names.split()]
        self.struct = type(name, (ctypes.Structure,), {"_fields_": [(n, k[0]) for n, k in fields]})
        form = struct.Struct("@" + "".join(k[1] for _, k in fields))
        self.pack = form.pack


_CONV = _Args("gdr_conv_args", [("p", "x weight bias h0 cu_seqlens"), ("l", "B T D n_seqs x_row x_batch"),
                                ("i", "W dtype silu"), ("p", "y ht dy dht dx dweight dbias dh0 workspace"),
                                ("z", "workspace_bytes")])
_CONV_STEP = _Args("gdr_conv_step_args", [("p", "x weight bias state slots"), ("l", "rows D n_slots x_row"),
                                          ("i", "W dtype silu"), ("p", "y")])
_SSM = _Args("gdr_ssm_args", [
    ("p", "x dt z Bm Cm A skip dt_bias h0 cu_seqlens"), ("l", "B T D G n_seqs"),
    ("l", "x_row x_batch dt_row dt_batch z_row z_batch b_row b_batch c_row c_batch"), ("i", "N dtype softplus"),
    ("p", "y ht states dy dht dx ddt dz dB dC dA dskip ddt_bias dh0 workspace"), ("z", "workspace_bytes")])
_SSM_STEP = _Args("gdr_ssm_step_args", [
    ("p", "x dt z Bm Cm A skip dt_bias state slots"), ("l", "rows D G n_slots x_row dt_row z_row b_row c_row"),
    ("i", "N dtype softplus"), ("p", "y")])
_NORM = _Args("gdr_norm_args", [("p", "x residual weight"), ("l", "M D x_row r_row"), ("f", "eps"), ("i", "dtype"),
                                ("p", "sum y q scales")])
_NORM_BWD = _Args("gdr_norm_bwd_args", [("p", "r dy dsum weight"), ("l", "M D"), ("f", "eps"), ("i", "dtype"),
                                        ("p", "dr dweight workspace"), ("z", "workspace_bytes")])
_FP8 = _Args("gdr_fp8_args", [("p", "a b a_scales b_scales"), ("l", "M N K"), ("i", "out_dtype"), ("p", "out")])
_ConvArgs, _ConvStepArgs, _SsmArgs, _SsmStepArgs, _NormArgs, _NormBwdArgs, _Fp8Args = (
    v.struct for v in (_CONV, _CONV_STEP, _SSM, _SSM_STEP, _NORM, _NORM_BWD, _FP8))

_lib = None


def _calls():
    global _lib
    if _lib is None:
        lib = load()
        for name in ("conv_fwd", "conv_bwd", "conv_step", "ssm_fwd", "ssm_bwd", "ssm_step", "norm_fwd", "norm_bwd",
                     "fp8_matmul"):
            f = getattr(lib, "gdr_" + name)
            f.argtypes, f.restype = [c_void_p, c_void_p], c_int
        for name, kinds in (("conv_bwd", [c_longlong] * 3 + [c_int]), ("ssm_fwd", [c_void_p]), ("ssm_bwd", [c_void_p]),
                            ("norm_bwd", [c_longlong] * 2)):
            f = getattr(lib, f"gdr_{name}_workspace_size")
            f.argtypes, f.restype = kinds, c_size_t
        _lib = lib
    return _lib


_current_device = torch.cuda.current_device
# The current stream's handle without building a Stream object, where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _run(call, args, dev):
    if dev != _current_device():
        with torch.cuda.device(dev):
            rc = call(args, _raw_stream(dev))
    else:
        rc = call(args, _raw_stream(dev))
    if rc:
        raise GdrError(rc, load().gdr_last_error().decode())


def _fail(code, msg):
    raise GdrError(code, msg)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _inputs(name, t):
    """A call's first input: its GPU and its type's code."""
    dev = t.get_device()
    if dev < 0:
        _fail(1, f"{name} must live on the GPU")
    code = _DTYPES.get(t.dtype)
    if code is None:
        _fail(3, f"{name}: unsupported dtype {t.dtype}")
    if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
        _fail(1, f"{name} must be contiguous along its last dimension")
    return dev, code


def _like(name, t, dev, dtype, shape):
    """Another activation of the call."""
    if t.get_device() == dev and t.dtype is dtype and t.shape == shape and (t.stride(-1) == 1 or t.shape[-1] <= 1):
        return
    if t.get_device() != dev:
        _fail(1, f"{name} must live on the GPU of the first input")
    if t.dtype != dtype:
        _fail(3, f"{name} must have the first input's dtype ({dtype}, got {t.dtype})")
    if t.shape != shape:
        _fail(2, f"{name} must be {tuple(shape)} (got {tuple(t.shape)})")
    _fail(1, f"{name} must be contiguous along its last dimension")


def _param(name, t, dev, shape, dtype=_F32):
    """A parameter, state or table: contiguous, of one type and shape."""
    if t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return
    if t.get_device() != dev:
        _fail(1, f"{name} must live on the GPU of the first input")
    if t.dtype != dtype:
        _fail(3, f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        _fail(2, f"{name} must be {tuple(shape)} (got {tuple(t.shape)})")
    _fail(1, f"{name} must be contiguous")


def _sequences(x, dev, cu_seqlens):
    if cu_seqlens is None:
        return x.shape[0]
    if cu_seqlens.get_device() != dev or not cu_seqlens.is_contiguous():
        _fail(1, "cu_seqlens must be contiguous and live on the GPU of the first input")
    if cu_seqlens.dtype != _I32:
        _fail(3, "cu_seqlens must be int32")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2 or x.shape[0] != 1:
        _fail(2, "packed sequences need B == 1 and cu_seqlens [n_seqs + 1]")
    return cu_seqlens.shape[0] - 1


def _slots(slots, dev, rows, n_slots):
    if slots is not None:
        _param("slots", slots, dev, (rows,), _I32)
    elif n_slots < rows:
        _fail(2, f"{n_slots} state slots for {rows} rows")


def _wants_grad(*ts):
    if torch.is_grad_enabled():
        for t in ts:
            if t is not None and t.requires_grad:
                return True
    return False


def _no_tangents(name, *ts):
    """Forward-mode derivatives are refused rather than dropped: a call without ``requires_grad`` meets no autograd."""
    if getattr(forward_ad, "_current_level", 0) >= 0:  # inside a dual level (asked at every call, so cheaply)
        for t in ts:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                _fail(1, f"{name} has no forward-mode derivative: detach its inputs or use reverse mode")


def _grad(g, like):
    """An incoming gradient as the kernels read it."""
    if g is None or (g.dtype is like.dtype and g.is_contiguous()):
        return g
    return g.to(like.dtype).contiguous()


def _once():
    if torch.is_grad_enabled():
        _fail(1, "the gradient of this operator is not differentiable itself")


# ---- short convolution ------------------------------------------------------


def _activation(activation):
    if activation not in ("silu", None):
        _fail(1, f"activation must be 'silu' or None (got {activation!r})")
    return 1 if activation else 0


def _conv_check(x, weight, bias, initial_state, cu_seqlens):
    dev, code = _inputs("x", x)
    if x.dim() != 3:
        _fail(2, f"x must be [B, T, D] (got {tuple(x.shape)})")
    n, d = _sequences(x, dev, cu_seqlens), x.shape[2]
    if weight.dim() != 2:
        _fail(2, f"weight must be [D, W] (got {tuple(weight.shape)})")
    w = weight.shape[1]
    _param("weight", weight, dev, (d, w))
    if bias is not None:
        _param("bias", bias, dev, (d,))
    if initial_state is not None:
        _param("initial_state", initial_state, dev, (n, w - 1, d), x.dtype)
    return dev, code, n, w


def _conv_fwd(x, weight, bias, silu, initial_state, output_final_state, cu_seqlens):
    dev, code, n, w = _conv_check(x, weight, bias, initial_state, cu_seqlens)
    b, t, d = x.shape
    y = _empty((b, t, d), dtype=x.dtype, device=x.device)
    ht = _empty((n, w - 1, d), dtype=x.dtype, device=x.device) if output_final_state and w > 1 else None
    row = x.stride()
    _run(_calls().gdr_conv_fwd,
         _CONV.pack(x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(initial_state), _ptr(cu_seqlens), b, t, d, n, row[1],
                    row[0], w, code, silu, y.data_ptr(), _ptr(ht), 0, 0, 0, 0, 0, 0, 0, 0), dev)
    return y, ht


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, silu, initial_state, output_final_state, cu_seqlens):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.silu = silu
        return _conv_fwd(x, weight, bias, silu, initial_state, output_final_state, cu_seqlens)

    @staticmethod
    def backward(ctx, dy, dht):
        _once()
        x, weight, bias, initial_state, cu_seqlens = ctx.saved_tensors
        (b, t, d), w, dev = x.shape, weight.shape[1], x.device
        n = b if cu_seqlens is None else cu_seqlens.shape[0] - 1
        dy = torch.zeros((b, t, d), dtype=x.dtype, device=dev) if dy is None else _grad(dy, x)
        dht = _grad(dht, x)
        dx = _empty((b, t, d), dtype=x.dtype, device=dev)
        dweight = _empty((d, w), dtype=_F32, device=dev)
        dbias = None if bias is None else _empty((d,), dtype=_F32, device=dev)
        dh0 = None if initial_state is None else _empty(initial_state.shape, dtype=x.dtype, device=dev)
        lib = _calls()
        size = lib.gdr_conv_bwd_workspace_size(b, t, d, w)
        ws = _empty(size, dtype=torch.uint8, device=dev)
        row = x.stride()
        _run(lib.gdr_conv_bwd,
             _CONV.pack(x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(initial_state), _ptr(cu_seqlens), b, t, d, n, row[1],
                        row[0], w, _DTYPES[x.dtype], ctx.silu, 0, 0, dy.data_ptr(), _ptr(dht), dx.data_ptr(),
                        dweight.data_ptr(), _ptr(dbias), _ptr(dh0), ws.data_ptr(), size), x.get_device())
        return dx, dweight, dbias, None, dh0, None, None


def short_conv(x, weight, bias=None, activation="silu", initial_state=None, output_final_state=False, cu_seqlens=None):
    """y_t = act(bias + sum_j weight[:, j] x_{t - W + 1 + j}) for every sequence and channel.

    x [B, T, D]; weight [D, W] fp32, W in 2..4; bias [D] fp32; initial_state [N, W - 1, D] in x's dtype, the inputs
    before each sequence, oldest first (zeros when absent).  Returns (y [B, T, D], final_state [N, W - 1, D] or None);
    differentiable in x, weight, bias and initial_state."""
    silu = _activation(activation)
    _no_tangents("short_conv", x, weight, bias, initial_state)
    if _wants_grad(x, weight, bias, initial_state):
        return _ShortConv.apply(x, weight, bias, silu, initial_state, bool(output_final_state), cu_seqlens)
    return _conv_fwd(x, weight, bias, silu, initial_state, output_final_state, cu_seqlens)


def short_conv_step(x, weight, state, bias=None, activation="silu", slots=None):
    """One token of every row: x [rows, D]; state [n_slots, W - 1, D] in x's dtype, updated in place; slots [rows]
    int32 names each row's state (row r uses slot r when absent), a negative one an idle row whose y is zero.
    Returns y [rows, D].  No gradient."""
    silu = _activation(activation)
    _no_tangents("short_conv_step", x, weight, state, bias)
    dev, code = _inputs("x", x)
    if x.dim() != 2 or weight.dim() != 2 or state.dim() != 3:
        _fail(2, "x must be [rows, D], weight [D, W] and state [n_slots, W - 1, D]")
    (rows, d), w, n = x.shape, weight.shape[1], state.shape[0]
    _param("weight", weight, dev, (d, w))
    _param("state", state, dev, (n, w - 1, d), x.dtype)
    if bias is not None:
        _param("bias", bias, dev, (d,))
    _slots(slots, dev, rows, n)
    if _wants_grad(x, weight, bias, state):
        _fail(1, "short_conv_step has no gradient: call it under torch.no_grad() or detach its inputs")
    y = _empty((rows, d), dtype=x.dtype, device=x.device)
    _run(_calls().gdr_conv_step,
         _CONV_STEP.pack(x.data_ptr(), weight.data_ptr(), _ptr(bias), state.data_ptr(), _ptr(slots), rows, d, n, x.stride(0),
                         w, code, silu, y.data_ptr()), dev)
    increment_version(state)  # as torch's own in-place operations: a backward that saved it raises
    return y


# ---- selective state space scan ---------------------------------------------


def _ssm_check(x, dt, A, B, C, D, z, dt_bias, lead):
    """Shapes of the scan (lead 2: [B, T, ...]) and of its step (lead 1: [rows, ...])."""
    dev, code = _inputs("x", x)
    shape, dtype = x.shape, x.dtype
    if len(shape) != lead + 1:
        _fail(2, f"x must be {'[B, T, D]' if lead == 2 else '[rows, D]'} (got {tuple(shape)})")
    d = shape[-1]
    if A.dim() != 2 or B.dim() != lead + 2:
        _fail(2, f"A must be [D, N] and B {'[B, T, G, N]' if lead == 2 else '[rows, G, N]'}")
    n, g = A.shape[1], B.shape[-2]
    if n not in STATE_SIZES:
        _fail(2, f"N must be one of {STATE_SIZES} (got {n})")
    if g < 1 or d % g:
        _fail(2, f"D ({d}) must be a multiple of G ({g})")
    _param("A", A, dev, (d, n))
    _like("dt", dt, dev, dtype, shape)
    inner = (*shape[:lead], g, n)
    _like("B", B, dev, dtype, inner)
    _like("C", C, dev, dtype, inner)
    if g > 1 and not B.stride(-2) == C.stride(-2) == n:
        _fail(1, "B and C must be contiguous over their last two dimensions")
    if z is not None:
        _like("z", z, dev, dtype, shape)
    if D is not None:
        _param("D", D, dev, (d,))
    if dt_bias is not None:
        _param("dt_bias", dt_bias, dev, (d,))
    return dev, code, d, n, g


def _ssm_head(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, cu_seqlens, n_seqs, code):
    """The first 28 fields of the scan's arguments: inputs, sizes, strides, kinds."""
    b, t, d = x.shape
    xs, ds, bs, cs = x.stride(), dt.stride(), B.stride(), C.stride()
    zs = (0, 0) if z is None else z.stride()
    return (x.data_ptr(), dt.data_ptr(), _ptr(z), B.data_ptr(), C.data_ptr(), A.data_ptr(), _ptr(D), _ptr(dt_bias),
            _ptr(initial_state), _ptr(cu_seqlens), b, t, d, B.shape[2], n_seqs, xs[1], xs[0], ds[1], ds[0], zs[1], zs[0],
            bs[1], bs[0], cs[1], cs[0], A.shape[1], code, softplus)


def _scan_fwd(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, output_final_state, cu_seqlens, keep):
    dev, code, d, n, _ = _ssm_check(x, dt, A, B, C, D, z, dt_bias, 2)
    n_seqs = _sequences(x, dev, cu_seqlens)
    if initial_state is not None:
        _param("initial_state", initial_state, dev, (n_seqs, d, n))
    b, t, where = x.shape[0], x.shape[1], x.device
    y = _empty((b, t, d), dtype=x.dtype, device=where)
    ht = _empty((n_seqs, d, n), dtype=_F32, device=where) if output_final_state else None
    states = _empty((b, -(-t // STATE_STRIDE), d, n), dtype=_F32, device=where) if keep else None
    head = _ssm_head(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, cu_seqlens, n_seqs, code)
    out = (y.data_ptr(), _ptr(ht), _ptr(states), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    lib = _calls()
    size = lib.gdr_ssm_fwd_workspace_size(_SSM.pack(*head, *out, 0, 0))
    ws = _empty(size, dtype=torch.uint8, device=where) if size else None
    _run(lib.gdr_ssm_fwd, _SSM.pack(*head, *out, _ptr(ws), size), dev)
    return y, ht, states


class _StateSpaceScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, output_final_state, cu_seqlens):
        ctx.set_materialize_grads(False)
        y, ht, states = _scan_fwd(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, output_final_state, cu_seqlens,
                                  True)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, states)
        ctx.softplus = softplus
        return y, ht

    @staticmethod
    def backward(ctx, dy, dht):
        _once()
        x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, states = ctx.saved_tensors
        where = x.device
        n_seqs = x.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
        dy = torch.zeros(x.shape, dtype=x.dtype, device=where) if dy is None else _grad(dy, x)
        dht = _grad(dht, A)
        if dht is not None and dht.data_ptr() % 16:  # states are read sixteen bytes at a time
            dht = dht.clone()
        new = lambda like: None if like is None else _empty(like.shape, dtype=like.dtype, device=where)  # noqa: E731
        dx, ddt, dA, dB, dC, dD, dz, db, dh0 = (new(v) for v in (x, dt, A, B, C, D, z, dt_bias, initial_state))
        head = _ssm_head(x, dt, A, B, C, D, z, dt_bias, ctx.softplus, initial_state, cu_seqlens, n_seqs, _DTYPES[x.dtype])
        out = (0, 0, states.data_ptr(), dy.data_ptr(), _ptr(dht), dx.data_ptr(), ddt.data_ptr(), _ptr(dz), dB.data_ptr(),
               dC.data_ptr(), dA.data_ptr(), _ptr(dD), _ptr(db), _ptr(dh0))
        lib = _calls()
        size = lib.gdr_ssm_bwd_workspace_size(_SSM.pack(*head, *out, 0, 0))
        ws = _empty(size, dtype=torch.uint8, device=where) if size else None
        _run(lib.gdr_ssm_bwd, _SSM.pack(*head, *out, _ptr(ws), size), x.get_device())
        return dx, ddt, dA, dB, dC, dD, dz, db, None, dh0, None, None


def state_space_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, initial_state=None,
                     output_final_state=False, cu_seqlens=None):
    """For every sequence and channel d of group g = d // (D / G), with s_t = softplus(dt_t + dt_bias) (dt_t + dt_bias
    without ``dt_softplus``):

        h_t = exp(s_t A) h_{t-1} + s_t x_t B_t,    y_t = (C_t . h_t + D x_t) silu(z_t).

    x, dt, z [B, T, D]; B, C [B, T, G, N]; A [D, N], D and dt_bias [D] fp32; initial_state [n_seqs, D, N] fp32 (zeros
    when absent); N in 8, 16, 32, 64.  Without z there is no gate, without D no skip.  Returns (y [B, T, D],
    final_state [n_seqs, D, N] fp32 or None); differentiable in every tensor but cu_seqlens.

    The backward's workspace, held for the call, is 8 N bytes a token for every 512 / N channels of a group (16 KiB a
    token at D = 4096, N = 16, one group; 256 KiB at N = 64), and a forward that keeps a gradient's states D N / 4 bytes
    a token."""
    softplus = 1 if dt_softplus else 0
    _no_tangents("state_space_scan", x, dt, A, B, C, D, z, dt_bias, initial_state)
    if _wants_grad(x, dt, A, B, C, D, z, dt_bias, initial_state):
        return _StateSpaceScan.apply(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, bool(output_final_state),
                                     cu_seqlens)
    return _scan_fwd(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, output_final_state, cu_seqlens, False)[:2]


def state_space_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus=True, slots=None):
    """One token of every row: x, dt, z [rows, D]; B, C [rows, G, N]; state [n_slots, D, N] fp32, updated in place;
    slots as in ``short_conv_step``.  Returns y [rows, D].  No gradient."""
    _no_tangents("state_space_step", x, dt, A, B, C, state, D, z, dt_bias)
    dev, code, d, n, g = _ssm_check(x, dt, A, B, C, D, z, dt_bias, 1)
    rows, n_slots = x.shape[0], state.shape[0]
    _param("state", state, dev, (n_slots, d, n))
    _slots(slots, dev, rows, n_slots)
    if _wants_grad(x, dt, A, B, C, D, z, dt_bias, state):
        _fail(1, "state_space_step has no gradient: call it under torch.no_grad() or detach its inputs")
    y = _empty((rows, d), dtype=x.dtype, device=x.device)
    _run(_calls().gdr_ssm_step,
         _SSM_STEP.pack(x.data_ptr(), dt.data_ptr(), _ptr(z), B.data_ptr(), C.data_ptr(), A.data_ptr(), _ptr(D), _ptr(dt_bias),
                        state.data_ptr(), _ptr(slots), rows, d, g, n_slots, x.stride(0), dt.stride(0),
                        0 if z is None else z.stride(0), B.stride(0), C.stride(0), n, code, 1 if dt_softplus else 0,
                        y.data_ptr()), dev)
    increment_version(state)
    return y


# ---- norm of the residual stream --------------------------------------------


def _rows(name, t, d):
    """[..., D] as rows of one stride."""
    if t.dim() == 2:
        return t
    try:
        return t.view(-1, d)
    except RuntimeError:
        _fail(1, f"{name} must be rows of one stride")


def _norm_fwd(x, weight, residual, eps, quantise):
    dev, code = _inputs("x", x)
    shape, where = x.shape, x.device
    if not shape or shape[-1] < 1:
        _fail(2, f"x must be [..., D] (got {tuple(shape)})")
    d = shape[-1]
    _param("weight", weight, dev, (d,))
    x2 = _rows("x", x, d)
    m, out, res, row = x2.shape[0], x, 0, 0
    if residual is not None:
        _like("residual", residual, dev, x.dtype, shape)
        r2 = _rows("residual", residual, d)
        res, row = r2.data_ptr(), r2.stride(0)
        out = _empty(shape, dtype=x.dtype, device=where)
    if quantise:
        y = _empty(shape, dtype=torch.float8_e4m3fn, device=where)
        scales = _empty((-(-d // 128), m), dtype=_F32, device=where)
        to = (0, y.data_ptr(), scales.data_ptr())
    else:
        y, scales = _empty(shape, dtype=x.dtype, device=where), None
        to = (y.data_ptr(), 0, 0)
    _run(_calls().gdr_norm_fwd,
         _NORM.pack(x2.data_ptr(), res, weight.data_ptr(), m, d, x2.stride(0), row, eps, code, out.data_ptr() if res else 0, *to),
         dev)
    return y, scales, out


class _ResidualRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        y, _, out = _norm_fwd(x, weight, residual, eps, False)
        ctx.eps, ctx.added = eps, residual is not None
        ctx.save_for_backward(out, weight)
        # without a residual the stream is x: handed out here all the same, so that its gradient is added in the kernel
        return y, out if ctx.added else x.view_as(x)

    @staticmethod
    def backward(ctx, dy, dsum):
        _once()
        r, weight = ctx.saved_tensors
        shape, where = r.shape, r.device
        d = shape[-1]
        m = r.numel() // d
        dy = torch.zeros(shape, dtype=r.dtype, device=where) if dy is None else _grad(dy, r)
        dsum = _grad(dsum, r)
        r = r.contiguous()
        dr = _empty(shape, dtype=r.dtype, device=where)
        dweight = _empty((d,), dtype=_F32, device=where)
        lib = _calls()
        size = lib.gdr_norm_bwd_workspace_size(m, d)
        ws = _empty(size, dtype=torch.uint8, device=where)
        _run(lib.gdr_norm_bwd,
             _NORM_BWD.pack(r.data_ptr(), dy.data_ptr(), _ptr(dsum), weight.data_ptr(), m, d, ctx.eps, _DTYPES[r.dtype],
                            dr.data_ptr(), dweight.data_ptr(), ws.data_ptr(), size), r.get_device())
        return dr, dweight, dr if ctx.added else None, None


def residual_rms_norm(x, weight, residual=None, eps=1e-6):
    """r = x + residual (rounded to x's dtype), y = r / sqrt(mean(r^2) + eps) * weight over the last dimension.

    x, residual [..., D]; weight [D] fp32; D at most 16384.  Returns (y, r); r is x itself without a residual.
    Differentiable in x, weight and residual, through y and r."""
    _no_tangents("residual_rms_norm", x, weight, residual)
    if _wants_grad(x, weight, residual):
        return _ResidualRmsNorm.apply(x, weight, residual, float(eps))
    y, _, r = _norm_fwd(x, weight, residual, eps, False)
    return y, r


def residual_rms_norm_fp8(x, weight, residual=None, eps=1e-6):
    """The same norm written in 8 bits: returns (q, scales, r) with q [..., D] float8_e4m3fn, scales
    [ceil(D / 128), M] fp32 (M rows) and y = q * scale of its row and block of 128 channels; a block's scale is
    max(max|y|, 1e-30) / 448.  What ``block_matmul_fp8`` reads.  No gradient."""
    _no_tangents("residual_rms_norm_fp8", x, weight, residual)
    if _wants_grad(x, weight, residual):
        _fail(1, "residual_rms_norm_fp8 has no gradient: call it under torch.no_grad() or use residual_rms_norm")
    return _norm_fwd(x, weight, residual, eps, True)


# ---- block-scaled 8-bit product ----------------------------------------------


def block_matmul_fp8(a, a_scales, b, b_scales, out_dtype=torch.bfloat16):
    """out[m, n] = sum over blocks k of 128 of a_scales[k, m] b_scales[n // 128, k] (a_k[m] . b_k[n]), summed in fp32.

    a [..., K] (M rows) and b [N, K] float8_e4m3fn, contiguous, N at least 1 and K a positive multiple of 16; a_scales
    [ceil(K / 128), M] and b_scales [ceil(N / 128), ceil(K / 128)] fp32; out_dtype bf16 or fp32.  Returns out [..., N].
    No gradient."""
    _no_tangents("block_matmul_fp8", a_scales, b_scales)
    f8, dev = torch.float8_e4m3fn, a.get_device()
    if dev < 0:
        _fail(1, "a must live on the GPU")
    if a.dim() < 1 or b.dim() != 2:
        _fail(2, f"a must be [..., K] and b [N, K] (got {tuple(a.shape)}, {tuple(b.shape)})")
    lead, k, n = a.shape[:-1], a.shape[-1], b.shape[0]
    m, blocks = lead.numel(), -(-k // 128)
    _param("a", a, dev, a.shape, f8)
    _param("b", b, dev, (n, k), f8)
    _param("a_scales", a_scales, dev, (blocks, m))
    _param("b_scales", b_scales, dev, (-(-n // 128), blocks))
    code = _DTYPES.get(out_dtype)
    if code is None:
        _fail(3, f"out_dtype must be torch.bfloat16 or torch.float32 (got {out_dtype})")
    if _wants_grad(a_scales, b_scales):
        _fail(1, "block_matmul_fp8 has no gradient: call it under torch.no_grad()")
    out = _empty((*lead, n), dtype=out_dtype, device=a.device)
    _run(_calls().gdr_fp8_matmul,
         _FP8.pack(a.data_ptr(), b.data_ptr(), a_scales.data_ptr(), b_scales.data_ptr(), m, n, k, code, out.data_ptr()), dev)
    return out
