"""The operators around the delta rule in a token mixer: short causal convolution, selective
state space, per-head q/k norm with rotation, and the delta rule for single tokens.

Marshalling only, as in ``api``: descriptors from torch tensors, outputs and scratch from
PyTorch's allocator, torch's current stream (or ``stream``, which outputs and scratch then belong
to as well).  Device tensors only.  Layouts and formulas are those of include/gdr.h.
"""
from __future__ import annotations

import ctypes
import functools
import struct
import threading
from typing import Optional, Tuple

import torch

from . import _native as nat

_DT = {torch.bfloat16: nat.GDR_BF16, torch.float32: nat.GDR_F32}
_ACT = {None: 0, "none": 0, "silu": 1}
_NORM = {"rms": 0, "l2": 1}

# Calls of one token cost a few microseconds on the GPU, so the marshalling is kept short: the
# stream's handle comes without a Stream object, and descriptors are packed into one buffer for
# each thread (the library reads them during the call only).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice

# a gdr_tensor_t (56 bytes: address, type, rank, extents, strides' address), then its strides
_COMPACT = [struct.Struct("@Qii%dq%dxQ" % (n, 8 * (4 - n))) for n in range(5)]
_STRIDED = [struct.Struct("@Qii%dq%dxQ%dq" % (n, 8 * (4 - n), n)) for n in range(5)]
_SIZE, _MOST = 96, 24


class _Buffer(threading.local):
    def __init__(self):
        self.buf = (ctypes.c_char * (_SIZE * _MOST))()
        self.base = ctypes.addressof(self.buf)


_local = _Buffer()


def _descs(index: int, *tensors):
    """Addresses of descriptors of the tensors (None for None), valid until the thread's next
    call.  All tensors must be on CUDA device ``index``."""
    buf, base = _local.buf, _local.base
    at = []
    off = 0
    for t in tensors:
        if t is None:
            at.append(None)
            continue
        if t.get_device() != index:
            raise ValueError("tensors must be on one CUDA device")
        code = _DT.get(t.dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {t.dtype}")
        shape = t.shape
        n = len(shape)
        if n < 1 or n > 4:
            raise ValueError("tensors must have 1..4 dims")
        if t.is_contiguous():
            _COMPACT[n].pack_into(buf, off, t.data_ptr(), code, n, *shape, 0)
        else:
            _STRIDED[n].pack_into(buf, off, t.data_ptr(), code, n, *shape, base + off + 56,
                                  *t.stride())
        at.append(base + off)
        off += _SIZE
    return at


def _device_call(f):
    """Runs f with its first tensor's device current and, where ``stream`` is given, with that
    stream current too, so that what the call allocates belongs to it."""

    name = f.__code__.co_varnames[0]

    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        index = (args[0] if args else kw[name]).get_device()
        if index < 0:
            raise ValueError("tensors must be on a CUDA device")
        if stream is not None:
            with torch.cuda.stream(stream):
                return f(*args, **kw)
        if index != _current_device():
            with torch.cuda.device(index):
                return f(*args, **kw)
        return f(*args, **kw)

    return call


def _like(t: torch.Tensor) -> torch.Tensor:
    """An uninitialised compact tensor of t's shape and type."""
    return (torch.empty_like(t) if t.is_contiguous()
            else torch.empty(t.shape, dtype=t.dtype, device=t.device))


def _indices(t: Optional[torch.Tensor], name: str, n: Optional[int], index: int):
    """The address of a compact int32 device array (None passes through)."""
    if t is None:
        return None
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.dim() != 1 or (n is not None and t.shape[0] != n) or not t.is_contiguous():
        raise ValueError(f"{name} must be compact, one-dimensional and of the call's length")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the call's device")
    return t.data_ptr()


def _segments(cu: Optional[torch.Tensor], index: int):
    """(address, n_seq) of cu_seqlens; None: one segment of all tokens."""
    if cu is None:
        return None, 1
    if cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError("cu_seqlens must hold n_seq + 1 offsets")
    return _indices(cu, "cu_seqlens", None, index), cu.shape[0] - 1


def _option(table, value, name):
    try:
        return table[value]
    except KeyError:
        raise ValueError(f"unknown {name} {value!r}") from None


def _rows(t: torch.Tensor, dims: int, name: str):
    """Ranks that the marshalling itself relies on; the library checks the rest."""
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims")
    return t.shape


def _scratch(nbytes: int, workspace: Optional[torch.Tensor], x: torch.Tensor):
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    elif workspace.get_device() != x.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be compact and on the call's device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------- short convolution

@_device_call
def conv_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
             initial_state: Optional[torch.Tensor] = None,
             cu_seqlens: Optional[torch.Tensor] = None, activation: Optional[str] = "silu",
             output_final_state: bool = False, out: Optional[torch.Tensor] = None,
             final_state: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None
             ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Short causal convolution of each channel over packed segments (libgdr ``gdr_conv_fwd``).

    x [T, C] bf16 or fp32; weight [C, W] (W = 2..4) and bias [C] fp32 or bf16; initial_state
    [N, W - 1, C] in x's type, the inputs before each segment, oldest first; cu_seqlens [N + 1]
    int32 (None: one segment); activation "silu" or None.  Returns (y [T, C], final_state
    [N, W - 1, C] or None).
    """
    index = x.get_device()
    _rows(x, 2, "x")
    _rows(weight, 2, "weight")
    cu, n_seq = _segments(cu_seqlens, index)
    y = _like(x) if out is None else out
    ht = None
    if output_final_state:
        ht = (torch.empty(n_seq, weight.shape[1] - 1, x.shape[1], dtype=x.dtype,
                          device=x.device) if final_state is None else final_state)
    d = _descs(index, x, weight, bias, initial_state, y, ht)
    rc = nat.lib().gdr_conv_fwd(d[0], d[1], d[2], d[3], cu, n_seq,
                                _option(_ACT, activation, "activation"), d[4], d[5],
                                _raw_stream(index))
    nat.check(rc, "gdr_conv_fwd")
    return y, ht


@_device_call
def conv_bwd(x: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor,
             bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
             cu_seqlens: Optional[torch.Tensor] = None, activation: Optional[str] = "silu",
             dfinal_state: Optional[torch.Tensor] = None, want_dinitial: bool = True,
             workspace: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """Gradients of ``conv_fwd`` (libgdr ``gdr_conv_bwd``): (dx [T, C] in x's type, dweight
    [C, W] fp32, dbias [C] fp32 or None, dinitial_state [N, W - 1, C] in x's type or None)."""
    index = x.get_device()
    T, C = _rows(x, 2, "x")
    W = _rows(weight, 2, "weight")[1]
    cu, n_seq = _segments(cu_seqlens, index)
    dev = x.device
    dx = _like(x)
    dw = torch.empty(C, W, dtype=torch.float32, device=dev)
    db = torch.empty(C, dtype=torch.float32, device=dev) if bias is not None else None
    dh0 = (torch.empty(n_seq, W - 1, C, dtype=x.dtype, device=dev) if want_dinitial else None)
    d = _descs(index, x, weight, bias, initial_state, dy, dfinal_state, dx, dw, db, dh0)
    lib = nat.lib()
    ws, wp, wn = _scratch(lib.gdr_conv_bwd_workspace_bytes(T, C, W), workspace, x)
    rc = lib.gdr_conv_bwd(d[0], d[1], d[2], d[3], cu, n_seq,
                          _option(_ACT, activation, "activation"), d[4], d[5], d[6], d[7],
                          d[8], d[9], wp, wn, _raw_stream(index))
    nat.check(rc, "gdr_conv_bwd")
    return dx, dw, db, dh0


@_device_call
def conv_step(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor,
              bias: Optional[torch.Tensor] = None, activation: Optional[str] = "silu",
              state_indices: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of ``conv_fwd`` for each row of x [B, C]: returns y [B, C] and moves x into
    state [slots, W - 1, C], in place.  state_indices [B] int32: each row's slot (None: row i,
    slot i; outside the pool: a padded row, y = 0)."""
    index = x.get_device()
    B, _ = _rows(x, 2, "x")
    idx = _indices(state_indices, "state_indices", B, index)
    y = _like(x) if out is None else out
    d = _descs(index, x, weight, bias, state, y)
    rc = nat.lib().gdr_conv_step(d[0], d[1], d[2], d[3], idx,
                                 _option(_ACT, activation, "activation"), d[4],
                                _raw_stream(index))
    nat.check(rc, "gdr_conv_step")
    return y


# ---------------------------------------------------------------- selective state space

@_device_call
def ssm_fwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
            C: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
            dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
            initial_state: Optional[torch.Tensor] = None,
            cu_seqlens: Optional[torch.Tensor] = None, output_final_state: bool = False,
            out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None
            ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Selective state space scan over packed segments (libgdr ``gdr_ssm_fwd``).

    x, dt, z [T, Dm] and B, C [T, G, N] bf16 or fp32; A [Dm, N], D, dt_bias [Dm] fp32;
    initial_state [N_seq, Dm, N] fp32; cu_seqlens [N_seq + 1] int32 (None: one segment).
    Returns (y [T, Dm], final_state [N_seq, Dm, N] fp32 or None).
    """
    index = x.get_device()
    T, Dm = _rows(x, 2, "x")
    _, G, N = _rows(B, 3, "B")
    cu, n_seq = _segments(cu_seqlens, index)
    y = _like(x) if out is None else out
    ht = None
    if output_final_state:
        ht = (torch.empty(n_seq, Dm, N, dtype=torch.float32, device=x.device)
              if final_state is None else final_state)
    d = _descs(index, x, dt, A, B, C, D, z, dt_bias, initial_state, y, ht)
    lib = nat.lib()
    ws, wp, wn = _scratch(lib.gdr_ssm_fwd_workspace_bytes(T, Dm, N, G), workspace, x)
    rc = lib.gdr_ssm_fwd(d[0], d[1], d[2], d[3], d[4], d[5], d[6], d[7], int(dt_softplus),
                         d[8], cu, n_seq, d[9], d[10], wp, wn, _raw_stream(index))
    nat.check(rc, "gdr_ssm_fwd")
    return y, ht


@_device_call
def ssm_bwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
            C: torch.Tensor, dy: torch.Tensor, D: Optional[torch.Tensor] = None,
            z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
            dt_softplus: bool = True, initial_state: Optional[torch.Tensor] = None,
            cu_seqlens: Optional[torch.Tensor] = None,
            dfinal_state: Optional[torch.Tensor] = None, want_dinitial: bool = True,
            workspace: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None):
    """Gradients of ``ssm_fwd`` (libgdr ``gdr_ssm_bwd``): (dx, ddt [T, Dm], dA [Dm, N] fp32,
    dB, dC [T, G, N], dD [Dm] fp32 or None, dz [T, Dm] or None, ddt_bias [Dm] fp32 or None,
    dinitial_state [N_seq, Dm, N] fp32 or None); the activations' in x's type."""
    index = x.get_device()
    T, Dm = _rows(x, 2, "x")
    _, G, N = _rows(B, 3, "B")
    cu, n_seq = _segments(cu_seqlens, index)
    f32 = dict(dtype=torch.float32, device=x.device)
    dx, ddt = _like(x), _like(dt)
    dA = torch.empty(Dm, N, **f32)
    dB, dC = _like(B), _like(C)
    dD = torch.empty(Dm, **f32) if D is not None else None
    dz = _like(z) if z is not None else None
    dbias = torch.empty(Dm, **f32) if dt_bias is not None else None
    dh0 = torch.empty(n_seq, Dm, N, **f32) if want_dinitial else None
    d = _descs(index, x, dt, A, B, C, D, z, dt_bias, initial_state, dy, dfinal_state, dx, ddt, dA,
                dB, dC, dD, dz, dbias, dh0)
    lib = nat.lib()
    ws, wp, wn = _scratch(lib.gdr_ssm_bwd_workspace_bytes(T, Dm, N, G), workspace, x)
    rc = lib.gdr_ssm_bwd(d[0], d[1], d[2], d[3], d[4], d[5], d[6], d[7], int(dt_softplus),
                         d[8], cu, n_seq, d[9], d[10], d[11], d[12], d[13], d[14], d[15],
                         d[16], d[17], d[18], d[19], wp, wn, _raw_stream(index))
    nat.check(rc, "gdr_ssm_bwd")
    return dx, ddt, dA, dB, dC, dD, dz, dbias, dh0


@_device_call
def ssm_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
             C: torch.Tensor, state: torch.Tensor, D: Optional[torch.Tensor] = None,
             z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
             dt_softplus: bool = True, state_indices: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of ``ssm_fwd`` for each row: x, dt, z [R, Dm], B, C [R, G, N]; state
    [slots, Dm, N] fp32 in place; state_indices as in ``conv_step``.  Returns y [R, Dm]."""
    index = x.get_device()
    R, _ = _rows(x, 2, "x")
    idx = _indices(state_indices, "state_indices", R, index)
    y = _like(x) if out is None else out
    d = _descs(index, x, dt, A, B, C, D, z, dt_bias, state, y)
    rc = nat.lib().gdr_ssm_step(d[0], d[1], d[2], d[3], d[4], d[5], d[6], d[7],
                                int(dt_softplus), d[8], idx, d[9], _raw_stream(index))
    nat.check(rc, "gdr_ssm_step")
    return y


# ---------------------------------------------------------------- q/k norm with rotation

@_device_call
def qk_fwd(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
           k_weight: Optional[torch.Tensor] = None, norm: str = "rms", eps: float = 1e-6,
           cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None,
           positions: Optional[torch.Tensor] = None, interleaved: bool = False,
           out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
           stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Norm of q [T, Hq, d] and k [T, Hk, d] (bf16 or fp32) over each head, "rms" or "l2", times
    the weights [d] (None: ones), then the rotation of each head's first 2 * cos.shape[1]
    elements by the tables' rows cos, sin [places, rot / 2] fp32 at positions [T] int32 (no
    tables: no rotation).  Pairs are element i with i + rot / 2, or interleaved 2 i with 2 i + 1.
    Returns new (q, k) (libgdr ``gdr_qk_fwd``)."""
    index = q.get_device()
    T = _rows(q, 3, "q")[0]
    pos = _indices(positions, "positions", T, index)
    if out is None:
        out = (_like(q), _like(k))
    d = _descs(index, q, k, q_weight, k_weight, cos, sin, out[0], out[1])
    rc = nat.lib().gdr_qk_fwd(d[0], d[1], d[2], d[3], _option(_NORM, norm, "norm"), eps, d[4],
                              d[5], pos, int(interleaved), d[6], d[7], _raw_stream(index))
    nat.check(rc, "gdr_qk_fwd")
    return out


@_device_call
def qk_bwd(q: torch.Tensor, k: torch.Tensor, dq_out: torch.Tensor, dk_out: torch.Tensor,
           q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
           norm: str = "rms", eps: float = 1e-6, cos: Optional[torch.Tensor] = None,
           sin: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
           interleaved: bool = False, workspace: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None):
    """Gradients of ``qk_fwd`` (libgdr ``gdr_qk_bwd``): (dq, dk in the activations' type,
    dq_weight, dk_weight [d] fp32 or None)."""
    index = q.get_device()
    T, Hq, dim = _rows(q, 3, "q")
    Hk = _rows(k, 3, "k")[1]
    pos = _indices(positions, "positions", T, index)
    dq, dk = _like(q), _like(k)
    f32 = dict(dtype=torch.float32, device=q.device)
    dqw = torch.empty(dim, **f32) if q_weight is not None else None
    dkw = torch.empty(dim, **f32) if k_weight is not None else None
    d = _descs(index, q, k, q_weight, k_weight, cos, sin, dq_out, dk_out, dq, dk, dqw, dkw)
    lib = nat.lib()
    ws, wp, wn = _scratch(lib.gdr_qk_bwd_workspace_bytes(T, Hq, Hk, dim), workspace, q)
    rc = lib.gdr_qk_bwd(d[0], d[1], d[2], d[3], _option(_NORM, norm, "norm"), eps, d[4], d[5],
                        pos, int(interleaved), d[6], d[7], d[8], d[9], d[10], d[11], wp, wn,
                        _raw_stream(index))
    nat.check(rc, "gdr_qk_bwd")
    return dq, dk, dqw, dkw


# ---------------------------------------------------------------- delta rule, single tokens

@_device_call
def delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
               beta: torch.Tensor, state: torch.Tensor, scale: Optional[float] = None,
               state_indices: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of ``chunk_fwd``'s recurrence for each of B requests (libgdr
    ``gdr_delta_step``): q, k [B, Hk, dk], v [B, H, dv], beta [B, H] bf16, g [B, H] fp32; state
    [slots, H, dk, dv] fp32 in place (``chunk_fwd``'s final states continue here);
    state_indices as in ``conv_step``.  Returns o [B, H, dv] bf16."""
    index = q.get_device()
    B, _, dim = _rows(q, 3, "q")
    idx = _indices(state_indices, "state_indices", B, index)
    o = _like(v) if out is None else out
    d = _descs(index, q, k, v, g, beta, state, o)
    rc = nat.lib().gdr_delta_step(d[0], d[1], d[2], d[3], d[4],
                                  dim ** -0.5 if scale is None else scale, d[5], idx, d[6],
                                  _raw_stream(index))
    nat.check(rc, "gdr_delta_step")
    return o


# ---------------------------------------------------------------- autograd

def _grad(t: Optional[torch.Tensor], like: torch.Tensor, dtype=None) -> torch.Tensor:
    """An output's gradient as the library takes it: the output's type, innermost contiguous;
    zeros where autograd has none."""
    if t is None:
        return torch.zeros(like.shape, dtype=like.dtype if dtype is None else dtype,
                           device=like.device)
    t = t.to(like.dtype if dtype is None else dtype)
    return t if t.stride(-1) == 1 else t.contiguous()


def _cast(t: Optional[torch.Tensor], like: Optional[torch.Tensor]):
    return None if t is None else t.to(like.dtype)


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, activation, output_final_state):
        ctx.set_materialize_grads(False)
        y, ht = conv_fwd(x, weight, bias, initial_state, cu_seqlens, activation,
                         output_final_state)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.activation = activation
        return y, ht

    @staticmethod
    def backward(ctx, dy, dht):
        x, w, b, h0, cu = ctx.saved_tensors
        dx, dw, db, dh0 = conv_bwd(
            x, w, _grad(dy, x), b, h0, cu, ctx.activation,
            None if dht is None else dht.to(x.dtype).contiguous(),
            want_dinitial=h0 is not None and ctx.needs_input_grad[3])
        return dx, _cast(dw, w), _cast(db, b), dh0, None, None, None


def short_conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation="silu",
               output_final_state: bool = False):
    """Differentiable ``conv_fwd``: (y, final_state or None)."""
    return _ShortConv.apply(x, weight, bias, initial_state, cu_seqlens, activation,
                            output_final_state)


class _SelectiveSsm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, cu_seqlens,
                output_final_state):
        ctx.set_materialize_grads(False)
        y, ht = ssm_fwd(x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, cu_seqlens,
                        output_final_state)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens)
        ctx.dt_softplus = dt_softplus
        return y, ht

    @staticmethod
    def backward(ctx, dy, dht):
        x, dt, A, B, C, D, z, dt_bias, h0, cu = ctx.saved_tensors
        dx, ddt, dA, dB, dC, dD, dz, dbias, dh0 = ssm_bwd(
            x, dt, A, B, C, _grad(dy, x), D, z, dt_bias, ctx.dt_softplus, h0, cu,
            None if dht is None else dht.float().contiguous(),
            want_dinitial=h0 is not None and ctx.needs_input_grad[9])
        return dx, ddt, dA, dB, dC, dD, dz, dbias, None, dh0, None, None


def selective_ssm(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = True,
                  initial_state=None, cu_seqlens=None, output_final_state: bool = False):
    """Differentiable ``ssm_fwd``: (y, final_state or None)."""
    return _SelectiveSsm.apply(x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state,
                               cu_seqlens, output_final_state)


class _QkNormRotate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, norm, eps, cos, sin, positions, interleaved):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        ctx.options = (norm, eps, interleaved)
        return qk_fwd(q, k, q_weight, k_weight, norm, eps, cos, sin, positions, interleaved)

    @staticmethod
    def backward(ctx, dqo, dko):
        q, k, qw, kw, cos, sin, pos = ctx.saved_tensors
        norm, eps, inter = ctx.options
        dq, dk, dqw, dkw = qk_bwd(q, k, _grad(dqo, q), _grad(dko, k), qw, kw, norm, eps, cos,
                                  sin, pos, inter)
        return dq, dk, _cast(dqw, qw), _cast(dkw, kw), None, None, None, None, None, None


def qk_norm_rotate(q, k, q_weight=None, k_weight=None, norm: str = "rms", eps: float = 1e-6,
                   cos=None, sin=None, positions=None, interleaved: bool = False):
    """Differentiable ``qk_fwd``: new (q, k)."""
    return _QkNormRotate.apply(q, k, q_weight, k_weight, norm, eps, cos, sin, positions,
                               interleaved)
