"""The operators around the delta rule in a token mixer: short causal convolution, selective
state space, per-head q/k norm with rotation, and the delta rule for single tokens.

Device tensors only; marshalling is in ``_mixer`` (csrc/mixer_binding.cpp): descriptors of the
tensors, outputs and scratch from PyTorch's allocator, torch's current stream.  With ``stream``,
that stream is made current for the call, so that what the call allocates belongs to it; inputs
that another stream may reuse while the call runs are the caller's to keep
(``Tensor.record_stream``).  Outputs that are given must not overlap inputs.  Layouts and formulas
are those of include/gdr.h.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _native as nat
from ._autograd import first_only

_ext = None


def _load():
    """The binding (raises if it has not been built: there is no fallback)."""
    global _ext
    if _ext is None:
        nat.lib()
        try:
            from . import _mixer
        except ImportError as e:
            raise RuntimeError(
                f"the mixer's binding cannot be loaded ({e}); build it with "
                "`python -m chunked_gated_delta_gdr_gb300.build`") from e
        _mixer.set_error(nat.GdrError)
        _ext = _mixer
    return _ext


# ---------------------------------------------------------------- short convolution

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
    [N, W - 1, C] or None); ``out`` and ``final_state`` may give them, and a final_state that is
    given is written whatever output_final_state says.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return conv_fwd(x, weight, bias, initial_state, cu_seqlens, activation,
                            output_final_state, out, final_state)
    return (_ext or _load()).conv_fwd(x, weight, bias, initial_state, cu_seqlens, activation,
                                      output_final_state, out, final_state)


def conv_bwd(x: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor,
             bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
             cu_seqlens: Optional[torch.Tensor] = None, activation: Optional[str] = "silu",
             dfinal_state: Optional[torch.Tensor] = None, want_dinitial: bool = True,
             workspace: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """Gradients of ``conv_fwd`` (libgdr ``gdr_conv_bwd``): (dx [T, C] in x's type, dweight
    [C, W] fp32, dbias [C] fp32 or None, dinitial_state [N, W - 1, C] in x's type or None)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return conv_bwd(x, weight, dy, bias, initial_state, cu_seqlens, activation,
                            dfinal_state, want_dinitial, workspace)
    return (_ext or _load()).conv_bwd(x, weight, dy, bias, initial_state, cu_seqlens, activation,
                                      dfinal_state, want_dinitial, workspace)


def conv_step(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor,
              bias: Optional[torch.Tensor] = None, activation: Optional[str] = "silu",
              state_indices: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of ``conv_fwd`` for each row of x [B, C]: returns y [B, C] and moves x into
    state [slots, W - 1, C], in place.  state_indices [B] int32: each row's slot (None: row i,
    slot i; outside the pool: a padded row, y = 0)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return conv_step(x, weight, state, bias, activation, state_indices, out)
    return (_ext or _load()).conv_step(x, weight, state, bias, activation, state_indices, out)


# ---------------------------------------------------------------- selective state space

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
    Returns (y [T, Dm], final_state [N_seq, Dm, N] fp32 or None); ``out`` and ``final_state``
    may give them, and a final_state that is given is written whatever output_final_state says.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return ssm_fwd(x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, cu_seqlens,
                           output_final_state, out, final_state, workspace)
    return (_ext or _load()).ssm_fwd(x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state,
                                     cu_seqlens, output_final_state, out, final_state, workspace)


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
    if stream is not None:
        with torch.cuda.stream(stream):
            return ssm_bwd(x, dt, A, B, C, dy, D, z, dt_bias, dt_softplus, initial_state,
                           cu_seqlens, dfinal_state, want_dinitial, workspace)
    return (_ext or _load()).ssm_bwd(x, dt, A, B, C, dy, D, z, dt_bias, dt_softplus,
                                     initial_state, cu_seqlens, dfinal_state, want_dinitial,
                                     workspace)


def ssm_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
             C: torch.Tensor, state: torch.Tensor, D: Optional[torch.Tensor] = None,
             z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
             dt_softplus: bool = True, state_indices: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of ``ssm_fwd`` for each row: x, dt, z [R, Dm], B, C [R, G, N]; state
    [slots, Dm, N] fp32 in place; state_indices as in ``conv_step``.  Returns y [R, Dm]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return ssm_step(x, dt, A, B, C, state, D, z, dt_bias, dt_softplus, state_indices, out)
    return (_ext or _load()).ssm_step(x, dt, A, B, C, state, D, z, dt_bias, dt_softplus,
                                      state_indices, out)


# ---------------------------------------------------------------- q/k norm with rotation

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
    Returns new (q, k), or those of ``out`` (libgdr ``gdr_qk_fwd``)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return qk_fwd(q, k, q_weight, k_weight, norm, eps, cos, sin, positions, interleaved,
                          out)
    qo, ko = (None, None) if out is None else out
    return (_ext or _load()).qk_fwd(q, k, q_weight, k_weight, norm, eps, cos, sin, positions,
                                    interleaved, qo, ko)


def qk_bwd(q: torch.Tensor, k: torch.Tensor, dq_out: torch.Tensor, dk_out: torch.Tensor,
           q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
           norm: str = "rms", eps: float = 1e-6, cos: Optional[torch.Tensor] = None,
           sin: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
           interleaved: bool = False, workspace: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None):
    """Gradients of ``qk_fwd`` (libgdr ``gdr_qk_bwd``): (dq, dk in the activations' type,
    dq_weight, dk_weight [d] fp32 or None)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return qk_bwd(q, k, dq_out, dk_out, q_weight, k_weight, norm, eps, cos, sin,
                          positions, interleaved, workspace)
    return (_ext or _load()).qk_bwd(q, k, dq_out, dk_out, q_weight, k_weight, norm, eps, cos, sin,
                                    positions, interleaved, workspace)


# ---------------------------------------------------------------- delta rule, single tokens

def delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
               beta: torch.Tensor, state: torch.Tensor, scale: Optional[float] = None,
               state_indices: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of ``chunk_fwd``'s recurrence for each of B requests (libgdr
    ``gdr_delta_step``): q, k [B, Hk, dk], v [B, H, dv], beta [B, H] bf16, g [B, H] fp32; state
    [slots, H, dk, dv] fp32 in place (``chunk_fwd``'s final states continue here);
    state_indices as in ``conv_step``.  Returns o [B, H, dv] bf16."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return delta_step(q, k, v, g, beta, state, scale, state_indices, out)
    return (_ext or _load()).delta_step(q, k, v, g, beta, state, scale, state_indices, out)


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
        return first_only("short_conv", (dx, _cast(dw, w), _cast(db, b), dh0, None, None, None),
                          x, w, b, h0, dy, dht)


def short_conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation="silu",
               output_final_state: bool = False):
    """Differentiable ``conv_fwd``, once: (y, final_state or None)."""
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
        return first_only("selective_ssm",
                          (dx, ddt, dA, dB, dC, dD, dz, dbias, None, dh0, None, None),
                          x, dt, A, B, C, D, z, dt_bias, h0, dy, dht)


def selective_ssm(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = True,
                  initial_state=None, cu_seqlens=None, output_final_state: bool = False):
    """Differentiable ``ssm_fwd``, once: (y, final_state or None)."""
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
        return first_only("qk_norm_rotate", (dq, dk, _cast(dqw, qw), _cast(dkw, kw), None, None,
                                             None, None, None, None), q, k, qw, kw, dqo, dko)


def qk_norm_rotate(q, k, q_weight=None, k_weight=None, norm: str = "rms", eps: float = 1e-6,
                   cos=None, sin=None, positions=None, interleaved: bool = False):
    """Differentiable ``qk_fwd``, once: new (q, k)."""
    return _QkNormRotate.apply(q, k, q_weight, k_weight, norm, eps, cos, sin, positions,
                               interleaved)
