"""The operators of a hybrid block beside its mixer: gated linear recurrence, the norms behind and
before a block with its gate and residual scale, attention of single tokens over a paged key-value
cache, and the cache's block tables, slots and writes.

Marshalling as in ``mixer`` (csrc/mixer_binding.cpp): device tensors only, torch's current stream or
``stream``, outputs and scratch from PyTorch's allocator.  Outputs that are given must not overlap
inputs but where a function says so.  Layouts and formulas are those of include/gdr.h.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import mixer as _m
from ._autograd import first_only
from .mixer import _cast, _grad


def _binding():
    return _m._ext or _m._load()


# ---------------------------------------------------------------- gated linear recurrence

def rec_fwd(x: torch.Tensor, r: torch.Tensor, A: torch.Tensor, i: Optional[torch.Tensor] = None,
            normalize: bool = True, initial_state: Optional[torch.Tensor] = None,
            cu_seqlens: Optional[torch.Tensor] = None, output_final_state: bool = False,
            output_checkpoints: bool = False, out: Optional[torch.Tensor] = None,
            final_state: Optional[torch.Tensor] = None,
            checkpoints: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None
            ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gated linear recurrence of each channel over packed segments (libgdr ``gdr_rec_fwd``):

        a = exp(A sigmoid(r)),  h = a h + sqrt(1 - a^2) sigmoid(i) x,  y = h

    x, r, i [T, D] bf16 or fp32 (i None: no such gate); A [D] fp32, not above 0 (where it
    is, the root is NaN); normalize False: 1 in place of the root, and A of any sign; initial_state
    [N, D] fp32; cu_seqlens [N + 1] int32 (None: one segment).  Returns (y [T, D], final_state [N, D]
    fp32 or None, checkpoints or None): the last are what ``rec_bwd`` of the same inputs would
    otherwise compute again.  ``out``, ``final_state`` and ``checkpoints`` [ceil(T / 8), D] fp32 may
    give them; what is given is written.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return rec_fwd(x, r, A, i, normalize, initial_state, cu_seqlens, output_final_state,
                           output_checkpoints, out, final_state, checkpoints)
    return _binding().rec_fwd(x, r, A, i, normalize, initial_state, cu_seqlens,
                              output_final_state, output_checkpoints, out, final_state,
                              checkpoints)


def rec_bwd(x: torch.Tensor, r: torch.Tensor, A: torch.Tensor, dy: torch.Tensor,
            i: Optional[torch.Tensor] = None, normalize: bool = True,
            initial_state: Optional[torch.Tensor] = None,
            cu_seqlens: Optional[torch.Tensor] = None,
            dfinal_state: Optional[torch.Tensor] = None, want_dinitial: bool = True,
            checkpoints: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None):
    """Gradients of ``rec_fwd`` (libgdr ``gdr_rec_bwd``): (dx, dr [T, D] in x's type, dA [D] fp32,
    di [T, D] or None, dinitial_state [N, D] fp32 or None).  ``checkpoints`` of the forward of the
    same inputs save computing its states again."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rec_bwd(x, r, A, dy, i, normalize, initial_state, cu_seqlens, dfinal_state,
                           want_dinitial, checkpoints, workspace)
    return _binding().rec_bwd(x, r, A, dy, i, normalize, initial_state, cu_seqlens, dfinal_state,
                              want_dinitial, checkpoints, workspace)


def rec_step(x: torch.Tensor, r: torch.Tensor, A: torch.Tensor, state: torch.Tensor,
             i: Optional[torch.Tensor] = None, normalize: bool = True,
             state_indices: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of ``rec_fwd`` for each row of x, r, i [B, D]: returns y [B, D]; state [slots, D]
    fp32 in place (``rec_fwd``'s final states continue here); state_indices as in ``conv_step``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rec_step(x, r, A, state, i, normalize, state_indices, out)
    return _binding().rec_step(x, r, A, state, i, normalize, state_indices, out)


# ---------------------------------------------------------------- norms of a block

def gated_norm_fwd(x: torch.Tensor, z: torch.Tensor, weight: Optional[torch.Tensor] = None,
                   activation: str = "silu", eps: float = 1e-6,
                   out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """RMS norm of x [T, H, d] over each head, times weight [d] (None: ones) and the activated gate
    z [T, H, d], "silu" or "sigmoid" (libgdr ``gdr_gated_norm_fwd``).  d <= 1024.  ``out`` may be x
    or z."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_norm_fwd(x, z, weight, activation, eps, out)
    return _binding().gated_norm_fwd(x, z, weight, activation, eps, out)


def gated_norm_bwd(x: torch.Tensor, z: torch.Tensor, dy: torch.Tensor,
                   weight: Optional[torch.Tensor] = None, activation: str = "silu",
                   eps: float = 1e-6, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """Gradients of ``gated_norm_fwd`` (libgdr ``gdr_gated_norm_bwd``): (dx, dz [T, H, d] in x's
    type, dweight [d] fp32 or None)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_norm_bwd(x, z, dy, weight, activation, eps, workspace)
    return _binding().gated_norm_bwd(x, z, dy, weight, activation, eps, workspace)


def residual_norm_fwd(x: torch.Tensor, residual: Optional[torch.Tensor],
                      weight: Optional[torch.Tensor] = None,
                      post_weight: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, scale: float = 1.0, eps: float = 1e-6,
                      post_norm: bool = False, out: Optional[torch.Tensor] = None,
                      residual_out: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None
                      ) -> Tuple[torch.Tensor, torch.Tensor]:
    """What lies between two blocks, of which the first gave x [T, C] (libgdr
    ``gdr_residual_norm_fwd``):

        h = residual + scale gate u,   y = rms_norm(h) weight

    with u = x, or rms_norm(x) post_weight where post_weight is given or post_norm says so.
    residual [T, C] in x's type or fp32 (None: zeros); weight, post_weight, gate [C] (None: ones);
    C <= 16384.  Returns (y in x's type, h in the residual's); ``out`` and ``residual_out`` may give
    them: residual_out may be the residual, out may be x."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return residual_norm_fwd(x, residual, weight, post_weight, gate, scale, eps, post_norm,
                                     out, residual_out)
    return _binding().residual_norm_fwd(x, residual, weight, post_norm or post_weight is not None,
                                        post_weight, gate, scale, eps, out, residual_out)


def residual_norm_bwd(x: torch.Tensor, residual: Optional[torch.Tensor], dy: torch.Tensor,
                      dh: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                      post_weight: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, scale: float = 1.0, eps: float = 1e-6,
                      post_norm: bool = False, workspace: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None):
    """Gradients of ``residual_norm_fwd`` (libgdr ``gdr_residual_norm_bwd``) from those of y and h
    (dh None: zeros): (dx, dresidual or None, dweight, dpost_weight, dgate [C] fp32, each or None)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return residual_norm_bwd(x, residual, dy, dh, weight, post_weight, gate, scale, eps,
                                     post_norm, workspace)
    return _binding().residual_norm_bwd(x, residual, dy, dh, weight,
                                        post_norm or post_weight is not None, post_weight, gate,
                                        scale, eps, workspace)


# ---------------------------------------------------------------- attention over a paged cache

def attn_step(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              block_table: torch.Tensor, lengths: torch.Tensor, scale: Optional[float] = None,
              window: int = 0, out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of one new token of each of B requests over a paged cache (libgdr
    ``gdr_attn_step``): q [B, Hq, d], k_cache, v_cache [pages, page_size, Hk, d] bf16 or fp32, Hq a
    multiple of Hk; block_table [B, width] int32 names each request's pages in order, lengths [B]
    int32 its keys, the new token's own among them.  scale None: d^-1/2; window: the last keys that
    are seen (0: all).  Returns o [B, Hq, d]; a request of length 0 gets zeros."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return attn_step(q, k_cache, v_cache, block_table, lengths, scale, window, out,
                             workspace)
    return _binding().attn_step(q, k_cache, v_cache, block_table, lengths, scale, window, out,
                                workspace)


def cache_plan(lengths: torch.Tensor, new_tokens: torch.Tensor, block_table: torch.Tensor,
               free_pages: torch.Tensor, taken: torch.Tensor, page_size: int, max_tokens: int,
               lengths_out: Optional[torch.Tensor] = None,
               taken_out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """Pages, slots and positions of the new tokens of B requests, on the GPU (libgdr
    ``gdr_cache_plan``).

    lengths, new_tokens [B] int32: tokens in the cache, and to add; block_table [B, width] int32 in
    place: the pages that are needed more are written behind those that a request has; free_pages
    [F] int32, handed out in order from the taken-th on, taken [1] int32.  Returns (slots
    [max_tokens], positions [max_tokens], cu_seqlens [B + 1], lengths [B] and taken [1] afterwards),
    int32: a token's slot is page * page_size + place; behind the last token slots are -1.  A request
    is given fewer tokens where its row, max_tokens or free_pages end; those of the requests behind it then
    follow at once, so that rows that lie as they were asked for find theirs by cu_seqlens: token j of
    request b at cu_seqlens[b] + j where that is below cu_seqlens[b + 1], and nowhere else.
    ``lengths_out`` may be lengths and ``taken_out`` taken, so that a captured step goes on from its own
    results.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return cache_plan(lengths, new_tokens, block_table, free_pages, taken, page_size,
                              max_tokens, lengths_out, taken_out)
    return _binding().cache_plan(lengths, new_tokens, block_table, free_pages, taken, page_size,
                                 max_tokens, lengths_out, taken_out)


def cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                slots: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Rows of k, v [T, Hk, d] into k_cache, v_cache [pages, page_size, Hk, d] (one type) at slots
    [T] int32, page * page_size + place; a slot outside the cache marks a row that is not written
    (libgdr ``gdr_cache_write``)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return cache_write(k, v, k_cache, v_cache, slots)
    return _binding().cache_write(k, v, k_cache, v_cache, slots)


# ---------------------------------------------------------------- autograd

class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, A, i, normalize, initial_state, cu_seqlens, output_final_state):
        ctx.set_materialize_grads(False)
        y, ht, kept = rec_fwd(x, r, A, i, normalize, initial_state, cu_seqlens,
                              output_final_state, any(ctx.needs_input_grad))
        ctx.save_for_backward(x, r, A, i, initial_state, cu_seqlens, kept)
        ctx.normalize = normalize
        return y, ht

    @staticmethod
    def backward(ctx, dy, dht):
        x, r, A, i, h0, cu, kept = ctx.saved_tensors
        dx, dr, dA, di, dh0 = rec_bwd(
            x, r, A, _grad(dy, x), i, ctx.normalize, h0, cu,
            None if dht is None else dht.float().contiguous(),
            want_dinitial=h0 is not None and ctx.needs_input_grad[5], checkpoints=kept)
        return first_only("gated_recurrence", (dx, dr, dA, di, None, dh0, None, None),
                          x, r, A, i, h0, dy, dht)


def gated_recurrence(x, r, A, i=None, normalize: bool = True, initial_state=None, cu_seqlens=None,
                     output_final_state: bool = False):
    """Differentiable ``rec_fwd``, once: (y, final_state or None)."""
    return _GatedRecurrence.apply(x, r, A, i, normalize, initial_state, cu_seqlens,
                                  output_final_state)


class _GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, weight, activation, eps):
        ctx.save_for_backward(x, z, weight)
        ctx.options = (activation, eps)
        return gated_norm_fwd(x, z, weight, activation, eps)

    @staticmethod
    def backward(ctx, dy):
        x, z, w = ctx.saved_tensors
        dx, dz, dw = gated_norm_bwd(x, z, _grad(dy, x), w, *ctx.options)
        return first_only("gated_norm", (dx, dz, _cast(dw, w), None, None), x, z, w, dy)


def gated_norm(x, z, weight=None, activation: str = "silu", eps: float = 1e-6):
    """Differentiable ``gated_norm_fwd``, once."""
    return _GatedNorm.apply(x, z, weight, activation, eps)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, post_weight, gate, scale, eps, post_norm):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, residual, weight, post_weight, gate)
        ctx.options = (scale, eps, post_norm)
        return residual_norm_fwd(x, residual, weight, post_weight, gate, scale, eps, post_norm)

    @staticmethod
    def backward(ctx, dy, dh):
        x, res, w, wp, g = ctx.saved_tensors
        like = x if res is None else res
        dx, dres, dw, dwp, dg = residual_norm_bwd(
            x, res, _grad(dy, x), None if dh is None else _grad(dh, like), w, wp, g, *ctx.options)
        return first_only("residual_norm",
                          (dx, dres, _cast(dw, w), _cast(dwp, wp), _cast(dg, g), None, None, None),
                          x, res, w, wp, g, dy, dh)


def residual_norm(x, residual=None, weight=None, post_weight=None, gate=None, scale: float = 1.0,
                  eps: float = 1e-6, post_norm: bool = False):
    """Differentiable ``residual_norm_fwd``, once: (y, h)."""
    return _ResidualNorm.apply(x, residual, weight, post_weight, gate, scale, eps, post_norm)
