"""A hybrid block's operators without a GPU: malformed calls are refused before any device access, the
scratch that is asked for holds what the passes keep in it, the Python binding refuses what it
cannot describe, and the plain implementation of the cache's plan follows its rules."""
import ctypes

import pytest
import torch

import block_testlib as ref
import chunked_gated_delta_gdr_gb300 as gdr
from chunked_gated_delta_gdr_gb300 import _native as nat
from test_mixer_abi import D, call, lib  # noqa: F401

F, I32 = nat.GDR_F32, nat.GDR_I32
NULL, DTYPE, SHAPE, STRIDE, DIM, HEADS, NSEQ, WORK, OPTION = -1, -2, -3, -4, -5, -6, -7, -8, -15
CU, WS = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x40000)
T, C, N_SEQ = 96, 64, 2
f32 = ctypes.c_float


def rec_fwd():
    return dict(x=D(T, C), r=D(T, C), i=D(T, C), A=D(C, dtype=F), normalize=1,
                h0=D(N_SEQ, C, dtype=F), cu=CU, n_seq=N_SEQ, y=D(T, C), ht=D(N_SEQ, C, dtype=F),
                kept=D(T // 8, C, dtype=F), stream=None)


def rec_bwd():
    return dict(x=D(T, C), r=D(T, C), i=D(T, C), A=D(C, dtype=F), normalize=1,
                h0=D(N_SEQ, C, dtype=F), cu=CU, n_seq=N_SEQ, kept=D(T // 8, C, dtype=F), dy=D(T, C),
                dht=D(N_SEQ, C, dtype=F), dx=D(T, C), dr=D(T, C), di=D(T, C), dA=D(C, dtype=F),
                dh0=D(N_SEQ, C, dtype=F), ws=WS, ws_bytes=1 << 40, stream=None)


def rec_step():
    return dict(x=D(5, C), r=D(5, C), i=D(5, C), A=D(C, dtype=F), normalize=1,
                state=D(9, C, dtype=F), idx=CU, y=D(5, C), stream=None)


def gated_norm_fwd():
    return dict(x=D(T, 4, 64), z=D(T, 4, 64), weight=D(64, dtype=F), act=1, eps=f32(1e-6),
                y=D(T, 4, 64), stream=None)


def gated_norm_bwd():
    return dict(x=D(T, 4, 64), z=D(T, 4, 64), weight=D(64, dtype=F), act=2, eps=f32(1e-6),
                dy=D(T, 4, 64), dx=D(T, 4, 64), dz=D(T, 4, 64), dw=D(64, dtype=F), ws=WS,
                ws_bytes=1 << 40, stream=None)


def residual_norm_fwd():
    return dict(x=D(T, C), res=D(T, C), weight=D(C, dtype=F), post=1, wp=D(C), gate=D(C, dtype=F),
                scale=f32(0.5), eps=f32(1e-6), y=D(T, C), h=D(T, C), stream=None)


def residual_norm_bwd():
    return dict(x=D(T, C), res=D(T, C, dtype=F), weight=D(C, dtype=F), post=1, wp=D(C),
                gate=D(C, dtype=F), scale=f32(0.5), eps=f32(1e-6), dy=D(T, C), dh=D(T, C, dtype=F),
                dx=D(T, C), dres=D(T, C, dtype=F), dw=D(C, dtype=F), dwp=D(C, dtype=F),
                dg=D(C, dtype=F), ws=WS, ws_bytes=1 << 40, stream=None)


def attn_step():
    return dict(q=D(3, 8, 64), kc=D(40, 16, 2, 64), vc=D(40, 16, 2, 64), table=D(3, 10, dtype=I32),
                lens=CU, scale=f32(0.125), window=0, o=D(3, 8, 64), ws=WS, ws_bytes=1 << 40,
                stream=None)


def cache_plan():
    return dict(lens=CU, new=CU, B=3, table=D(3, 10, dtype=I32), free=D(30, dtype=I32), taken=CU,
                page=16, slots=CU, pos=CU, most=7, cu=CU, lens_out=CU, taken_out=CU, stream=None)


def cache_write():
    return dict(k=D(7, 2, 64), v=D(7, 2, 64), kc=D(40, 16, 2, 64), vc=D(40, 16, 2, 64), slots=CU,
                stream=None)


MAKERS = [rec_fwd, rec_bwd, rec_step, gated_norm_fwd, gated_norm_bwd, residual_norm_fwd,
          residual_norm_bwd, attn_step, cache_plan, cache_write]

REFUSED = [
    (rec_fwd, dict(x=None), NULL), (rec_fwd, dict(r=None), NULL), (rec_fwd, dict(A=None), NULL),
    (rec_fwd, dict(y=None), NULL), (rec_fwd, dict(cu=None), NULL), (rec_fwd, dict(n_seq=-1), NSEQ),
    (rec_fwd, dict(x=D(T, C, dtype=I32)), DTYPE), (rec_fwd, dict(r=D(T, C, dtype=F)), DTYPE),
    (rec_fwd, dict(i=D(T - 1, C)), SHAPE), (rec_fwd, dict(A=D(C)), DTYPE),
    (rec_fwd, dict(A=D(C + 1, dtype=F)), SHAPE), (rec_fwd, dict(x=D(1 << 31, C)), SHAPE),
    (rec_fwd, dict(h0=D(N_SEQ + 1, C, dtype=F)), NSEQ), (rec_fwd, dict(h0=D(N_SEQ, C)), DTYPE),
    (rec_fwd, dict(ht=D(N_SEQ, C, dtype=F, strides=[C + 1, 1])), STRIDE),
    (rec_fwd, dict(y=D(T, C, strides=[C - 1, 1])), STRIDE), (rec_fwd, dict(normalize=2), OPTION),
    (rec_fwd, dict(kept=D(T // 8 + 1, C, dtype=F)), SHAPE),
    (rec_fwd, dict(kept=D(T // 8, C)), DTYPE), (rec_fwd, dict(x=D(T, 0)), SHAPE),
    (rec_bwd, dict(di=None), OPTION), (rec_bwd, dict(i=None), OPTION), (rec_bwd, dict(dA=None), NULL),
    (rec_bwd, dict(dy=None), NULL), (rec_bwd, dict(dx=D(T, C, strides=[0, 1])), STRIDE),
    (rec_bwd, dict(dht=D(1, C, dtype=F)), NSEQ), (rec_bwd, dict(dr=D(T, C, dtype=F)), DTYPE),
    (rec_bwd, dict(kept=D(T, C, dtype=F)), SHAPE),
    (rec_step, dict(state=D(9, C)), DTYPE), (rec_step, dict(state=D(9, C + 1, dtype=F)), SHAPE),
    (rec_step, dict(idx=None, state=D(4, C, dtype=F)), SHAPE),
    (gated_norm_fwd, dict(z=None), NULL), (gated_norm_fwd, dict(z=D(T, 4, 64, dtype=F)), DTYPE),
    (gated_norm_fwd, dict(z=D(T, 3, 64)), SHAPE), (gated_norm_fwd, dict(act=0), OPTION),
    (gated_norm_fwd, dict(act=3), OPTION), (gated_norm_fwd, dict(eps=f32(-1.0)), OPTION),
    (gated_norm_fwd, dict(eps=f32(float("nan"))), OPTION),
    (gated_norm_fwd, dict(weight=D(63, dtype=F)), SHAPE),
    (gated_norm_fwd, dict(x=D(T, 4, 1025)), DIM), (gated_norm_fwd, dict(x=D(T, 4, 0)), DIM),
    (gated_norm_fwd, dict(y=D(T, 4, 64, strides=[256, 32, 1])), STRIDE),
    (gated_norm_bwd, dict(dz=None), NULL), (gated_norm_bwd, dict(dw=D(64)), DTYPE),
    (gated_norm_bwd, dict(dx=D(T, 4, 64, strides=[0, 64, 1])), STRIDE),
    (residual_norm_fwd, dict(post=0), OPTION), (residual_norm_fwd, dict(post=2), OPTION),
    (residual_norm_fwd, dict(x=D(T, C, dtype=F)), DTYPE),  # a residual in fewer bits than x
    (residual_norm_fwd, dict(h=D(T, C, dtype=F)), DTYPE), (residual_norm_fwd, dict(y=None), NULL),
    (residual_norm_fwd, dict(res=D(T, C, dtype=I32)), DTYPE),
    (residual_norm_fwd, dict(gate=D(C + 1, dtype=F)), SHAPE),
    (residual_norm_fwd, dict(x=D(T, 16385)), DIM), (residual_norm_fwd, dict(eps=f32(-1e-9)), OPTION),
    (residual_norm_bwd, dict(dh=D(T, C)), DTYPE), (residual_norm_bwd, dict(dres=D(T, C)), DTYPE),
    (residual_norm_bwd, dict(dx=None), NULL), (residual_norm_bwd, dict(post=0, wp=None), OPTION),
    (residual_norm_bwd, dict(dg=D(C - 1, dtype=F)), SHAPE),
    (attn_step, dict(q=None), NULL), (attn_step, dict(lens=None), NULL),
    (attn_step, dict(table=None), NULL), (attn_step, dict(table=D(3, 10, dtype=F)), DTYPE),
    (attn_step, dict(table=D(2, 10, dtype=I32)), SHAPE),
    (attn_step, dict(table=D(3, 10, dtype=I32, strides=[10, 2])), STRIDE),
    (attn_step, dict(table=D(3, 1 << 28, dtype=I32)), SHAPE),  # more places than are counted
    (attn_step, dict(vc=D(40, 16, 2, 64, dtype=F)), DTYPE), (attn_step, dict(vc=D(40, 8, 2, 64)), SHAPE),
    (attn_step, dict(kc=D(40, 16, 2, 32), vc=D(40, 16, 2, 32)), SHAPE),
    (attn_step, dict(kc=D(40, 16, 3, 64), vc=D(40, 16, 3, 64)), HEADS),
    (attn_step, dict(kc=D(40, 0, 2, 64), vc=D(40, 0, 2, 64)), SHAPE),
    (attn_step, dict(q=D(3, 8, 257)), DIM), (attn_step, dict(window=-1), OPTION),
    (attn_step, dict(o=D(3, 8, 64, dtype=F)), DTYPE), (attn_step, dict(o=D(3, 4, 64)), SHAPE),
    (attn_step, dict(o=D(3, 8, 64, strides=[512, 0, 1])), STRIDE),
    (cache_plan, dict(taken=None), NULL), (cache_plan, dict(slots=None), NULL),
    (cache_plan, dict(cu=None), NULL), (cache_plan, dict(lens_out=None), NULL),
    (cache_plan, dict(table=D(4, 10, dtype=I32)), SHAPE), (cache_plan, dict(page=0), SHAPE),
    (cache_plan, dict(most=-1), SHAPE), (cache_plan, dict(B=-1), SHAPE),
    (cache_plan, dict(table=D(3, 10, dtype=I32, strides=[0, 1])), STRIDE),
    (cache_plan, dict(free=D(30)), DTYPE),
    (cache_write, dict(slots=None), NULL), (cache_write, dict(v=D(7, 2, 64, dtype=F)), DTYPE),
    (cache_write, dict(v=D(6, 2, 64)), SHAPE), (cache_write, dict(kc=D(40, 16, 3, 64)), SHAPE),
    (cache_write, dict(kc=D(40, 16, 2, 64, strides=[0, 128, 64, 1])), STRIDE),
    (cache_write, dict(vc=D(40, 16, 2, 64, strides=[1024, 64, 64, 1])), STRIDE),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_refused_before_the_device(lib, case):  # noqa: F811
    make, over, code = REFUSED[case]
    assert call(getattr(lib, "gdr_" + make.__name__), make(), **over) == code


@pytest.mark.parametrize("make", MAKERS)
def test_well_formed_calls_reach_the_device_check(lib, make):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    args = make()
    # heads before places is a layout of a cache, too
    for k in ("kc", "vc"):
        if k in args:
            args[k] = D(40, 16, 2, 64, strides=[2048, 64, 1024, 1])
    assert call(getattr(lib, "gdr_" + make.__name__), args) in (-10, -12)


def test_scratch_sizes(lib):  # noqa: F811
    for T_, D_, n in ((1, 1, 1), (17, 64, 3), (8192, 2560, 6), (70001, 66, 2000)):
        assert lib.gdr_rec_checkpoint_rows(T_) == -(-T_ // 8)
        least = 4 * (n + 1)
        assert lib.gdr_rec_bwd_workspace_bytes(T_, D_, n, 1) >= least
        assert lib.gdr_rec_bwd_workspace_bytes(T_, D_, n, 0) >= least + -(-T_ // 8) * D_ * 4
    for T_, H, d in ((1, 1, 1), (8191, 16, 128), (3, 2, 1024)):
        assert lib.gdr_gated_norm_bwd_workspace_bytes(T_, H, d) >= 4 * d
    for T_, C_ in ((1, 1), (16384, 4096), (5, 16384)):
        assert lib.gdr_residual_norm_bwd_workspace_bytes(T_, C_) >= 12 * C_
    for d in (1, 64, 65, 128, 256):
        assert lib.gdr_attn_step_workspace_bytes(3, 8, 2, d) >= 2 * 16 * (d + 2) * 4
    assert lib.gdr_rec_checkpoint_rows(-1) == 0 and lib.gdr_rec_bwd_workspace_bytes(9, 0, 1, 0) == 0
    assert lib.gdr_gated_norm_bwd_workspace_bytes(9, 2, 1025) == 0
    assert lib.gdr_residual_norm_bwd_workspace_bytes(9, 16385) == 0
    assert lib.gdr_attn_step_workspace_bytes(3, 8, 2, 257) == 0


def test_the_binding_refuses(lib):  # noqa: F811
    x, h = torch.zeros(4, 8), torch.zeros(4, 2, 8)
    A, i32 = torch.zeros(8), torch.zeros(4, dtype=torch.int32)
    pages = torch.zeros(3, 4, 2, 8)
    table = torch.zeros(4, 3, dtype=torch.int32)
    for f in (lambda: gdr.rec_fwd(x, x, A), lambda: gdr.rec_bwd(x, x, A, x),
              lambda: gdr.rec_step(x, x, A, x), lambda: gdr.gated_norm_fwd(h, h),
              lambda: gdr.gated_norm_bwd(h, h, h), lambda: gdr.residual_norm_fwd(x, x),
              lambda: gdr.residual_norm_bwd(x, x, x), lambda: gdr.attn_step(h, pages, pages, table, i32),
              lambda: gdr.cache_plan(i32, i32, table, i32, i32[:1], 4, 4),
              lambda: gdr.cache_write(h, h, pages, pages, i32),
              lambda: gdr.rec_fwd(torch.zeros(4), x, A), lambda: gdr.gated_norm_fwd(x, x),
              lambda: gdr.gated_norm_fwd(h, h, activation="gelu")):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        gdr.rec_fwd(None, x, A)
    with pytest.raises(TypeError):
        gdr.attn_step(h, pages, pages, table, None)


def test_the_plan_by_hand():
    # pages of 4: request 0 has 3 tokens on page 9, wants 2; request 1 none, wants 5; request 2 waits
    table = [[9, -1], [-1, -1], [-1, -1]]
    slots, pos, cu, after, taken, table = ref.plan([3, 0, 0], [2, 5, 1], table, [7, 8, 5], 0, 4, 9)
    assert slots == [39, 28, 32, 33, 34, 35, 20, -1, -1]
    assert pos == [3, 4, 0, 1, 2, 3, 4, 0, 0]
    assert (cu, after, taken) == ([0, 2, 7, 7], [5, 5, 0], 3)
    assert table == [[9, 7], [8, 5], [-1, -1]]
