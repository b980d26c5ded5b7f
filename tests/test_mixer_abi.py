"""The mixer's operators without a GPU: malformed calls are refused before any device access, the
scratch that is asked for holds what the passes keep in it, and the Python binding refuses what
it cannot describe."""
import ctypes

import pytest
import torch

import chunked_gated_delta_gdr_gb300 as gdr
from chunked_gated_delta_gdr_gb300 import _native as nat

BF, F = nat.GDR_BF16, nat.GDR_F32
NULL, DTYPE, SHAPE, STRIDE, DIM, HEADS, NSEQ, OPTION = -1, -2, -3, -4, -5, -6, -7, -15


@pytest.fixture(scope="module")
def lib():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    return nat.lib()


class D:
    """A descriptor with a plausible device address."""

    def __init__(self, *shape, dtype=BF, strides=None):
        self.shape = (ctypes.c_int64 * 4)(*(list(shape) + [0] * (4 - len(shape))))
        self.strides = (ctypes.c_int64 * len(strides))(*strides) if strides else None
        self.t = nat.GdrTensor(ctypes.c_void_p(0x10000), dtype, len(shape), self.shape,
                               ctypes.cast(self.strides, ctypes.POINTER(ctypes.c_int64))
                               if strides else None)


def call(fn, args, **over):
    """fn's status with the named arguments replaced."""
    args = {**args, **over}
    assert set(over) <= set(args)
    return fn(*(ctypes.byref(a.t) if isinstance(a, D) else a for a in args.values()))


CU, WS = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x40000)
T, C, W, N_SEQ = 96, 64, 4, 2


def conv_fwd():
    return dict(x=D(T, C), weight=D(C, W, dtype=F), bias=D(C, dtype=F), h0=D(N_SEQ, W - 1, C),
                cu=CU, n_seq=N_SEQ, act=1, y=D(T, C), ht=D(N_SEQ, W - 1, C), stream=None)


def conv_bwd():
    return dict(x=D(T, C), weight=D(C, W, dtype=F), bias=D(C, dtype=F), h0=D(N_SEQ, W - 1, C),
                cu=CU, n_seq=N_SEQ, act=1, dy=D(T, C), dht=D(N_SEQ, W - 1, C), dx=D(T, C),
                dweight=D(C, W, dtype=F), dbias=D(C, dtype=F), dh0=D(N_SEQ, W - 1, C), ws=WS,
                ws_bytes=1 << 40, stream=None)


def conv_step():
    return dict(x=D(5, C), weight=D(C, W, dtype=F), bias=D(C, dtype=F), state=D(9, W - 1, C),
                idx=CU, act=1, y=D(5, C), stream=None)


def ssm_in(n, Dm=64, G=2, N=16):
    return dict(x=D(n, Dm), dt=D(n, Dm), A=D(Dm, N, dtype=F), B=D(n, G, N), C=D(n, G, N),
                D=D(Dm, dtype=F), z=D(n, Dm), dt_bias=D(Dm, dtype=F), softplus=1)


def ssm_fwd():
    st = lambda: D(N_SEQ, 64, 16, dtype=F)
    return dict(ssm_in(T), h0=st(), cu=CU, n_seq=N_SEQ, y=D(T, 64), ht=st(), ws=WS,
                ws_bytes=1 << 40, stream=None)


def ssm_bwd():
    st = lambda: D(N_SEQ, 64, 16, dtype=F)
    return dict(ssm_in(T), h0=st(), cu=CU, n_seq=N_SEQ, dy=D(T, 64), dht=st(), dx=D(T, 64),
                ddt=D(T, 64), dA=D(64, 16, dtype=F), dB=D(T, 2, 16), dC=D(T, 2, 16),
                dD=D(64, dtype=F), dz=D(T, 64), ddt_bias=D(64, dtype=F), dh0=st(), ws=WS,
                ws_bytes=1 << 40, stream=None)


def ssm_step():
    return dict(ssm_in(5), state=D(9, 64, 16, dtype=F), idx=CU, y=D(5, 64), stream=None)


def qk_in():
    return dict(q=D(T, 4, 64), k=D(T, 2, 64), qw=D(64, dtype=F), kw=D(64, dtype=F), norm=0,
                eps=ctypes.c_float(1e-6), cos=D(100, 16, dtype=F), sin=D(100, 16, dtype=F),
                pos=CU, inter=0)


def qk_fwd():
    return dict(qk_in(), q_out=D(T, 4, 64), k_out=D(T, 2, 64), stream=None)


def qk_bwd():
    return dict(qk_in(), dqo=D(T, 4, 64), dko=D(T, 2, 64), dq=D(T, 4, 64), dk=D(T, 2, 64),
                dqw=D(64, dtype=F), dkw=D(64, dtype=F), ws=WS, ws_bytes=1 << 40, stream=None)


def delta_step():
    return dict(q=D(5, 2, 64), k=D(5, 2, 64), v=D(5, 4, 64), g=D(5, 4, dtype=F), beta=D(5, 4),
                scale=ctypes.c_float(0.125), state=D(9, 4, 64, 64, dtype=F), idx=CU,
                o=D(5, 4, 64), stream=None)


REFUSED = [
    (conv_fwd, dict(x=None), NULL), (conv_fwd, dict(weight=None), NULL),
    (conv_fwd, dict(cu=None), NULL), (conv_fwd, dict(x=D(T, C, dtype=nat.GDR_I32)), DTYPE),
    (conv_fwd, dict(y=D(T, C, dtype=F)), DTYPE), (conv_fwd, dict(bias=D(C)), DTYPE),
    (conv_fwd, dict(weight=D(C, 5, dtype=F)), DIM), (conv_fwd, dict(weight=D(C, 1, dtype=F)), DIM),
    (conv_fwd, dict(weight=D(C + 1, W, dtype=F)), SHAPE), (conv_fwd, dict(y=D(T - 1, C)), SHAPE),
    (conv_fwd, dict(x=D(T * C)), SHAPE), (conv_fwd, dict(x=D(1 << 31, C)), SHAPE),
    (conv_fwd, dict(h0=D(N_SEQ + 1, W - 1, C)), NSEQ), (conv_fwd, dict(n_seq=-1), NSEQ),
    (conv_fwd, dict(h0=D(N_SEQ, W, C)), SHAPE), (conv_fwd, dict(act=2), OPTION),
    (conv_fwd, dict(y=D(T, C, strides=[C - 1, 1])), STRIDE),
    (conv_fwd, dict(x=D(T, C, strides=[2 * C, 2])), STRIDE),
    (conv_fwd, dict(ht=D(N_SEQ, W - 1, C, strides=[W * C, C, 1])), STRIDE),
    (conv_bwd, dict(dy=None), NULL), (conv_bwd, dict(dweight=None), NULL),
    (conv_bwd, dict(dx=D(T, C, strides=[0, 1])), STRIDE),
    (conv_bwd, dict(dweight=D(C, W)), DTYPE), (conv_bwd, dict(dh0=D(1, W - 1, C)), NSEQ),
    (conv_step, dict(state=D(9, W, C)), SHAPE), (conv_step, dict(state=D(9, W - 1, C, dtype=F)),
                                                 DTYPE),
    (conv_step, dict(idx=None, state=D(4, W - 1, C)), SHAPE), (conv_step, dict(y=None), NULL),
    (ssm_fwd, dict(A=None), NULL), (ssm_fwd, dict(B=None), NULL), (ssm_fwd, dict(dt=None), NULL),
    (ssm_fwd, dict(A=D(64, 16)), DTYPE), (ssm_fwd, dict(z=D(T, 64, dtype=F)), DTYPE),
    (ssm_fwd, dict(B=D(T, 2, 65), C=D(T, 2, 65)), DIM),
    (ssm_fwd, dict(B=D(T, 3, 16), C=D(T, 3, 16)), HEADS), (ssm_fwd, dict(C=D(T, 2, 8)), SHAPE),
    (ssm_fwd, dict(B=D(T - 1, 2, 16)), SHAPE), (ssm_fwd, dict(softplus=2), OPTION),
    (ssm_fwd, dict(h0=D(1, 64, 16, dtype=F)), NSEQ),
    (ssm_fwd, dict(A=D(64, 16, dtype=F, strides=[20, 1])), STRIDE),
    (ssm_bwd, dict(dz=None), OPTION), (ssm_bwd, dict(z=None), OPTION),
    (ssm_bwd, dict(dA=None), NULL), (ssm_bwd, dict(ddt=None), NULL),
    (ssm_bwd, dict(dB=D(T, 2, 16, strides=[40, 16, 1])), STRIDE),
    (ssm_bwd, dict(dht=D(N_SEQ, 64, 8, dtype=F)), SHAPE),
    (ssm_step, dict(state=D(9, 64, 16)), DTYPE), (ssm_step, dict(state=D(9, 64, 8, dtype=F)),
                                                 SHAPE),
    (ssm_step, dict(idx=None, state=D(4, 64, 16, dtype=F)), SHAPE),
    (qk_fwd, dict(k=None), NULL), (qk_fwd, dict(pos=None), NULL), (qk_fwd, dict(sin=None), OPTION),
    (qk_fwd, dict(k=D(T, 2, 32)), SHAPE), (qk_fwd, dict(qw=D(63, dtype=F)), SHAPE),
    (qk_fwd, dict(cos=D(100, 33, dtype=F), sin=D(100, 33, dtype=F)), DIM),
    (qk_fwd, dict(sin=D(99, 16, dtype=F)), SHAPE), (qk_fwd, dict(norm=2), OPTION),
    (qk_fwd, dict(eps=ctypes.c_float(-1.0)), OPTION),
    (qk_fwd, dict(eps=ctypes.c_float(float("nan"))), OPTION),
    (qk_fwd, dict(inter=3), OPTION), (qk_fwd, dict(q_out=D(T, 4, 64, dtype=F)), DTYPE),
    (qk_fwd, dict(q=D(T, 4, 257), k=D(T, 2, 257)), DIM),
    (qk_fwd, dict(q_out=D(T, 4, 64, strides=[256, 32, 1])), STRIDE),
    (qk_bwd, dict(dq=D(T, 4, 64, strides=[0, 64, 1])), STRIDE), (qk_bwd, dict(dko=None), NULL),
    (qk_bwd, dict(dqw=D(64)), DTYPE),
    (delta_step, dict(q=None), NULL), (delta_step, dict(q=D(5, 2, 64, dtype=F)), DTYPE),
    (delta_step, dict(v=D(5, 3, 64), beta=D(5, 3), g=D(5, 3, dtype=F), o=D(5, 3, 64),
                      state=D(9, 3, 64, 64, dtype=F)), HEADS),
    (delta_step, dict(q=D(5, 2, 96), k=D(5, 2, 96), v=D(5, 4, 96), o=D(5, 4, 96),
                      state=D(9, 4, 96, 96, dtype=F)), DIM),
    (delta_step, dict(state=D(9, 4, 64, 64)), DTYPE), (delta_step, dict(g=D(5, 4)), DTYPE),
    (delta_step, dict(idx=None, state=D(4, 4, 64, 64, dtype=F)), SHAPE),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_refused_before_the_device(lib, case):
    make, over, code = REFUSED[case]
    assert call(getattr(lib, "gdr_" + make.__name__), make(), **over) == code


@pytest.mark.parametrize("make", [conv_fwd, conv_bwd, conv_step, ssm_fwd, ssm_bwd, ssm_step,
                                  qk_fwd, qk_bwd, delta_step])
def test_well_formed_calls_reach_the_device_check(lib, make):
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    # no GB300 here: the device check or the CUDA call behind it fails
    assert call(getattr(lib, "gdr_" + make.__name__), make()) in (-10, -12)


def test_scratch_sizes(lib):
    for T_, C_, W_ in ((1, 1, 2), (17, 64, 4), (16384, 6144, 4), (70000, 8, 3)):
        assert lib.gdr_conv_bwd_workspace_bytes(T_, C_, W_) >= (W_ + 1) * C_ * 4
    for T_, D_, N_, G_ in ((1, 1, 1, 1), (1000, 96, 5, 3), (8192, 2048, 16, 1), (300, 640, 64, 4),
                           (5003, 4096, 16, 1)):
        # dB and dC: parts of at least one channel tile a group; a state and a gradient of one range
        need = 8 * T_ * G_ * N_ + 8 * D_ * N_
        assert lib.gdr_ssm_bwd_workspace_bytes(T_, D_, N_, G_) >= need
        # with ranges of 64 tokens at most, those of every range
        assert lib.gdr_ssm_bwd_workspace_bytes(T_, D_, N_, G_) >= 8 * D_ * N_ * -(-T_ // 64)
        # the forward asks for none where one range is enough, else for two ranges' states at least
        fwd = lib.gdr_ssm_fwd_workspace_bytes(T_, D_, N_, G_)
        assert fwd == 0 or fwd >= 2 * D_ * (N_ + 1) * 4
    for d in (1, 64, 152, 256):
        assert lib.gdr_qk_bwd_workspace_bytes(100, 4, 2, d) >= 2 * d * 4
    for bad in ((-1, 64, 16, 1), (10, 0, 16, 1), (10, 64, 0, 1), (10, 64, 65, 1), (10, 64, 16, 5)):
        assert lib.gdr_ssm_fwd_workspace_bytes(*bad) == 0
        assert lib.gdr_ssm_bwd_workspace_bytes(*bad) == 0
    assert lib.gdr_conv_bwd_workspace_bytes(10, 64, 5) == 0


def test_option_status_has_a_text(lib):
    assert lib.gdr_status_string(OPTION).decode() != "unknown status"


def test_host_tensors_are_refused(lib):
    x, w = torch.zeros(4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError):
        gdr.conv_fwd(x, w)
    with pytest.raises(ValueError):
        gdr.conv_step(x, w, torch.zeros(4, 3, 8))
    with pytest.raises(ValueError):
        gdr.ssm_fwd(x, x, w, torch.zeros(4, 1, 4), torch.zeros(4, 1, 4))
    h = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError):
        gdr.qk_fwd(h, h)
    with pytest.raises(ValueError):
        gdr.delta_step(h, h, h, x, x, torch.zeros(4, 2, 8, 8))
    with pytest.raises(TypeError):
        gdr.conv_fwd(None, w)
    with pytest.raises(ValueError):
        gdr.conv_fwd(torch.zeros(4), w)


def test_an_unknown_activation_is_refused(lib):
    with pytest.raises((ValueError, gdr.GdrError)):
        gdr.conv_fwd(torch.zeros(4, 8), torch.zeros(8, 4), activation="gelu")
