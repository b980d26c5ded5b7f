"""The mixer's calls as users vary them."""
import pytest
import torch

import chunked_gated_delta_gdr_gb300 as gdr
import mixer_testlib as ref
from mixer_testlib import BF16, F32, assert_close

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    if torch.cuda.get_device_capability() != (10, 3):
        pytest.skip("needs sm_103 (GB300)")


def normal(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s, std=1.0, dtype=F32: (std * torch.randn(*s, generator=g, device=DEV)).to(dtype)


# ------------------------------------------------------------------ final states given

def test_a_final_state_that_is_given_is_written():
    """With or without output_final_state: a caller that hands over a buffer decodes from it."""
    r = normal(1)
    cu = torch.tensor([0, 30, 50], dtype=torch.int32, device=DEV)
    x, w = r(50, 64, dtype=BF16), r(64, 4)
    _, want = gdr.conv_fwd(x, w, cu_seqlens=cu, output_final_state=True)
    buf = torch.full_like(want, 9.0)
    _, ht = gdr.conv_fwd(x, w, cu_seqlens=cu, final_state=buf)
    assert ht is not None and ht.data_ptr() == buf.data_ptr() and torch.equal(buf, want)
    A, B = -r(64, 16).abs(), r(50, 1, 16, dtype=BF16)
    _, want = gdr.ssm_fwd(x, x, A, B, B, cu_seqlens=cu, output_final_state=True)
    buf = torch.full_like(want, 9.0)
    _, ht = gdr.ssm_fwd(x, x, A, B, B, cu_seqlens=cu, final_state=buf)
    assert ht is not None and ht.data_ptr() == buf.data_ptr() and torch.equal(buf, want)
    assert gdr.conv_fwd(x, w, cu_seqlens=cu)[1] is None
    assert gdr.ssm_fwd(x, x, A, B, B, cu_seqlens=cu)[1] is None


# ------------------------------------------------------------------ alignment of a step's parameters

def off(t, by):
    """The same values, compact, `by` elements behind a 16-byte boundary."""
    flat = torch.empty(t.numel() + 4, dtype=t.dtype, device=t.device)
    view = flat[by:by + t.numel()].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("N", [16, 5])
@pytest.mark.parametrize("a_off,s_off", [(1, 0), (0, 1), (3, 2), (2, 0)])
def test_state_space_step_with_parameters_anywhere(N, a_off, s_off):
    """A and the pool at any float: a channel slice of a larger parameter, a view into a flat buffer.
    The prompt's call takes the same A."""
    B, D, slots = 3, 72, 5
    r = normal(N)
    x, z, dt = r(B, D, dtype=BF16), r(B, D, dtype=BF16), r(B, D, dtype=BF16, std=0.5)
    A, skip, bias = -r(D, N).abs(), r(D), r(D, std=0.3)
    Bv, Cv = r(B, 1, N, dtype=BF16), r(B, 1, N, dtype=BF16)
    st = r(slots, D, N)
    idx = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    pool = off(st, s_off)
    y = gdr.ssm_step(x, dt, off(A, a_off), Bv, Cv, pool, skip, z, bias, True, idx)
    for row, slot in enumerate(idx.tolist()):
        one = [t[row:row + 1].double().cpu() for t in (x, dt, Bv, Cv, z)]
        yr, hr, _ = ref.ssm(one[0], one[1], A.double().cpu(), one[2], one[3], skip.double().cpu(),
                            one[4], bias.double().cpu(), True, st[slot:slot + 1].double().cpu(), [0, 1])
        assert_close(y[row:row + 1], yr, 4, "y")
        assert_close(pool[slot:slot + 1], hr, 4, "state")
    for slot in (1, 3):
        assert torch.equal(pool[slot], st[slot])
    yp, _ = gdr.ssm_fwd(x, dt, off(A, a_off), Bv, Cv)
    ya, _ = gdr.ssm_fwd(x, dt, A, Bv, Cv)
    assert_close(yp, ya.double().cpu(), 4, "prompt")


# ------------------------------------------------------------------ steps of no length, states that last

def states_kept(T, D, N, cu, zero, dtype=F32):
    """Forward and backward of segments whose tokens must not change a state: steps of zero, or
    A = 0 and nothing added."""
    r = normal(T + D)
    n = len(cu) - 1
    x, B, C = r(T, D, dtype=dtype), r(T, 1, N, dtype=dtype), r(T, 1, N, dtype=dtype)
    A, dt, h0, dht = -r(D, N).abs() - 0.1, r(T, D).abs().to(dtype), r(n, D, N), r(n, D, N)
    if zero == "dt":
        dt = torch.zeros_like(dt)
    else:
        A, x = torch.zeros_like(A), torch.zeros_like(x)
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    _, ht = gdr.ssm_fwd(x, dt, A, B, C, dt_softplus=False, initial_state=h0, cu_seqlens=cud,
                        output_final_state=True)
    assert torch.equal(ht, h0), "states"
    g = gdr.ssm_bwd(x, dt, A, B, C, torch.zeros_like(x), dt_softplus=False, initial_state=h0,
                    cu_seqlens=cud, dfinal_state=dht)
    assert torch.equal(g[8], dht), "gradients of the states"


@pytest.mark.parametrize("zero", ["dt", "A"])
@pytest.mark.parametrize("T,D,N,cu", [
    (260, 64, 16, list(range(0, 261, 2))),    # tiles that a bound cuts short
    (300, 48, 5, [0, 1, 100, 103, 300]),
    (700, 36, 64, [0, 700]),
    (1501, 2048, 16, [0, 700, 701, 1501]),
    (1300, 4096, 8, [0, 1300]),
    (5003, 4096, 16, [0, 2101, 5003]),        # one thread a channel
])
def test_states_that_must_last_are_kept_exactly(T, D, N, cu, zero):
    states_kept(T, D, N, cu, zero)


def test_states_beside_one_that_must_last():
    """One state of each channel with A = 0, the others decaying."""
    r = normal(6)
    T, D, N = 600, 64, 16
    A, h0 = -r(D, N).abs() - 0.1, r(1, D, N)
    A[:, 3] = 0
    x, B = torch.zeros(T, D, device=DEV), r(T, 1, N)
    dt = r(T, D).abs() * 0.01
    _, ht = gdr.ssm_fwd(x, dt, A, B, B, dt_softplus=False, initial_state=h0, output_final_state=True)
    want = h0.double() * torch.exp(dt.double().sum(0)[:, None] * A.double())
    assert torch.equal(ht[:, :, 3], h0[:, :, 3])
    assert_close(ht, want, 600, "states")


@pytest.mark.parametrize("zero", ["dt", "A"])
@pytest.mark.parametrize("D,N,G", [(128, 16, 1), (100, 16, 2), (48, 5, 1), (64, 64, 1)])
def test_steps_that_must_keep_a_state(D, N, G, zero):
    r = normal(D)
    x, B, C = r(3, D), r(3, G, N), r(3, G, N)
    A, dt, st = -r(D, N).abs() - 0.1, r(3, D).abs(), r(3, D, N)
    if zero == "dt":
        dt = torch.zeros_like(dt)
    else:
        A, x = torch.zeros_like(A), torch.zeros_like(x)
    pool = st.clone()
    for _ in range(50):
        gdr.ssm_step(x, dt, A, B, C, pool, dt_softplus=False)
    assert torch.equal(pool, st)


# ------------------------------------------------------------------ derivatives of derivatives

def test_second_derivatives_are_refused():
    """The backwards are kernels without a derivative: a loss of their gradients is an error, where
    the gradients' share of it would otherwise be left out."""
    r = normal(2)
    x, w = r(20, 64).requires_grad_(), r(64, 4).requires_grad_()
    A, B = (-r(64, 16).abs()).requires_grad_(), r(20, 1, 16)
    q = r(20, 2, 64).requires_grad_()
    for f, leaf in ((lambda: gdr.short_conv(x, w)[0], x),
                    (lambda: gdr.selective_ssm(x, x, A, B, B)[0], A),
                    (lambda: gdr.qk_norm_rotate(q, q)[0], q)):
        for loss in (lambda y: (y * y).sum(), lambda y: y.sum()):  # with and without y's own gradient
            value = loss(f())
            grad, = torch.autograd.grad(value, leaf, create_graph=True)
            with pytest.raises(RuntimeError, match="first derivatives only"):
                (value + (grad * grad).sum()).backward()
            plain, = torch.autograd.grad(loss(f()), leaf)
            assert torch.equal(grad, plain)
    # gradients that keep their graph can still be added up and set to zero
    for _ in range(2):
        gdr.short_conv(x, w)[0].sum().backward(create_graph=True)
    torch.optim.SGD([x, w], 0.1).zero_grad(set_to_none=False)
    assert float(x.grad.abs().sum()) == 0


def test_second_derivatives_of_the_chunk_function_are_refused():
    from chunked_gated_delta_gdr_gb300.inputs import make_workload
    w = make_workload("twice", 3, [70, 30], 1, 2, 64).to(DEV)
    leaves = [t.detach().requires_grad_() for t in (w.q, w.k, w.v, w.g, w.beta)]

    def value():
        return gdr.chunk_gated_delta_rule(*leaves, scale=w.scale, cu_seqlens=w.cu_seqlens)[0].float().sum()

    v = value()
    grads = torch.autograd.grad(v, leaves, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        (v + sum((t.float() ** 2).sum() for t in grads)).backward()
    for a, b in zip(torch.autograd.grad(value(), leaves), grads):
        assert torch.equal(a, b)
