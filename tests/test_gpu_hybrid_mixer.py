"""The example's mixer, all operators together: a prompt and the tokens decoded after it against a
plain 64-bit mixer that runs token by token, and the gradients of a training step.

Tolerance of the outputs: what passes between the operators is rounded to bf16, at most 2^-9 of an
element each time: the projection, the convolution, q and k (which the delta rule multiplies), the
delta rule's own operands and its output, both branches' outputs and the last product: ten
roundings that add up like errors of random sign to sqrt(10) 2^-9 = 0.6 % of the outputs' norm;
three times that is allowed.  Gradients pass twice as many, 0.9 %, three times that; and the chunked
backward keeps a cosine of 0.9995 to its exact gradients, 3.2 % of their norm: 6 % in all."""
import importlib.util
import os

import pytest
import torch
from torch.nn import functional as F

import mixer_testlib as ref
from mixer_testlib import BF16

pytestmark = pytest.mark.gpu

_spec = importlib.util.spec_from_file_location(
    "hybrid_mixer", os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples",
                                 "hybrid_mixer.py"))


@pytest.fixture(scope="module")
def ex():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    if torch.cuda.get_device_capability() != (10, 3):
        pytest.skip("needs sm_103 (GB300)")
    m = importlib.util.module_from_spec(_spec)
    _spec.loader.exec_module(m)
    return m


def plain(m, p, hidden, pos, lengths):
    """The mixer in 64 bits on the CPU; p: its parameters and tables there."""
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    T = hidden.shape[0]
    both = hidden @ p["in_proj.weight"].t()
    C = sum(m.conv_sizes)
    dt, z, B, Cm, g, beta = both[:, C:].split(m.rest_sizes, 1)
    mixed, _, _ = ref.conv(both[:, :C], p["conv_weight"], p["conv_bias"], None, cu, True)
    q, k, v, x = mixed.split(m.conv_sizes, 1)
    q, k = (ref.qk_row(t.reshape(T, m.Hk, m.d), None, "l2", 1e-6, p["cos"], p["sin"], pos, False)
            for t in (q, k))
    v = v.reshape(T, m.H, m.d)
    g = -F.softplus(g + p["g_bias"])
    beta = torch.sigmoid(beta)
    o = []
    for s, e in zip(cu[:-1], cu[1:]):
        S = hidden.new_zeros(m.H, m.d, m.d)
        for t in range(s, e):
            y, S = ref.delta(q[t], k[t], v[t], g[t], beta[t], S, m.d ** -0.5)
            o.append(y[None])
    y, _, _ = ref.ssm(x, dt, -p["A_log"].exp(), B.reshape(T, m.G, m.N),
                      Cm.reshape(T, m.G, m.N), p["D"], z, p["dt_bias"], True, None, cu)
    return torch.cat([torch.cat(o).flatten(1), y], 1) @ p["out_proj.weight"].t()


def off(got, want):
    got, want = got.detach().cpu().double(), want.detach().double()
    return float((got - want).norm() / want.norm())


def parameters(mixer):
    p = {n: t.detach().cpu().double().requires_grad_() for n, t in mixer.named_parameters()}
    p.update({n: t.cpu().double() for n, t in mixer.named_buffers()})
    return p


@pytest.mark.parametrize("lengths,more", [([1, 70, 130], 5), ([3, 64], 2)])
def test_prompts_and_decoded_tokens(ex, lengths, more):
    torch.manual_seed(3)
    mixer = ex.HybridMixer(hidden=96, H=4, Hk=2, d=64, Dm=96, G=2, N=8, rot=32, places=256)
    whole = [n + more for n in lengths]
    hidden = torch.randn(sum(whole), 96).to(BF16)
    pos, cu = ex.place_of_tokens(whole, "cpu")
    with torch.no_grad():
        want = plain(mixer, parameters(mixer), hidden.double(), pos, whole)
    at = [int(c) for c in cu[:-1]]
    rows = torch.cat([torch.arange(a, a + n) for a, n in zip(at, lengths)])
    p, c = ex.place_of_tokens(lengths)
    out, states = mixer.prefill(hidden[rows].cuda(), p, c)
    assert off(out, want[rows]) < 0.018
    # decoding in the states' places in reverse order, behind a padded row
    order = list(range(len(lengths)))[::-1]
    slots = torch.tensor([-1, *order], dtype=torch.int32, device="cuda")
    got, rows = [], []
    for i in range(more):
        r = torch.tensor([at[n] + lengths[n] + i for n in order])
        token = torch.cat([hidden[:1], hidden[r]]).cuda()
        place = torch.tensor([0, *(lengths[n] + i for n in order)], dtype=torch.int32).cuda()
        y = mixer.step(token, place, states, slots)
        assert not y[0].any()
        got.append(y[1:])
        rows.append(r)
    assert off(torch.cat(got), want[torch.cat(rows)]) < 0.018


def test_training_step(ex):
    torch.manual_seed(4)
    lengths = [1, 66, 35]
    mixer = ex.HybridMixer(hidden=96, H=4, Hk=2, d=64, Dm=96, G=2, N=8, rot=32, places=256)
    hidden, dy = torch.randn(102, 96).to(BF16), torch.randn(102, 96).to(BF16)
    pos, cu = ex.place_of_tokens(lengths)
    out = mixer(hidden.cuda(), pos, cu)
    out.backward(dy.cuda())
    p = parameters(mixer)
    want = plain(mixer, p, hidden.double(), pos.cpu(), lengths)
    want.backward(dy.double())
    assert off(out, want) < 0.018
    for name, t in mixer.named_parameters():
        assert off(t.grad, p[name].grad) < 0.06, name
