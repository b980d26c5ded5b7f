"""The example's blocks, all operators together: prompts and the tokens decoded after them against
plain 64-bit blocks over the whole sequences, and the gradients of a training step.

Tolerance of the outputs: what passes between the operators is rounded to bf16, at most 2^-9 of an
element on average over its range each time.  A recurrence block rounds its input, the projection,
y, the gated norm and the last product; an attention block its input, the projection, q and k, the
probabilities and outputs of the prompt's attention and the last product: five and seven roundings,
and four blocks 24, and the last norm's.  Errors of random sign add up to sqrt(25) 2^-9 = 1 % of the
outputs' norm; three times that is allowed, and for gradients, which pass twice as many, 4.2 %."""
import importlib.util
import os

import pytest
import torch

import block_testlib as ref
import mixer_testlib as mref
from mixer_testlib import BF16

pytestmark = pytest.mark.gpu

_spec = importlib.util.spec_from_file_location(
    "hybrid_block", os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples",
                                 "hybrid_block.py"))


@pytest.fixture(scope="module")
def ex():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    if torch.cuda.get_device_capability() != (10, 3):
        pytest.skip("needs sm_103 (GB300)")
    m = importlib.util.module_from_spec(_spec)
    _spec.loader.exec_module(m)
    return m


def parameters(model):
    p = {n: t.detach().cpu().double().requires_grad_() for n, t in model.named_parameters()}
    p.update({n: t.cpu().double() for n, t in model.named_buffers()})
    return p


def plain(model, p, hidden, lengths):
    """All blocks in 64 bits on the CPU; p: the parameters and tables there."""
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    pos = torch.cat([torch.arange(n) for n in lengths])
    y, h = ref.residual(hidden, None, p["norms.0"], None, None, 1.0, 1e-6, False)
    for j, b in enumerate(model.blocks):
        w = lambda name: p[f"blocks.{j}.{name}"]
        if j % 2 == 0:
            x, r, i, z = (y @ w("in_proj.weight").t()).split(b.D, 1)
            o, _, _ = ref.rec(x, r, -w("A_log").exp(), i, True, None, cu)
            heads = lambda t: t.unflatten(1, (b.heads, -1))
            o = ref.gated(heads(o), heads(z), w("norm"), "silu", 1e-6).flatten(1)
        else:
            q, k, v = (y @ w("qkv.weight").t()).unflatten(1, (-1, b.d)).split(b.sizes, 1)
            q, k = (mref.qk_row(t, w(n), "rms", 1e-6, w("cos"), w("sin"), pos, False)
                    for t, n in ((q, "q_norm"), (k, "k_norm")))
            rep = b.sizes[0] // b.sizes[1]
            k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
            out = []
            for s, e in zip(cu[:-1], cu[1:]):
                a = torch.einsum("thd,shd->hts", q[s:e], k[s:e]) * b.d ** -0.5
                late = torch.ones(e - s, e - s).triu(1).bool()
                out.append(torch.einsum("hts,shd->thd", torch.softmax(
                    a.masked_fill(late, float("-inf")), -1), v[s:e]))
            o = torch.cat(out).flatten(1)
        y, h = ref.residual(o @ w("out_proj.weight").t(), h, p[f"norms.{j + 1}"], p[f"posts.{j}"],
                            p[f"gates.{j}"], model.scale, 1e-6, True)
    return y


def off(got, want):
    got, want = got.detach().cpu().double(), want.detach().double()
    return float((got - want).norm() / want.norm())


def small(ex):
    torch.manual_seed(3)
    return ex.HybridBlocks(hidden=96, layers=4, D=128, heads=2, Hq=4, Hk=2, d=64, places=512)


@pytest.mark.parametrize("lengths,more", [([1, 70, 130], 6), ([16, 33], 40)])
def test_prompts_and_decoded_tokens(ex, lengths, more):
    model = small(ex)
    whole = [n + more for n in lengths]
    hidden = torch.randn(sum(whole), 96).to(BF16)
    with torch.no_grad():
        want = plain(model, parameters(model), hidden.double(), whole)
    at = [sum(whole[:n]) for n in range(len(whole))]
    rows = torch.cat([torch.arange(a, a + n) for a, n in zip(at, lengths)])
    cache = ex.Cache(model, len(lengths), pages=sum(-(-n // 4) for n in whole) + 2, page=4, longest=200)
    out = model.prefill(hidden[rows].cuda(), ex.packed(lengths), cache)
    assert off(out, want[rows]) < 0.03
    # the rest token by token: two on their own, then replays of a captured step
    token = torch.empty(len(lengths), 96, dtype=BF16, device="cuda")
    got, graph = [], None
    for i in range(more):
        r = torch.tensor([a + n + i for a, n in zip(at, lengths)])
        token.copy_(hidden[r])
        if i < 2:
            got.append((model.step(token, cache).clone(), r))
            continue
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = model.step(token, cache)
        graph.replay()
        got.append((y.clone(), r))
    assert cache.lengths.tolist() == whole
    y, r = (torch.cat(t) for t in zip(*got))
    assert off(y, want[r]) < 0.03


def test_training_step(ex):
    model = small(ex)
    lengths = [1, 66, 35]
    hidden, dy = torch.randn(102, 96).to(BF16), torch.randn(102, 96).to(BF16)
    out = model(hidden.cuda(), ex.packed(lengths))
    out.backward(dy.cuda())
    p = parameters(model)
    want = plain(model, p, hidden.double(), lengths)
    want.backward(dy.double())
    assert off(out, want) < 0.03
    for name, t in model.named_parameters():
        assert off(t.grad, p[name].grad) < 0.042, name
