"""Requests that are given no place in the cache, among others that are: the example's prompts and steps, and
the README's step.  The others' outputs are those of plain 64-bit blocks, with the tolerance of the example's
own test; nothing is written into another request's pages."""
import os
import re

import pytest
import torch

import block_testlib as ref
import chunked_gated_delta_gdr_gb300 as gdr
from mixer_testlib import BF16
from test_gpu_hybrid_block import ex, off, parameters, plain, small  # noqa: F401

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "README.md")


def keys_of(cache, room, request, n):
    """The first n keys and values of a request, through the table."""
    table = cache.table[request].long()
    at = torch.arange(n, device=table.device)
    return [t[table[at // cache.page], at % cache.page].clone() for t in room]


# prompts, tokens of a request at most, pages, tokens that each request is given beside its prompt
DECODE = [([5, 8, 6], 8, 20, [3, 0, 2]),    # the one in the middle has a full row
          ([8, 3, 8, 4], 8, 20, [0, 5, 0, 4]),
          ([4, 4, 3], 40, 4, [4, 0, 1])]    # pages run out: the first takes the last, the third has a place left


@pytest.mark.parametrize("lengths,longest,pages,more", DECODE)
def test_steps_of_requests_without_room(ex, lengths, longest, pages, more):  # noqa: F811
    model = small(ex)
    whole = [n + m for n, m in zip(lengths, more)]
    hidden = torch.randn(sum(whole), 96).to(BF16)
    with torch.no_grad():
        want = plain(model, parameters(model), hidden.double(), whole)
    at = [sum(whole[:n]) for n in range(len(whole))]
    rows = torch.cat([torch.arange(a, a + n) for a, n in zip(at, lengths)])
    cache = ex.Cache(model, len(lengths), pages=pages, page=4, longest=longest)
    model.prefill(hidden[rows].cuda(), ex.packed(lengths), cache)
    assert cache.lengths.tolist() == lengths
    still = [b for b, m in enumerate(more) if m == 0]
    before = {b: [keys_of(cache, r, b, lengths[b]) if isinstance(r, list) else r[b].clone()
                  for r in cache.rooms] for b in still}
    token = torch.empty(len(lengths), 96, dtype=BF16, device="cuda")
    got, graph = [], None
    for i in range(max(more)):
        live = [b for b, m in enumerate(more) if i < m]
        token.normal_()  # of the others: anything
        r = torch.tensor([at[b] + lengths[b] + i for b in live])
        token[live] = hidden[r].cuda()
        if i == 0:
            y = model.step(token, cache)
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    y = model.step(token, cache)
            graph.replay()
        got.append((y[live].clone(), r))
        for b in live:
            assert int(cache.lengths[b]) == lengths[b] + i + 1
    assert cache.lengths.tolist() == whole
    y, r = (torch.cat(t) for t in zip(*got))
    assert off(y, want[r]) < 0.03
    for b in still:  # states and pages as they were
        for old, room in zip(before[b], cache.rooms):
            if isinstance(room, list):
                assert all(torch.equal(a, c) for a, c in zip(old, keys_of(cache, room, b, lengths[b])))
            else:
                assert torch.equal(old, room[b])


def test_prompts_longer_than_their_row(ex):  # noqa: F811
    # the second prompt's last token has no place: it goes nowhere, and the third's tokens to their own
    model = small(ex)
    lengths, has = [6, 9, 3], [6, 8, 3]
    hidden = torch.randn(sum(lengths), 96).to(BF16).cuda()
    caches = [ex.Cache(model, 3, pages=20, page=4, longest=n) for n in (8, 12)]
    for cache in caches:
        model.prefill(hidden, ex.packed(lengths), cache)
    assert caches[0].lengths.tolist() == has and caches[1].lengths.tolist() == lengths
    for short, full in zip(*(c.rooms for c in caches)):
        if isinstance(short, list):
            for b in range(3):
                for a, c in zip(keys_of(caches[0], short, b, has[b]), keys_of(caches[1], full, b, has[b])):
                    assert torch.equal(a, c)


def test_the_readme_step(ex):  # noqa: F811
    block = re.search(r"((?:    .*\n)*    slots, pos, cu, lengths, taken = (?:.*\n)(?:    .*\n)*)",
                      open(README).read()).group(1)
    code = "\n".join(line[4:] for line in block.splitlines())
    gen = torch.Generator().manual_seed(4)
    B, Hq, Hk, d, page = 4, 4, 2, 64, 4
    lens, new = [5, 8, 0, 6], [1, 1, 0, 1]  # the second has a full row, the third wants nothing
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table = i32([[0, 1], [2, 3], [-1, -1], [4, 5]])
    kc, vc = (torch.randn(8, page, Hk, d, generator=gen).to(BF16).cuda() for _ in range(2))
    q = torch.randn(B, Hq, d, generator=gen).to(BF16).cuda()
    k, v = (torch.randn(B, Hk, d, generator=gen).to(BF16).cuda() for _ in range(2))
    wk, wv = kc.clone(), vc.clone()
    for b, (p, place) in {0: (1, 1), 3: (5, 2)}.items():
        wk[p, place], wv[p, place] = k[b], v[b]
    space = dict(gdr=gdr, torch=torch, lengths=i32(lens), new=i32(new), table=table, free=i32([6, 7]),
                 taken=i32([0]), page=page, B=B, q=q, k=k, v=v, k_cache=kc, v_cache=vc)
    exec(code, space)
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    assert space["lengths"].tolist() == [6, 8, 0, 7] and space["taken"].tolist() == [0]
    want, tol = ref.attention(q.cpu(), wk.cpu(), wv.cpu(), table.cpu(), [6, 0, 0, 7], d ** -0.5, 0)
    ref.assert_attention(space["o"], want, tol)
