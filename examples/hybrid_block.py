"""Blocks of a hybrid model from the library's operators: gated linear recurrences and attention in
turn, joined by residual norms.  Packed prompts, decoding one token at a time over the recurrences'
states and a paged key-value cache inside a CUDA graph, and a training step.

    hidden -> [norm -> block -> norm, gate, residual scale -> + residual] x layers -> norm
    recurrence block: in_proj -> x, r, i, z;  gated recurrence of x;  norm times gate z;  out_proj
    attention block:  qkv -> q/k norm and rotation -> attention over the request's tokens -> out_proj

Prompts' attention is PyTorch's; everything else is the library's.  Run it on a GB300 after building:

    python examples/hybrid_block.py --tokens 2048 --decode 64
"""
import argparse
import os
import sys

import torch
from torch import nn
from torch.nn import functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import chunked_gated_delta_gdr_gb300 as gdr

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class RecurrenceBlock(nn.Module):
    def __init__(self, hidden, D, heads, device):
        super().__init__()
        self.D, self.heads = D, heads
        kw = dict(device=device, dtype=BF16)
        self.in_proj = nn.Linear(hidden, 4 * D, bias=False, **kw)
        self.out_proj = nn.Linear(D, hidden, bias=False, **kw)
        # decays between 0.9 and 0.999 at an open gate, to the eighth power
        u = 0.9 + 0.099 * torch.rand(D, device=device, dtype=F32)
        self.A_log = nn.Parameter((-8 * u.log()).log())
        self.norm = nn.Parameter(torch.ones(D // heads, device=device, dtype=F32))

    def parts(self, y):
        """x, r, i, z: views of one product."""
        return self.in_proj(y).split(self.D, 1)

    def gated(self, y, z, norm):
        heads = lambda t: t.unflatten(1, (self.heads, -1))
        return self.out_proj(norm(heads(y), heads(z), self.norm).flatten(1))

    def forward(self, y, at):
        x, r, i, z = self.parts(y)
        y, _ = gdr.gated_recurrence(x, r, -self.A_log.exp(), i, cu_seqlens=at.cu)
        return self.gated(y, z, gdr.gated_norm)

    def prefill(self, y, at, state):
        x, r, i, z = self.parts(y)
        y, ht, _ = gdr.rec_fwd(x, r, -self.A_log.exp(), i, cu_seqlens=at.cu, output_final_state=True)
        state[at.slots.long()] = ht
        return self.gated(y, z, gdr.gated_norm_fwd)

    def step(self, y, at, state):
        x, r, i, z = self.parts(y)
        y = gdr.rec_step(x, r, -self.A_log.exp(), state, i, state_indices=at.slots)
        return self.gated(y, z, gdr.gated_norm_fwd)

    def room(self, cache):
        return torch.zeros(cache.requests, self.D, device=cache.device, dtype=F32)


class AttentionBlock(nn.Module):
    def __init__(self, hidden, Hq, Hk, d, places, device):
        super().__init__()
        self.sizes, self.d = (Hq, Hk, Hk), d
        kw = dict(device=device, dtype=BF16)
        self.qkv = nn.Linear(hidden, (Hq + 2 * Hk) * d, bias=False, **kw)
        self.out_proj = nn.Linear(Hq * d, hidden, bias=False, **kw)
        f = dict(device=device, dtype=F32)
        self.q_norm, self.k_norm = (nn.Parameter(torch.ones(d, **f)) for _ in range(2))
        angle = torch.arange(places, **f)[:, None] * 10000.0 ** (-torch.arange(d // 2, **f) * 2 / d)
        self.register_buffer("cos", angle.cos())
        self.register_buffer("sin", angle.sin())

    def heads(self, y, positions, norm):
        q, k, v = self.qkv(y).unflatten(1, (-1, self.d)).split(self.sizes, 1)
        q, k = norm(q, k, self.q_norm, self.k_norm, cos=self.cos, sin=self.sin, positions=positions)
        return q, k, v

    def prompt(self, q, k, v, at):
        """Causal attention inside each segment."""
        rep = self.sizes[0] // self.sizes[1]
        out = []
        for s, n in zip(at.starts, at.lengths):
            one = [t[s:s + n].transpose(0, 1)[None] for t in (q, k, v)]
            one[1:] = [t.repeat_interleave(rep, 1) for t in one[1:]]
            out.append(F.scaled_dot_product_attention(*one, is_causal=True)[0].transpose(0, 1))
        return self.out_proj(torch.cat(out).flatten(1))

    def forward(self, y, at):
        return self.prompt(*self.heads(y, at.positions, gdr.qk_norm_rotate), at)

    def prefill(self, y, at, pages):
        q, k, v = self.heads(y, at.positions, gdr.qk_fwd)
        gdr.cache_write(k, v, *pages, at.cells)
        return self.prompt(q, k, v, at)

    def step(self, y, at, pages):
        q, k, v = self.heads(y, at.positions, gdr.qk_fwd)
        gdr.cache_write(k, v, *pages, at.cells)
        o = gdr.attn_step(q, *pages, at.table, at.seen)
        return self.out_proj(o.flatten(1))

    def room(self, cache):
        shape = (cache.pages, cache.page, self.sizes[1], self.d)
        return [torch.zeros(shape, device=cache.device, dtype=BF16) for _ in range(2)]


class Cache:
    """What decoding keeps: each request's length and pages, and the blocks' states and pages."""

    def __init__(self, model, requests, pages, page=16, longest=4096, device="cuda"):
        self.requests, self.pages, self.page, self.device = requests, pages, page, device
        i32 = dict(device=device, dtype=I32)
        self.table = torch.full((requests, -(-longest // page)), -1, **i32)
        self.free = torch.arange(pages, **i32)
        self.taken, self.lengths = torch.zeros(1, **i32), torch.zeros(requests, **i32)
        self.one, self.rows = torch.ones(requests, **i32), torch.arange(requests, device=device)
        self.rooms = [b.room(self) for b in model.blocks]


class Place:
    """Where a call's tokens lie: positions, and what its blocks ask for."""

    def __init__(self, **kw):
        self.__dict__.update(kw)


def packed(lengths, device="cuda"):
    """The place of packed sequences of these lengths."""
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    pos = torch.cat([torch.arange(n) for n in lengths]).to(device, I32)
    return Place(lengths=lengths, starts=starts[:-1], positions=pos,
                 cu=torch.tensor(starts, dtype=I32, device=device),
                 slots=torch.arange(len(lengths), dtype=I32, device=device))


def granted(plan, request, token):
    """Slots and positions of a call's rows, from what cache_plan returned: row t is new token token[t] of
    request[t].  The plan packs the tokens that it grants, so that behind a request that is given fewer
    than it wants they are not where its rows are.  Rows that were given nothing: slot -1."""
    slots, positions, cu = plan[:3]
    at = cu[request] + token
    given = at < cu[request + 1]
    at = at.clamp(max=slots.shape[0] - 1)
    return torch.where(given, slots[at], -1), torch.where(given, positions[at], 0), given


class HybridBlocks(nn.Module):
    def __init__(self, hidden=1024, layers=4, D=1024, heads=8, Hq=8, Hk=2, d=128, places=65536,
                 device="cuda"):
        super().__init__()
        self.blocks = nn.ModuleList(
            AttentionBlock(hidden, Hq, Hk, d, places, device) if i % 2 else
            RecurrenceBlock(hidden, D, heads, device) for i in range(layers))
        f = dict(device=device, dtype=F32)
        self.norms = nn.ParameterList(torch.ones(hidden, **f) for _ in range(layers + 1))
        self.posts = nn.ParameterList(torch.ones(hidden, **f) for _ in range(layers))
        self.gates = nn.ParameterList(torch.ones(hidden, **f) for _ in range(layers))
        self.scale = layers ** -0.5

    def through(self, hidden, blocks, norm):
        """The residual stream is fp32; a block sees its norm in bf16."""
        y, h = norm(hidden, None, self.norms[0])
        h = h.float()
        for i, f in enumerate(blocks):
            y, h = norm(f(y), h, self.norms[i + 1], self.posts[i], self.gates[i], self.scale)
        return y

    def forward(self, hidden, at):
        """Differentiable: packed [T, hidden] -> [T, hidden]."""
        return self.through(hidden, [lambda y, b=b: b(y, at) for b in self.blocks], gdr.residual_norm)

    def plan(self, cache, new, most):
        return gdr.cache_plan(cache.lengths, new, cache.table, cache.free, cache.taken, cache.page, most,
                              cache.lengths, cache.taken)

    @torch.no_grad()
    def prefill(self, hidden, at, cache):
        """Packed prompts of the cache's requests, in their order.  Tokens for which there is no room are left
        out of the cache: cache.lengths then says less than their prompt's length."""
        new = torch.tensor(at.lengths, dtype=I32, device=cache.device)
        request = torch.repeat_interleave(cache.rows, new.long(), output_size=hidden.shape[0])
        at.cells, _, _ = granted(self.plan(cache, new, hidden.shape[0]), request, at.positions)
        return self.through(hidden, [lambda y, b=b, r=r: b.prefill(y, at, r)
                                     for b, r in zip(self.blocks, cache.rooms)],
                            gdr.residual_norm_fwd)

    @torch.no_grad()
    def step(self, hidden, cache):
        """One token of each request: hidden [requests, hidden].  A request without room for it is a padded row:
        its states and pages stay as they are, and its row of the result means nothing."""
        cells, pos, given = granted(self.plan(cache, cache.one, cache.requests), cache.rows, 0)
        at = Place(cells=cells, positions=pos, slots=torch.where(given, cache.rows, -1).to(I32),
                   table=cache.table, seen=torch.where(given, cache.lengths, 0))
        return self.through(hidden, [lambda y, b=b, r=r: b.step(y, at, r)
                                     for b, r in zip(self.blocks, cache.rooms)],
                            gdr.residual_norm_fwd)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=2048, help="tokens of the packed prompts")
    p.add_argument("--requests", type=int, default=4)
    p.add_argument("--decode", type=int, default=64, help="tokens decoded for each request")
    p.add_argument("--hidden", type=int, default=1024)
    a = p.parse_args()
    torch.manual_seed(0)
    model = HybridBlocks(hidden=a.hidden)
    cuts = sorted(torch.randint(1, a.tokens, (a.requests - 1,)).tolist())
    lengths = [e - s for s, e in zip([0, *cuts], [*cuts, a.tokens])]
    prompt = torch.randn(a.tokens, a.hidden, device="cuda", dtype=BF16)
    longest = max(lengths) + a.decode + 2
    pages = sum(-(-(n + a.decode + 2) // 16) for n in lengths)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(2):
        cache = Cache(model, a.requests, pages, longest=longest)
        start.record()
        model.prefill(prompt, packed(lengths), cache)
        end.record()
    torch.cuda.synchronize()
    print(f"prompts of {lengths} tokens: {start.elapsed_time(end):.3f} ms")

    # decoding: a step's launches are few and short, so they are captured once and replayed; the
    # cache's lengths and pages move on inside the graph
    token = torch.randn(a.requests, a.hidden, device="cuda", dtype=BF16)
    model.step(token, cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nxt = model.step(token, cache)
    start.record()
    for _ in range(a.decode):
        graph.replay()
        token.copy_(nxt)
    end.record()
    torch.cuda.synchronize()
    print(f"{a.decode} steps of {a.requests} requests: "
          f"{start.elapsed_time(end) / max(a.decode, 1):.4f} ms a step; lengths {cache.lengths.tolist()}")

    opt = torch.optim.Adam(model.parameters(), lr=1e-3)
    target = torch.randn_like(prompt)
    for i in range(3):
        opt.zero_grad()
        loss = F.mse_loss(model(prompt, packed(lengths)).float(), target.float())
        loss.backward()
        opt.step()
        print(f"training step {i}: loss {loss.item():.6f}")


if __name__ == "__main__":
    main()
