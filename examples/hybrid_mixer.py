"""A token mixer with two branches, built from the library's operators: packed prompts, decoding
one token at a time from their states, and a training step.

    hidden -> in_proj -> convolution -> q, k -> norm + rotation -> gated delta rule -+-> out_proj
                                     -> x (with dt, B, C, z)    -> state space scan -+

Run it on a GB300 after building the library:

    python examples/hybrid_mixer.py --tokens 2048 --decode 64
"""
import argparse
import os
import sys

import torch
from torch import nn
from torch.nn import functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import chunked_gated_delta_gdr_gb300 as gdr

BF16, F32 = torch.bfloat16, torch.float32


class HybridMixer(nn.Module):
    """H value heads over Hk query/key heads of d for the delta rule; Dm channels in G groups with
    N states each for the state space branch; one convolution of W taps in front of both."""

    def __init__(self, hidden=1024, H=8, Hk=4, d=128, Dm=1024, G=1, N=16, W=4, rot=64,
                 places=65536, device="cuda"):
        super().__init__()
        self.H, self.Hk, self.d, self.Dm, self.G, self.N, self.W = H, Hk, d, Dm, G, N, W
        self.conv_sizes = [Hk * d, Hk * d, H * d, Dm]
        self.rest_sizes = [Dm, Dm, G * N, G * N, H, H]
        C = sum(self.conv_sizes)
        kw = dict(device=device, dtype=BF16)
        self.in_proj = nn.Linear(hidden, C + sum(self.rest_sizes), bias=False, **kw)
        self.out_proj = nn.Linear(H * d + Dm, hidden, bias=False, **kw)
        f = dict(device=device, dtype=F32)
        self.conv_weight = nn.Parameter(torch.randn(C, W, **f) * W ** -0.5)
        self.conv_bias = nn.Parameter(torch.zeros(C, **f))
        self.A_log = nn.Parameter(torch.arange(1, N + 1, **f).log().repeat(Dm, 1))
        self.D = nn.Parameter(torch.ones(Dm, **f))
        self.dt_bias = nn.Parameter(torch.full((Dm,), -2.0, **f))
        self.g_bias = nn.Parameter(torch.full((H,), -2.0, **f))
        angle = torch.arange(places, **f)[:, None] * \
            10000.0 ** (-torch.arange(rot // 2, **f) * 2 / rot)
        self.register_buffer("cos", angle.cos())
        self.register_buffer("sin", angle.sin())

    def project(self, hidden):
        """The convolution's input and the other branches' inputs, views of one product."""
        C = sum(self.conv_sizes)
        both = self.in_proj(hidden)
        dt, z, B, Cm, g, beta = both[:, C:].split(self.rest_sizes, 1)
        n = hidden.shape[0]
        g = -F.softplus(g.float() + self.g_bias)
        return (both[:, :C], dt, z, B.view(n, self.G, self.N), Cm.view(n, self.G, self.N), g,
                torch.sigmoid(beta.float()).to(BF16))

    def heads(self, mixed):
        q, k, v, x = mixed.split(self.conv_sizes, 1)
        n = mixed.shape[0]
        return (q.view(n, self.Hk, self.d), k.view(n, self.Hk, self.d),
                v.view(n, self.H, self.d), x)

    def forward(self, hidden, positions, cu_seqlens):
        """Differentiable: [T, hidden] -> [T, hidden]."""
        c, dt, z, B, Cm, g, beta = self.project(hidden)
        mixed, _ = gdr.short_conv(c, self.conv_weight, self.conv_bias, cu_seqlens=cu_seqlens)
        q, k, v, x = self.heads(mixed)
        q, k = gdr.qk_norm_rotate(q, k, norm="l2", cos=self.cos, sin=self.sin,
                                  positions=positions)
        o, _ = gdr.chunk_gated_delta_rule(q, k, v.contiguous(), g, beta, cu_seqlens=cu_seqlens)
        y, _ = gdr.selective_ssm(x, dt, -self.A_log.exp(), B, Cm, self.D, z, self.dt_bias,
                                 cu_seqlens=cu_seqlens)
        return self.out_proj(torch.cat([o.flatten(1), y], 1))

    @torch.no_grad()
    def prefill(self, hidden, positions, cu_seqlens):
        """Packed prompts: the output and the states after each of them."""
        c, dt, z, B, Cm, g, beta = self.project(hidden)
        mixed, conv = gdr.conv_fwd(c, self.conv_weight, self.conv_bias, cu_seqlens=cu_seqlens,
                                   output_final_state=True)
        q, k, v, x = self.heads(mixed)
        q, k = gdr.qk_fwd(q, k, norm="l2", cos=self.cos, sin=self.sin, positions=positions)
        o, delta = gdr.chunk_fwd(q, k, v, g, beta, cu_seqlens=cu_seqlens,
                                 output_final_state=True)
        y, ssm = gdr.ssm_fwd(x, dt, -self.A_log.exp(), B, Cm, self.D, z, self.dt_bias,
                             cu_seqlens=cu_seqlens, output_final_state=True)
        return self.out_proj(torch.cat([o.flatten(1), y], 1)), (conv, delta, ssm)

    @torch.no_grad()
    def step(self, hidden, positions, states, slots=None):
        """One token of each request, the states advanced in place.  slots [B] int32: each row's
        place in the states (None: row i, place i; negative: a padded row)."""
        conv, delta, ssm = states
        c, dt, z, B, Cm, g, beta = self.project(hidden)
        mixed = gdr.conv_step(c, self.conv_weight, conv, self.conv_bias, state_indices=slots)
        q, k, v, x = self.heads(mixed)
        q, k = gdr.qk_fwd(q, k, norm="l2", cos=self.cos, sin=self.sin, positions=positions)
        o = gdr.delta_step(q, k, v, g, beta, delta, state_indices=slots)
        y = gdr.ssm_step(x, dt, -self.A_log.exp(), B, Cm, ssm, self.D, z, self.dt_bias,
                         state_indices=slots)
        return self.out_proj(torch.cat([o.flatten(1), y], 1))


def place_of_tokens(lengths, device="cuda"):
    """(positions [T], cu_seqlens [N + 1]), int32, of packed segments of these lengths."""
    pos = torch.cat([torch.arange(n) for n in lengths]).to(torch.int32)
    cu = torch.tensor([0, *lengths]).cumsum(0).to(torch.int32)
    return pos.to(device), cu.to(device)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=2048, help="tokens of the packed prompts")
    p.add_argument("--requests", type=int, default=4)
    p.add_argument("--decode", type=int, default=64, help="tokens decoded for each request")
    p.add_argument("--hidden", type=int, default=1024)
    a = p.parse_args()
    torch.manual_seed(0)
    mixer = HybridMixer(hidden=a.hidden)
    cuts = sorted(torch.randint(1, a.tokens, (a.requests - 1,)).tolist())
    lengths = [e - s for s, e in zip([0, *cuts], [*cuts, a.tokens])]
    pos, cu = place_of_tokens(lengths)
    prompt = torch.randn(a.tokens, a.hidden, device="cuda", dtype=BF16)

    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    mixer.prefill(prompt, pos, cu)
    start.record()
    out, states = mixer.prefill(prompt, pos, cu)
    end.record()
    torch.cuda.synchronize()
    print(f"prompts of {lengths} tokens: {start.elapsed_time(end):.3f} ms")

    # decoding: a step's launches are few and short, so they are captured once and replayed
    token = torch.randn(a.requests, a.hidden, device="cuda", dtype=BF16)
    at = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    saved = [s.clone() for s in states]
    mixer.step(token, at, states)
    for s, b in zip(states, saved):
        s.copy_(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nxt = mixer.step(token, at, states)

    def decode(n):
        for _ in range(n):
            graph.replay()
            token.copy_(F.normalize(nxt.float(), dim=-1) * a.hidden ** 0.5)
            at.add_(1)

    decode(1)
    for s, b in zip(states, saved):
        s.copy_(b)
    at.sub_(1)
    start.record()
    decode(a.decode)
    end.record()
    torch.cuda.synchronize()
    print(f"{a.decode} steps of {a.requests} requests: "
          f"{start.elapsed_time(end) / max(a.decode, 1):.4f} ms a step")

    opt = torch.optim.Adam(mixer.parameters(), lr=1e-3)
    target = torch.randn_like(prompt)
    for i in range(3):
        opt.zero_grad()
        loss = F.mse_loss(mixer(prompt, pos, cu).float(), target.float())
        loss.backward()
        opt.step()
        print(f"training step {i}: loss {loss.item():.6f}")


if __name__ == "__main__":
    main()
