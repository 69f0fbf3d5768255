"""A small gated-delta-rule language model on the library's operators.

    python examples/gated_delta.py [--steps 200]

It trains on associative recall (pairs "key value", then keys whose values are
asked for), the task the delta rule's overwriting memory is made for, then
serves: prompts are prefilled into slots of one pool of states, and tokens are
decoded one at a time from it.  Training runs qk_rope and causal_product_delta
with autograd; serving runs causal_product_qk_rope, causal_product_fwd_delta
and causal_product_decode_delta on the same weights, and its logits are
compared with the training pass's.  Everything is synthetic.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn as nn
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import prefix_sum_outer_gb300 as cp  # noqa: E402


def rotation(positions: torch.Tensor, half: int):
    """cos, sin of the positions' angles: float32 [.., half]."""
    freq = 10000.0 ** (-torch.arange(half, device=positions.device, dtype=torch.float32) / half)
    angle = positions.float()[..., None] * freq
    return angle.cos(), angle.sin()


class Layer(nn.Module):
    """x + mix(norm x), then x + mlp(norm x); the mix is the gated delta rule
    with ``heads`` value heads on ``key_heads`` query/key heads."""

    def __init__(self, width: int, heads: int, key_heads: int, dim: int):
        super().__init__()
        self.heads, self.key_heads, self.dim = heads, key_heads, dim
        self.norm1, self.norm2 = nn.RMSNorm(width), nn.RMSNorm(width)
        self.qk = nn.Linear(width, 2 * key_heads * dim, bias=False)
        self.v = nn.Linear(width, heads * dim, bias=False)
        self.gates = nn.Linear(width, 2 * heads)
        self.wq, self.wk = nn.Parameter(torch.ones(dim)), nn.Parameter(torch.ones(dim))
        self.out = nn.Linear(heads * dim, width, bias=False)
        self.up, self.down = nn.Linear(width, 2 * width), nn.Linear(2 * width, width)
        nn.init.zeros_(self.gates.weight)
        with torch.no_grad():  # a long memory to begin with: a = 0.98
            self.gates.bias.copy_(torch.cat([torch.full((heads,), -4.0), torch.zeros(heads)]))

    def project(self, x):
        """The raw q, k ([B,Hk,N,D] views of one projection), v, log decay and
        write strength of rows x [B,N,E]."""
        B, N, _ = x.shape
        y = self.norm1(x)
        qk = F.linear(y.bfloat16(), self.qk.weight.bfloat16())
        xq, xk = (t.view(B, N, self.key_heads, self.dim).transpose(1, 2) for t in qk.chunk(2, -1))
        v = F.linear(y.bfloat16(), self.v.weight.bfloat16())
        v = v.view(B, N, self.heads, self.dim).transpose(1, 2).contiguous()
        a, b = self.gates(y).chunk(2, -1)
        return (xq, xk, v, (-F.softplus(a)).transpose(1, 2).contiguous(),
                torch.sigmoid(b).transpose(1, 2).contiguous())

    def finish(self, x, o):
        """The layer's output from its input and the mix's out [B,H,N,D]."""
        B, _, N, _ = o.shape
        o = o.transpose(1, 2).reshape(B, N, self.heads * self.dim)
        x = x + F.linear(o, self.out.weight.bfloat16()).float()
        return x + self.down(F.silu(self.up(self.norm2(x))))

    def weights(self):
        return self.wq.bfloat16(), self.wk.bfloat16()

    def forward(self, x, cos, sin):
        xq, xk, v, g, beta = self.project(x)
        q, k = cp.qk_rope(xq, xk, *self.weights(), cos, sin, norm="l2")
        return self.finish(x, cp.causal_product_delta(q, k, v, g, beta))

    def prefill(self, x, cos, sin, state, slots):
        """forward, leaving every sequence's state in its slot of the pool."""
        xq, xk, v, g, beta = self.project(x)
        q, k = cp.causal_product_qk_rope(xq, xk, *self.weights(), cos, sin, norm="l2")
        o, s = cp.causal_product_fwd_delta(q, k, v, g, beta, return_state=True)
        state[slots.long()] = s
        return self.finish(x, o)

    def step(self, x, cos, sin, state, slots):
        """One token of every sequence: x [B,1,E], cos and sin [B,1,R/2]."""
        xq, xk, v, g, beta = self.project(x)
        q, k = cp.causal_product_qk_rope(xq, xk, *self.weights(), cos, sin, norm="l2")
        o = cp.causal_product_decode_delta(q[:, :, 0], k[:, :, 0], v[:, :, 0], g[:, :, 0],
                                           beta[:, :, 0], state, slots=slots)
        return self.finish(x, o[:, :, None])


class Model(nn.Module):
    def __init__(self, vocab: int, width: int = 128, layers: int = 2, heads: int = 4,
                 key_heads: int = 2, dim: int = 64):
        super().__init__()
        self.half = dim // 4  # half of the features turn
        # a place sees its token and the one before it
        self.embed, self.last = nn.Embedding(vocab, width), nn.Embedding(vocab, width)
        for e in (self.embed, self.last):
            nn.init.normal_(e.weight, std=0.05)
        self.layers = nn.ModuleList(Layer(width, heads, key_heads, dim) for _ in range(layers))
        self.norm = nn.RMSNorm(width)

    def head(self, x):
        return F.linear(self.norm(x), self.embed.weight)

    def rows(self, tokens):
        x = self.embed(tokens)
        return x + F.pad(self.last(tokens[:, :-1]), (0, 0, 1, 0))

    def forward(self, tokens):
        x = self.rows(tokens)
        cos, sin = rotation(torch.arange(tokens.shape[1], device=tokens.device), self.half)
        for layer in self.layers:
            x = layer(x, cos, sin)
        return self.head(x)

    def new_states(self, pool: int):
        """One pool of states per layer, for ``pool`` sequences."""
        dev = self.embed.weight.device
        return [torch.zeros(pool, l.heads, l.dim, l.dim, device=dev) for l in self.layers]

    @torch.no_grad()
    def prefill(self, tokens, states, slots):
        x = self.rows(tokens)
        cos, sin = rotation(torch.arange(tokens.shape[1], device=tokens.device), self.half)
        for layer, state in zip(self.layers, states):
            x = layer.prefill(x, cos, sin, state, slots)
        return self.head(x)

    @torch.no_grad()
    def step(self, tokens, last, positions, states, slots):
        """Logits [B,V] after one token of every sequence (tokens, the ones
        before them and positions [B], slots int32 [B]: each sequence's place
        in the pools)."""
        x = (self.embed(tokens) + self.last(last))[:, None]
        cos, sin = rotation(positions[:, None], self.half)
        for layer, state in zip(self.layers, states):
            x = layer.step(x, cos, sin, state, slots)
        return self.head(x)[:, 0]


def recall_batch(batch: int, pairs: int, asked: int, keys: int, values: int, gen, device):
    """Sequences k v k v .. then k v of keys seen before; the loss mask marks
    the places whose next token is an asked value."""
    ks = torch.stack([torch.randperm(keys, generator=gen)[:pairs] for _ in range(batch)])
    vs = keys + torch.randint(values, (batch, pairs), generator=gen)
    pick = torch.stack([torch.randperm(pairs, generator=gen)[:asked] for _ in range(batch)])
    told = torch.stack([ks, vs], -1).flatten(1)
    ask = torch.stack([ks.gather(1, pick), vs.gather(1, pick)], -1).flatten(1)
    tokens = torch.cat([told, ask], 1)
    mask = torch.zeros(tokens.shape, dtype=torch.bool)
    mask[:, 2 * pairs::2] = True
    return tokens.to(device), mask.to(device)


def train(model, steps: int, batch: int = 64, pairs: int = 24, seed: int = 0, log=print):
    gen = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3, weight_decay=0.01)
    dev = model.embed.weight.device
    losses = []
    for i in range(steps):
        tokens, mask = recall_batch(batch, pairs, 8, 64, 64, gen, dev)
        logits = model(tokens[:, :-1])
        loss = F.cross_entropy(logits[mask[:, :-1]], tokens[:, 1:][mask[:, :-1]])
        opt.zero_grad(set_to_none=True)
        loss.backward()
        nn.utils.clip_grad_norm_(model.parameters(), 1.0)
        opt.step()
        losses.append(float(loss.detach()))
        if log is not None and (i % 50 == 0 or i + 1 == steps):
            log(f"step {i:4d}  loss {losses[-1]:.3f}")
    return losses


@torch.no_grad()
def serve(model, batch: int = 6, pairs: int = 24, pool: int = 16, seed: int = 1):
    """(largest difference of the served logits from the full pass's, relative
    to the logits' size; share of asked values answered rightly)."""
    gen = torch.Generator().manual_seed(seed)
    dev = model.embed.weight.device
    tokens, mask = recall_batch(batch, pairs, 8, 64, 64, gen, dev)
    full = model(tokens)
    slots = torch.randperm(pool, generator=gen)[:batch].to(device=dev, dtype=torch.int32)
    states = model.new_states(pool)
    prompt = 2 * pairs
    got = [model.prefill(tokens[:, :prompt], states, slots)[:, -1]]
    for i in range(prompt, tokens.shape[1]):
        pos = torch.full((batch,), i, device=dev)
        got.append(model.step(tokens[:, i], tokens[:, i - 1], pos, states, slots))
    got, want = torch.stack(got, 1), full[:, prompt - 1:]
    asked = mask[:, prompt - 1:]
    right = got[:, :-1].argmax(-1)[asked[:, :-1]] == tokens[:, prompt:][asked[:, :-1]]
    return float((got - want).abs().max() / want.abs().max()), float(right.float().mean())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=300)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    model = Model(128).cuda()
    train(model, a.steps)
    diff, right = serve(model)
    print(f"served logits within {diff:.1e} of the full pass; {right:.0%} of the asked values right")


if __name__ == "__main__":
    main()
