"""A small recurrent language model on the operators around the scan: token
embedding, and blocks of a short causal convolution and a gated recurrence.

Training runs packed documents (segment positions restart both the convolution
and the recurrence) through the autograd functions; serving keeps a pool of
windows and states, one slot a request, fills a request's slot from its prompt in
one call and then moves all requests on by a token a step.

    python examples/recurrent_lm.py        # trains on a toy corpus, then continues prompts
"""
from __future__ import annotations

import math
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_recurrence_scan_lrscan_gb300 import lrscan as L  # noqa: E402


def norm(x, weight):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight).to(x.dtype)


class Block(torch.nn.Module):
    """norm -> (recurrent branch: projection, convolution, gated recurrence) *
    (gelu branch) -> projection, added to the input."""

    def __init__(self, width: int, lanes: int, taps: int, dtype):
        super().__init__()
        self.lanes, self.taps = lanes, taps
        self.norm = torch.nn.Parameter(torch.ones(width))
        self.inp = torch.nn.Linear(width, 2 * lanes, bias=False, dtype=dtype)
        self.conv_w = torch.nn.Parameter(torch.randn(lanes, taps) / math.sqrt(taps))
        self.conv_b = torch.nn.Parameter(torch.zeros(lanes))
        self.gates = torch.nn.Linear(lanes, 2 * lanes, dtype=dtype)
        # a = exp(-8 softplus(lam) sigmoid(r)): decays of 0.9 to 0.999 where the gate is open
        decay = torch.linspace(0.9, 0.999, lanes)
        self.lam = torch.nn.Parameter(torch.log(torch.expm1(-torch.log(decay) / 8.0)))
        self.out = torch.nn.Linear(lanes, width, bias=False, dtype=dtype)

    def forward(self, x, segment_pos=None, window=None, state=None):
        """x [B, T, width]; returns (y, the last tokens of the window, the final state)."""
        u, v = self.inp(norm(x, self.norm)).split(self.lanes, -1)
        u, window = L.causal_conv(u, self.conv_w, self.conv_b, window, segment_pos)
        r, i = self.gates(u).split(self.lanes, -1)
        h, state = L.gate_scan(r, i, u, self.lam, state, segment_pos)
        return x + self.out(h * F.gelu(v)), window, state

    def step(self, x, windows, states, slots):
        """One token of each request, x [B, width]; its rows of the pools move on in place."""
        u, v = self.inp(norm(x, self.norm)).split(self.lanes, -1)
        u = L.lrscan_step_conv(u, self.conv_w, windows, bias=self.conv_b, slots=slots)
        r, i = self.gates(u).split(self.lanes, -1)
        h = L.lrscan_step_gates(r, i, u, self.lam, states, slots=slots)
        return x + self.out(h * F.gelu(v))


class RecurrentLM(torch.nn.Module):
    def __init__(self, vocab: int, width: int = 128, lanes: int = 192, blocks: int = 2, taps: int = 4,
                 dtype=torch.bfloat16):
        super().__init__()
        self.dtype, self.scale = dtype, math.sqrt(width)
        self.table = torch.nn.Parameter(torch.randn(vocab, width) / math.sqrt(width))
        self.blocks = torch.nn.ModuleList([Block(width, lanes, taps, dtype) for _ in range(blocks)])
        self.norm = torch.nn.Parameter(torch.ones(width))

    def logits(self, x):
        return F.linear(norm(x, self.norm), self.table.to(self.dtype)).float()

    def positions(self, ids):
        """Of one document a row.  A document's first token enters the state whole
        (its position is 0), not scaled as after a state of zeros."""
        return torch.arange(ids.shape[1], dtype=torch.int32, device=ids.device).repeat(ids.shape[0], 1)

    def forward(self, ids, segment_pos=None):
        segment_pos = self.positions(ids) if segment_pos is None else segment_pos
        x = L.embed(ids, self.table, self.scale, self.dtype)
        for block in self.blocks:
            x, _, _ = block(x, segment_pos)
        return self.logits(x)


class Server:
    """A model with a pool of `slots` requests."""

    def __init__(self, model: RecurrentLM, slots: int):
        b = model.blocks[0]
        dev = model.table.device
        self.model = model
        self.windows = [torch.zeros(slots, b.taps - 1, b.lanes, device=dev, dtype=model.dtype) for _ in model.blocks]
        self.states = [torch.zeros(slots, b.lanes, device=dev) for _ in model.blocks]

    @torch.no_grad()
    def prefill(self, slot: int, prompt):
        """Fills `slot` from a prompt [T]; returns the logits of the token after it."""
        m = self.model
        x = L.lrscan_fwd_embed(prompt[None], m.table, scale=m.scale, dtype=m.dtype)
        pos = m.positions(prompt[None])
        for n, block in enumerate(m.blocks):
            x, window, state = block(x, pos)
            self.windows[n][slot] = window[0]
            self.states[n][slot] = state[0]
        return m.logits(x[0, -1])

    @torch.no_grad()
    def step(self, ids, slots):
        """The next token of each request: ids [B], slots int32 [B] (negative: no
        request in this row); returns logits [B, vocab]."""
        m = self.model
        x = L.lrscan_fwd_embed(ids, m.table, scale=m.scale, dtype=m.dtype)
        for n, block in enumerate(m.blocks):
            x = block.step(x, self.windows[n], self.states[n], slots)
        return m.logits(x)


def corpus(vocab: int, rows: int, tokens: int, generator):
    """Packed documents that count up from a random token by a random step of one
    to three: (ids [rows, tokens], segment positions)."""
    ids = torch.empty(rows, tokens, dtype=torch.int64)
    pos = torch.empty(rows, tokens, dtype=torch.int32)
    for b in range(rows):
        t = 0
        while t < tokens:
            n = min(int(torch.randint(8, 40, (1,), generator=generator)), tokens - t)
            first, by = (int(torch.randint(*r, (1,), generator=generator)) for r in ((0, vocab), (1, 4)))
            ids[b, t:t + n] = (first + by * torch.arange(n)) % vocab
            pos[b, t:t + n] = torch.arange(n)
            t += n
    return ids, pos


def train(model, vocab, steps, rows=8, tokens=256, lr=3e-3, generator=None):
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        ids, pos = (t.cuda() for t in corpus(vocab, rows, tokens, generator))
        logits = model(ids, pos)[:, :-1]
        same = pos[:, 1:] > 0  # the next token is of the same document
        loss = F.cross_entropy(logits[same], ids[:, 1:][same])
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


def main():
    torch.manual_seed(0)
    g = torch.Generator().manual_seed(0)
    vocab = 97
    model = RecurrentLM(vocab).cuda()
    losses = train(model, vocab, 200, generator=g)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    server = Server(model, slots=8)
    prompts = [torch.arange(5, 5 + 8 * by, by, device="cuda") % vocab for by in (1, 2, 3)]
    slots = torch.tensor([6, 0, 3], dtype=torch.int32, device="cuda")
    ids = torch.stack([server.prefill(int(s), p).argmax(-1) for s, p in zip(slots, prompts)])
    said = [ids]
    for _ in range(7):
        ids = server.step(ids, slots).argmax(-1)
        said.append(ids)
    for p, s in zip(prompts, torch.stack(said, 1).tolist()):
        print(p.tolist(), "->", s)


if __name__ == "__main__":
    main()
