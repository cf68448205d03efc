"""A small character model around the graph recurrence: the sequence operators
as a text model uses them, in training and in answering.

    embedding -> short convolution -> selective scan (gated) -> dropout + residual
              -> drives of the graph's input nodes -> leaky-tanh recurrence
              -> readout of the node states -> next character

Training runs whole windows: the recurrence carries its state through the
window, the mixer's own states start at zero.  Answering reads the prompt as a
window, keeps the last state of each of the three (convolution, scan,
recurrence) and then takes one character at a time with the single-token
calls.  Run it on a GPU:

    python examples/text_mixer.py [--steps 120]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_graph_recurrent_amd as sgr  # noqa: E402
import synthetic  # noqa: E402

TEXT = ("a node sums what its edges bring, adds its drive and its bias, "
        "and moves a little towards the tanh of it. ") * 40


class TextMixer(torch.nn.Module):
    """Characters to logits through the mixer and the recurrence on `graph`."""

    def __init__(self, graph: sgr.SparseGraph, vocab: int, states: int = 8, taps: int = 4,
                 microsteps: int = 2, p: float = 0.1):
        super().__init__()
        D, N, E = graph.num_inputs, graph.num_nodes, graph.num_edges
        self.graph, self.states, self.microsteps, self.p = graph, states, microsteps, p
        new = lambda *shape, scale=1.0: torch.nn.Parameter(
            scale * torch.randn(*shape, device="cuda"))
        self.embedding = new(vocab, D)
        self.project = new(D, 2 * D, scale=D ** -0.5)          # input and gate
        self.conv_weight, self.conv_bias = new(D, taps, scale=taps ** -0.5), new(D, scale=0.1)
        self.project_bc = new(D, D + 2 * states, scale=D ** -0.5)   # time steps, B and C
        self.delta_bias = torch.nn.Parameter(torch.full((D,), -2.0, device="cuda"))
        self.log_a = torch.nn.Parameter(
            torch.log(torch.arange(1, states + 1, device="cuda").float()).repeat(D, 1))
        self.skip = torch.nn.Parameter(torch.ones(D, device="cuda"))
        self.edge_values = new(E, scale=(N / E) ** 0.5)
        self.raw_leak, self.bias = new(N, scale=0.5), new(N, scale=0.1)
        self.readout = new(N, vocab, scale=N ** -0.5)

    def _inputs(self, y):
        """dt, B and C of the convolution's output y [.., D]."""
        D, S = y.shape[-1], self.states
        dbc = y @ self.project_bc
        return (dbc[..., :D], dbc[..., D:D + S].unflatten(-1, (1, S)),
                dbc[..., D + S:].unflatten(-1, (1, S)))

    def _recur(self, x, node_state):
        """The recurrence on drives x [T, B, n_in]; (states [T, B, N], the last one)."""
        out = sgr.sparse_recurrence(self.edge_values, torch.sigmoid(self.raw_leak), self.bias,
                                    x.transpose(1, 2).contiguous(), node_state, self.graph,
                                    microsteps=self.microsteps)
        return out, out[-1].contiguous()

    def forward(self, tokens, seed=None, lengths=None):
        """tokens [T, B] -> (logits [T, B, vocab], carried states).  seed: dropout
        with this seed (training); lengths: int32 [B], texts of unequal length
        (their node states run on past their ends; the mixer's do not)."""
        T, B = tokens.shape
        x = self.embedding[tokens]
        u, z = (x @ self.project).chunk(2, dim=-1)            # slices, taken as they are
        y, conv_state = sgr.short_conv(u, self.conv_weight, self.conv_bias, lengths=lengths,
                                       activation="silu")
        delta, b, c = self._inputs(y)
        out, scan_state = sgr.selective_scan(y, delta, -torch.exp(self.log_a), b, c, self.skip,
                                             z=z, delta_bias=self.delta_bias, lengths=lengths,
                                             delta_softplus=True)
        if seed is None:
            x = x + out
        else:
            x = sgr.dropout(out, self.p, seed, residual=x, held=True)
        states, node_state = self._recur(x, torch.zeros(B, self.graph.num_nodes, device="cuda"))
        return states @ self.readout, (conv_state, scan_state, node_state)

    @torch.no_grad()
    def step(self, token, carried):
        """One character a row: token [B] -> (logits [B, vocab], carried states);
        the convolution's and the scan's states are updated in place."""
        conv_state, scan_state, node_state = carried
        x = self.embedding[token]
        u, z = (x @ self.project).chunk(2, dim=-1)
        y, _ = sgr.short_conv_step(conv_state, u, self.conv_weight, self.conv_bias, "silu")
        delta, b, c = self._inputs(y)
        out, _ = sgr.selective_scan_step(scan_state, y, delta, -torch.exp(self.log_a), b, c,
                                         self.skip, z=z, delta_bias=self.delta_bias,
                                         delta_softplus=True)
        states, node_state = self._recur((x + out).unsqueeze(0), node_state)
        return states[0] @ self.readout, (conv_state, scan_state, node_state)


def build(seed: int = 0):
    """(model on the tiny workload's graph, the text as indices, its characters)."""
    w = synthetic.make("tiny")
    dev = lambda a: torch.from_numpy(a).cuda()
    graph = sgr.SparseGraph(dev(w.src), dev(w.dst), w.num_nodes, dev(w.input_nodes))
    chars = sorted(set(TEXT))
    torch.manual_seed(seed)
    index = torch.tensor([chars.index(ch) for ch in TEXT], device="cuda")
    return TextMixer(graph, len(chars)), index, chars


def train(model: TextMixer, text: torch.Tensor, steps: int, T: int = 64, B: int = 16):
    """Adam on random windows; the losses."""
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    gen = torch.Generator().manual_seed(1)
    losses = []
    for i in range(steps):
        at = torch.randint(0, len(text) - T - 1, (B,), generator=gen)
        window = torch.stack([text[s:s + T + 1] for s in at.tolist()], dim=1)
        logits, _ = model(window[:-1], seed=i)
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), window[1:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


@torch.no_grad()
def answer(model: TextMixer, prompt: torch.Tensor, n: int):
    """n characters after the prompt [T, B], the likeliest each time."""
    logits, carried = model(prompt)
    token, out = logits[-1].argmax(-1), []
    for _ in range(n):
        out.append(token)
        logits, carried = model.step(token, carried)
        token = logits.argmax(-1)
    return torch.stack(out)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=120)
    a = ap.parse_args()
    model, text, chars = build()
    losses = train(model, text, a.steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} after {a.steps} steps")
    prompt = text[:40].unsqueeze(1)
    said = answer(model, prompt, 60)[:, 0].tolist()
    print("prompt: " + "".join(chars[i] for i in prompt[:, 0].tolist()))
    print("answer: " + "".join(chars[i] for i in said))


if __name__ == "__main__":
    main()
