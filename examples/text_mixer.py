"""A small character model around the graph recurrence: the sequence operators
as a text model uses them, in training and in answering.

    embedding -> short convolution -> selective scan (gated) -> dropout + residual
              -> drives of the graph's input nodes -> leaky-tanh recurrence
              -> readout of the node states -> next character

(or, with mixer="gated", the gated scan in the selective one's place).
Training runs whole windows: the recurrence carries its state through the
window, the mixer's own states start at zero; the gradients' norm can be
limited.  Answering reads the prompt as a window, keeps the last state of each
of the three (convolution, scan, recurrence) and then takes one character at a
time with the single-token calls, the likeliest or by a search with several
beams.  Run it on a GPU:

    python examples/text_mixer.py [--steps 120] [--mixer gated] [--max-norm 1] [--beams 4]
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
                 microsteps: int = 2, p: float = 0.1, mixer: str = "selective"):
        super().__init__()
        if mixer not in ("selective", "gated"):
            raise ValueError(f"mixer must be 'selective' or 'gated', got {mixer!r}")
        D, N, E = graph.num_inputs, graph.num_nodes, graph.num_edges
        self.graph, self.states, self.microsteps, self.p = graph, states, microsteps, p
        self.mixer = mixer
        new = lambda *shape, scale=1.0: torch.nn.Parameter(
            scale * torch.randn(*shape, device="cuda"))
        self.embedding = new(vocab, D)
        self.project = new(D, 2 * D, scale=D ** -0.5)          # input and gate
        self.conv_weight, self.conv_bias = new(D, taps, scale=taps ** -0.5), new(D, scale=0.1)
        if mixer == "gated":
            self.project_gates = new(D, 2 * D, scale=D ** -0.5)     # forget and input gate
            self.f_bias = torch.nn.Parameter(torch.linspace(1.0, 5.0, D, device="cuda"))
            self.i_bias = torch.nn.Parameter(torch.zeros(D, device="cuda"))
        else:
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

    def _mix(self, y, z, lengths):
        """The scan of the convolution's output y with output gate z; (out, its state)."""
        if self.mixer == "gated":
            f, i = (y @ self.project_gates).chunk(2, dim=-1)
            return sgr.gated_scan(y, f, i, z, self.f_bias, self.i_bias, lengths=lengths)
        delta, b, c = self._inputs(y)
        return sgr.selective_scan(y, delta, -torch.exp(self.log_a), b, c, self.skip, z=z,
                                  delta_bias=self.delta_bias, lengths=lengths,
                                  delta_softplus=True)

    def _mix_step(self, scan_state, y, z):
        """One character of ``_mix``; the state is updated in place."""
        if self.mixer == "gated":
            f, i = (y @ self.project_gates).chunk(2, dim=-1)
            return sgr.gated_scan_step(scan_state, y, f, i, z, self.f_bias, self.i_bias)[0]
        delta, b, c = self._inputs(y)
        return sgr.selective_scan_step(scan_state, y, delta, -torch.exp(self.log_a), b, c,
                                       self.skip, z=z, delta_bias=self.delta_bias,
                                       delta_softplus=True)[0]

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
        out, scan_state = self._mix(y, z, lengths)
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
        out = self._mix_step(scan_state, y, z)
        states, node_state = self._recur((x + out).unsqueeze(0), node_state)
        return states[0] @ self.readout, (conv_state, scan_state, node_state)


def build(seed: int = 0, mixer: str = "selective"):
    """(model on the tiny workload's graph, the text as indices, its characters)."""
    w = synthetic.make("tiny")
    dev = lambda a: torch.from_numpy(a).cuda()
    graph = sgr.SparseGraph(dev(w.src), dev(w.dst), w.num_nodes, dev(w.input_nodes))
    chars = sorted(set(TEXT))
    torch.manual_seed(seed)
    index = torch.tensor([chars.index(ch) for ch in TEXT], device="cuda")
    return TextMixer(graph, len(chars), mixer=mixer), index, chars


def train(model: TextMixer, text: torch.Tensor, steps: int, T: int = 64, B: int = 16,
          max_norm: float | None = None):
    """Adam on random windows, the gradients' norm limited to max_norm if there is one;
    the losses."""
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
        if max_norm is not None:
            sgr.clip_grad_norm([p.grad for p in model.parameters() if p.grad is not None],
                               max_norm)
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


@torch.no_grad()
def search(model: TextMixer, prompt: torch.Tensor, n: int, beams: int = 4, eos: int | None = None):
    """The likeliest n characters after the prompt [T, B] that a search with `beams`
    beams finds; (characters [n, B, beams] best first, their log-probabilities [B,
    beams]).  eos: a character that ends a beam."""
    T, B = prompt.shape
    logits, carried = model(prompt)
    # every text's beams begin alike: the first alone has a score
    carried = [carried[0].repeat_interleave(beams, 1)] + \
        [t.repeat_interleave(beams, 0) for t in carried[1:]]
    logits = logits[-1].unsqueeze(1).expand(B, beams, -1)
    scores = torch.full((B, beams), -float("inf"), device="cuda")
    scores[:, 0] = 0
    said, finished = torch.empty(0, B, beams, dtype=torch.int64, device="cuda"), None
    for k in range(n):
        scores, parents, tokens, finished = sgr.beam_select(logits, scores, finished, eos)
        conv_state, scan_state, node_state = carried
        history = said.permute(1, 2, 0).reshape(B * beams, k)
        sgr.beam_reorder([conv_state.transpose(0, 1), scan_state, node_state, history], parents)
        said = torch.cat([history.view(B, beams, k).permute(2, 0, 1), tokens.unsqueeze(0)])
        if k + 1 < n:
            logits, carried = model.step(tokens.view(-1), carried)
            logits = logits.unflatten(0, (B, beams))
    return said, scores


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=120)
    ap.add_argument("--mixer", choices=("selective", "gated"), default="selective")
    ap.add_argument("--max-norm", type=float, default=None)
    ap.add_argument("--beams", type=int, default=1)
    a = ap.parse_args()
    model, text, chars = build(mixer=a.mixer)
    losses = train(model, text, a.steps, max_norm=a.max_norm)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} after {a.steps} steps")
    prompt = text[:40].unsqueeze(1)
    said = answer(model, prompt, 60)[:, 0].tolist()
    print("prompt: " + "".join(chars[i] for i in prompt[:, 0].tolist()))
    print("answer: " + "".join(chars[i] for i in said))
    if a.beams > 1:
        found, scores = search(model, prompt, 60, a.beams)
        print(f"found ({scores[0, 0].item():.2f}): " +
              "".join(chars[i] for i in found[:, 0, 0].tolist()))


if __name__ == "__main__":
    main()
