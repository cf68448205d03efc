"""The text example with the gated scan, limited gradients and a search with beams:
the operators together, as a program runs them."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import sparse_graph_recurrent_amd as sgr

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "text_mixer.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("text_mixer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_training_with_limited_gradients(example):
    """Every parameter gets a gradient, and the limit holds at every step."""
    model, text, _ = example.build(mixer="gated")
    before = {k: p.detach().clone() for k, p in model.named_parameters()}
    losses = example.train(model, text, 5, max_norm=0.5)
    assert np.all(np.isfinite(losses))
    for name, p in model.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.any(), name
        assert not torch.equal(p, before[name]), name
    # 2^-23: the norm's rounding and that of each gradient
    assert sgr.grad_norm([p.grad for p in model.parameters()]).item() <= 0.5 * (1 + 2.0 ** -22)


def test_gradients_of_the_model_against_differences(example):
    """The loss's slope along a direction in all parameters."""
    model, text, _ = example.build(seed=2, mixer="gated")
    window = torch.stack([text[s:s + 25] for s in (0, 40, 90)], dim=1)
    names = [k for k, _ in model.named_parameters()]
    params = [p for _, p in model.named_parameters()]

    def loss():
        logits, _ = model(window[:-1])
        return torch.nn.functional.cross_entropy(logits.double().flatten(0, 1),
                                                 window[1:].flatten())

    grads = torch.autograd.grad(loss(), params)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for name, p, g in zip(names, params, grads):
        step = torch.randn(p.shape, generator=gen, device="cuda")
        step *= 1e-2 * (p.detach().norm() + 1e-2) / step.norm()
        with torch.no_grad():
            old = p.clone()
            p.add_(step)
            hi = loss().item()
            p.copy_(old - step)
            lo = loss().item()
            p.copy_(old)
        want = (g.double() * step.double()).sum().item()
        # central differences: a third of the step squared of the function's bend, and the
        # rounding of the loss's fp32 parts
        assert abs((hi - lo) / 2 - want) <= 0.05 * abs(want) + 2e-6, name


def test_tokens_continue_the_window(example):
    model, text, _ = example.build(seed=3, mixer="gated")
    T, B, cut = 30, 3, 17
    window = torch.stack([text[s:s + T] for s in (0, 50, 101)], dim=1)
    with torch.no_grad():
        whole, _ = model(window)
        head, carried = model(window[:cut])
        tail = []
        for t in range(cut, T):
            logits, carried = model.step(window[t], carried)
            tail.append(logits)
    got = torch.cat([head, torch.stack(tail)])
    # the same sums in other kernels: fp32 rounding, grown by T steps of a contracting network
    assert (got - whole).abs().max().item() <= 1e-4 * whole.abs().max().item()


@pytest.mark.parametrize("mixer", ["selective", "gated"])
def test_search_finds_what_its_scores_say(example, mixer):
    """A beam's score is the sum of the log-probabilities that the model, given the whole
    text, has for its characters; one beam is the greedy answer; beams differ."""
    model, text, _ = example.build(seed=4, mixer=mixer)
    prompt, n = torch.stack([text[:20], text[33:53]], dim=1), 6
    greedy = example.answer(model, prompt, n)
    said, scores = example.search(model, prompt, n, beams=1)
    assert torch.equal(said[:, :, 0], greedy)
    said, scores = example.search(model, prompt, n, beams=4)
    assert said.shape == (n, 2, 4) and (scores[:, :-1] >= scores[:, 1:]).all()
    for b in range(2):
        assert len({tuple(said[:, b, k].tolist()) for k in range(4)}) == 4
        for k in range(4):
            full = torch.cat([prompt[:, b], said[:, b, k]]).unsqueeze(1)
            with torch.no_grad():
                logits, _ = model(full[:-1])
            logp = torch.log_softmax(logits[-n:, 0].double(), -1)
            want = logp.gather(1, said[:, b, k:k + 1]).sum().item()
            # n sums of logits that are off as above
            assert abs(scores[b, k].item() - want) <= n * 2e-4 * logits.abs().max().item()


def test_search_with_an_end(example):
    """A beam that has ended says nothing else, at the score that it ended with."""
    model, text, chars = example.build(seed=5)
    eos = chars.index(" ")
    said, scores = example.search(model, text[:15].unsqueeze(1), 8, beams=3, eos=eos)
    ended = (said == eos).cumsum(0)[:-1] > 0
    assert (said[1:][ended] == eos).all()
