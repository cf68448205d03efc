"""The text example end to end: the sequence operators and the recurrence train
together, and the single-token path continues a window as the window itself
would."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from gpu_helpers import log

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


def test_training_reduces_the_loss(example):
    model, text, chars = example.build()
    losses = example.train(model, text, 60)
    log(f"text example: loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    assert np.all(np.isfinite(losses))
    # the text's own character entropy is about 2.8 nats; windows are learned well below it
    assert losses[-1] < 0.7 * losses[0]
    for name, p in model.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.any(), name


def test_tokens_continue_the_window(example):
    model, text, _ = example.build(seed=3)
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
