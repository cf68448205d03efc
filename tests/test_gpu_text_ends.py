"""The text example's search with a character that ends a beam: beams do end, say nothing
else from there on, and keep the score that they ended with."""
import importlib.util
import os

import pytest
import torch

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


@pytest.mark.parametrize("mixer", ["selective", "gated"])
def test_ended_beams_keep_their_scores(example, mixer):
    """Each beam's score is the sum of the log-probabilities of its characters up to and
    with the first that ends it, which the model gives to the whole text."""
    model, text, _ = example.build(seed=5, mixer=mixer)
    prompt, n, beams = torch.stack([text[:15], text[31:46]], dim=1), 8, 4
    free, _ = example.search(model, prompt, n, beams)
    # a character that the free search says early, so that it is likely enough to end beams
    eos = free[1, 0, 0].item()
    said, scores = example.search(model, prompt, n, beams, eos=eos)
    assert (scores[:, :-1] >= scores[:, 1:]).all()
    ended = (said == eos).cumsum(0) > 0
    assert ended[:-1].any() and not ended.all(0).all(), "beams that end early, and such as go on"
    for b in range(2):
        for k in range(beams):
            full = torch.cat([prompt[:, b], said[:, b, k]]).unsqueeze(1)
            with torch.no_grad():
                logits, _ = model(full[:-1])
            logp = torch.log_softmax(logits[-n:, 0].double(), -1)
            each = logp.gather(1, said[:, b, k:k + 1]).squeeze(1)
            last = int(ended[:, b, k].float().argmax()) if ended[-1, b, k] else n - 1
            assert (said[last + 1:, b, k] == eos).all()
            # n sums of logits from other kernels, as for beams that do not end
            assert abs(scores[b, k].item() - each[:last + 1].sum().item()) <= \
                n * 2e-4 * logits.abs().max().item(), (b, k, last)
            if last < n - 1:    # (what it would have if the text behind its end counted)
                assert abs(each[last + 1:].sum().item()) > n * 2e-3 * logits.abs().max().item()
