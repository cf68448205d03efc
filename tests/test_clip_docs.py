"""The call of ``clip_grad_norm`` as the documents and the example write it, for a model
with a parameter that no loss reaches: it passes the gradients that are there."""
import ast
import os

import pytest
import torch

import sparse_graph_recurrent_amd.clip as clip

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def lines(text):
    """The statements of a document's code that end in a call of clip_grad_norm."""
    rows = [ln.strip() for ln in text.splitlines()]
    at = next(k for k, ln in enumerate(rows) if "clip_grad_norm(" in ln and "`" not in ln)
    return "\n".join(ln for ln in rows[at - 1:at + 1] if "grad" in ln)


def documented():
    with open(os.path.join(ROOT, "README.md")) as f:
        yield "README.md", lines(f.read())
    yield "clip.py", lines(clip.__doc__)
    path = os.path.join(ROOT, "examples", "text_mixer.py")
    with open(path) as f:
        source = f.read()
    call = next(n for n in ast.walk(ast.parse(source)) if isinstance(n, ast.Call)
                and ast.unparse(n.func).endswith("clip_grad_norm"))
    yield "text_mixer.py", "norm, _ = " + ast.unparse(call)


@pytest.mark.parametrize("name,code", list(documented()), ids=lambda c: c if "." in c[:12] else "")
def test_only_gradients_that_are_there(name, code):
    model = torch.nn.Sequential(torch.nn.Linear(3, 2), torch.nn.Linear(5, 4))   # one is not used
    model[0](torch.ones(1, 3)).sum().backward()
    seen = []

    class Calls:
        @staticmethod
        def clip_grad_norm(grads, max_norm):
            seen.extend(grads)
            return None, None

    exec(code, {"model": model, "ck": Calls, "sgr": Calls, "max_norm": 1.0,
                "clip_grad_norm": Calls.clip_grad_norm})
    want = [p.grad for p in model[0].parameters()]
    assert len(seen) == 2 and all(a is b for a, b in zip(seen, want))
