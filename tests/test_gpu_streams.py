"""Recurrence and LIF calls on a given stream: what they allocate is that
stream's own memory, never a block that the caller has freed on the current
stream, where queued work may still read it."""
import numpy as np
import pytest
import torch

import sparse_graph_recurrent_amd as sgr
import synthetic
from gpu_helpers import make_graph, to_dev

pytestmark = pytest.mark.gpu


def _flat(res):
    return [t for r in res for t in (r.values() if isinstance(r, dict) else
                                     r if isinstance(r, tuple) else (r,))]


def _check(work):
    """work(stream): a list of calls' results.  Equal on another stream, in other memory."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    old = [work(None), work(None)]
    torch.cuda.synchronize()
    freed = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
             for res in old for t in _flat(res)]
    del old
    side = torch.cuda.Stream()
    before = torch.cuda.current_stream()
    res = work(side)
    assert torch.cuda.current_stream() == before
    before.wait_stream(side)
    for t in _flat(res):
        lo, hi = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
        assert not any(lo < b and a < hi for a, b in freed), (lo, hi)
    want = work(None)
    torch.cuda.synchronize()
    for a, b in zip(_flat(res), _flat(want)):
        if a.dtype == torch.float32 or a.dtype == torch.int32:
            assert torch.equal(a, b)


@pytest.mark.parametrize("path", ["resident", "per_microstep"])
def test_recurrence_on_another_stream(path):
    w = synthetic.make("tiny")
    g = make_graph(w, path)
    ev, lk, bs, dr, st, go = (to_dev(x) for x in (w.edge_values, w.leak, w.bias, w.drives,
                                                  w.state0, w.grad_out))

    def work(stream):
        f = sgr.recurrence_forward(g, ev, lk, bs, dr, st, w.microsteps, stream=stream)
        return f, sgr.recurrence_backward(g, ev, lk, st, w.microsteps, f[1], go, stream=stream)

    _check(work)


def test_export_on_another_stream():
    g = make_graph(synthetic.make("tiny"))
    _check(lambda stream: [g.export(stream=stream)])


def test_lif_on_another_stream():
    w = synthetic.make("tiny")
    g = make_graph(w)
    r = np.random.default_rng(5)
    imp = to_dev(r.integers(-50, 200, w.num_edges).astype(np.int16))
    dly = to_dev(r.integers(1, 4, w.num_edges).astype(np.int32))
    v0 = to_dev(r.integers(0, 100, w.num_nodes).astype(np.int32))
    args = dict(T=6, threshold=90, reset=0, refractory_steps=1, decay_shifts=(3,))

    def work(stream):
        ws = sgr.lif_prepare(g, imp, dly, stream=stream)
        return (sgr.lif_forward(g, imp, dly, v0, stream=stream, **args), ws,
                sgr.lif_run(g, ws, v0, stream=stream, **args))

    _check(work)
