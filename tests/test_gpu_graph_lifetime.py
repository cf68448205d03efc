"""A graph that is let go of while a HIP graph is being captured, by the garbage collector
or by hand: the capture goes on, and the graph's memory is freed behind it."""
import gc

import numpy as np
import pytest
import torch

import sparse_graph_recurrent_amd as sgr
import synthetic
from gpu_helpers import log, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sgr.lib()


def make():
    w = synthetic.make("tiny")
    return w, sgr.SparseGraph(to_dev(w.src), to_dev(w.dst), w.num_nodes, to_dev(w.input_nodes))


@pytest.mark.parametrize("how", ["collected", "deleted", "destroyed"])
def test_a_graph_goes_during_a_capture(how):
    log(f"graph {how} during a capture")
    w, graph = make()
    ins = [to_dev(x) for x in (w.edge_values, w.leak, w.bias, w.drives, w.state0)]
    sb, wb = sgr.recurrence_sizes(graph, w.T, w.B, w.microsteps)
    out = torch.empty((w.T, w.B, w.num_nodes), device="cuda")
    saved, ws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (sb, wb))
    step = lambda: sgr.recurrence_forward(graph, *ins, w.microsteps, out=out, saved=saved,
                                          workspace=ws)
    step()
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    _, other = make()
    kept = other if how == "destroyed" else None
    if how == "collected":
        other.itself = other            # only the garbage collector frees it
    captured = torch.cuda.CUDAGraph()
    gc.disable()
    try:
        with torch.cuda.graph(captured):
            step()
            if how == "destroyed":
                kept.destroy()
            del other
            if how == "collected":
                gc.collect()
            step()
    finally:
        gc.enable()
    assert len(sgr._waiting) == 1
    if kept is not None:
        with pytest.raises(sgr.CkError):
            kept.sizes()
    for _ in range(3):
        out.zero_()
        captured.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(out.cpu().numpy(), want.cpu().numpy())
    _, new = make()                     # frees what waits
    assert not sgr._waiting
    new.destroy()
    new.destroy()
    assert not sgr._waiting


def test_a_graph_goes_at_once_otherwise():
    _, graph = make()
    graph.sizes()
    del graph
    assert not sgr._waiting
