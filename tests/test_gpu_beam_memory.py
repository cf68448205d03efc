"""Selection and reordering where inputs and outputs are slices of one tensor: the values
of separate ones."""
import pytest
import torch

import sparse_graph_recurrent_amd as sgr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sgr.lib()


def test_reorder_slices_of_one_tensor():
    """States and outputs take turns in the rows of one tensor."""
    wide = torch.randint(0, 100, (8, 60), device="cuda", dtype=torch.int32)
    states = [wide[:, 0:7], wide[:, 14:30], wide[:, 46:50]]
    outs = [wide[:, 7:14], wide[:, 30:46], states[2]]
    parents = torch.tensor([[1, 1, 0, 3], [2, 0, 2, 1]], device="cuda")
    at = (parents + torch.tensor([[0], [4]], device="cuda")).view(-1)
    want = wide.clone()
    for t, a, b in ((states[0], 7, 14), (states[1], 30, 46), (states[2], 46, 50)):
        want[:, a:b] = t[at]
    sgr.beam_reorder(states, parents, out=outs)
    assert torch.equal(wide, want)


def test_reorder_over_other_states_is_refused():
    buf = torch.arange(200, device="cuda", dtype=torch.float32)
    before = buf.clone()
    parents = torch.zeros(1, 4, dtype=torch.int64, device="cuda")
    a, b = buf[:40].view(4, 10), buf[30:70].view(4, 10)
    for states, outs in (([a, b], None), ([a], [b]), ([b], [a]), ([a], [buf[5:45].view(4, 10)])):
        with pytest.raises(sgr.CkError):
            sgr.beam_reorder(states, parents, out=outs)
    parents = torch.zeros(2, 2, dtype=torch.int64, device="cuda")
    with pytest.raises(sgr.CkError, match="parents"):
        sgr.beam_reorder([parents.view(4, 1)], parents)
    torch.cuda.synchronize()
    assert torch.equal(buf, before)


def test_select_writes_into_the_padding_of_its_logits():
    """Rows of a padded projection, whose last elements hold the outputs."""
    x = torch.randn(1, 4, 32, device="cuda")
    scores = -torch.rand(1, 4, device="cuda")
    logits = x[:, :, :20]
    want = sgr.beam_select(logits.clone(), scores)
    out = (x[:, 0, 20:24], x[0, 1, 20:28].view(torch.int64).view(1, 4),
           x[0, 2, 20:28].view(torch.int64).view(1, 4), None)
    got = sgr.beam_select(logits, scores, out=out)
    assert all(map(torch.equal, want[:3], got[:3]))
    for bad in ((x[:, 0, 16:20], *out[1:]), (out[0], out[1], out[1], None)):
        with pytest.raises(sgr.CkError, match="must not lie over"):
            sgr.beam_select(logits, scores, out=bad)
