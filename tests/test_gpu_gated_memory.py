"""The gated scan where inputs and outputs share one tensor without lying over one
another, and single tokens in place: the bits of separate tensors."""
import pytest
import torch

import sparse_graph_recurrent_amd as sgr
from gpu_helpers import log

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sgr.lib()


@pytest.mark.parametrize("T,B,D,dtype", [(40, 2, 65, "bf16"), (300, 3, 129, "fp16"),
                                         (17, 1, 1, "fp32"), (9, 4, 3, "bf16")])
@pytest.mark.parametrize("batch", [False, True])
def test_slices_of_one_tensor(T, B, D, dtype, batch):
    log(f"slices {T} {B} {D} {dtype} batch={batch}")
    gen = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.randn(B if batch else T, T if batch else B, 10 * D, generator=gen,
                       device="cuda").to(DT[dtype])
    if batch:
        wide = wide.transpose(0, 1)
    x, f, i, z, go, out, *grads = wide.split(D, dim=-1)
    grads = dict(zip(("g_x", "g_f", "g_i", "g_z"), grads))
    state0 = torch.randn(2 * B, D, generator=gen, device="cuda")  # the new one behind the old
    own = [t.contiguous() for t in (x, f, i, z, go)]
    want, state, saved, _ = sgr.gated_scan_forward(*own[:4], state0=state0[:B].clone())
    sgr.gated_scan_forward(x, f, i, z, state0=state0[:B], out=out, state=state0[B:])
    assert torch.equal(out, want) and torch.equal(state0[B:], state)
    want = sgr.gated_scan_backward(own[0], own[1], saved, own[4], own[2], own[3])
    sgr.gated_scan_backward(x, f, saved, go, i, z, grads=grads)
    for k, t in grads.items():
        assert torch.equal(t, want[k]), k
    for a, b in zip((x, f, i, z, go), own):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,D,dtype", [(1, 1, "fp32"), (3, 65, "bf16"), (70, 64, "fp16")])
@pytest.mark.parametrize("over", [0, 1, 2, 3])
def test_a_token_in_place(B, D, dtype, over):
    gen = torch.Generator(device="cuda").manual_seed(2)
    new = lambda: torch.randn(B, 2 * D, generator=gen, device="cuda").to(DT[dtype])[:, 1:1 + D]
    parts = [new() for _ in range(4)]
    state = torch.randn(B, D, generator=gen, device="cuda")
    want, after = sgr.gated_scan_step(state.clone(), *parts)
    out, same = sgr.gated_scan_step(state, *parts, out=parts[over])
    assert out is parts[over] and same is state
    assert torch.equal(out, want) and torch.equal(state, after)


def test_calls_over_their_inputs_are_refused():
    x, f = (torch.randn(40, 2, 65, device="cuda").bfloat16() for _ in range(2))
    state = torch.randn(3, 65, device="cuda")
    before = x.clone()
    for kw in (dict(out=x), dict(out=f), dict(state0=state[:2], state=state[1:])):
        with pytest.raises(sgr.CkError, match="must not lie over"):
            sgr.gated_scan_forward(x, f, **kw)
    _, _, saved, _ = sgr.gated_scan_forward(x, f)
    g = sgr.gated_scan_backward(x, f, saved, x)
    for k, t in (("g_x", f), ("g_f", g["g_x"])):
        with pytest.raises(sgr.CkError, match="must not lie over"):
            sgr.gated_scan_backward(x, f, saved, before, grads={**g, k: t})
    torch.cuda.synchronize()
    assert torch.equal(x, before)
