"""States of the gated scan that are not finite: what lies behind a row's text changes
none of them, and they reach no other channel, row or earlier step."""
import pytest
import torch

import sparse_graph_recurrent_amd as sgr
from gpu_helpers import log

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sgr.lib()


def make(T, B, D, dtype, own, z):
    gen = torch.Generator(device="cuda").manual_seed(3)
    new = lambda on=True: torch.randn(T, B, D, generator=gen, device="cuda").to(DT[dtype]) \
        if on else None
    return new(), new(), new(own), new(z), torch.randn(B, D, generator=gen, device="cuda")


CASES = [  # T, B, D, dtype, own, z, lengths: few columns (windows of their own) and many
    (40, 3, 5, "fp32", True, True, [40, 33, 1]), (300, 4, 65, "bf16", False, True, [300, 297, 128, 3]),
    (1030, 2, 33, "fp16", True, False, [1029, 515]), (130, 40, 420, "bf16", True, True, None)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])))
def test_an_infinite_last_step_stays_behind_the_text(case):
    """The last step of each row's text makes some states infinite: they come out so, with
    steps behind the text as without any."""
    log(f"gated infinite {case}")
    T, B, D, dtype, own, z, lengths = case
    x, f, i, zt, state0 = make(T, B, D, dtype, own, z)
    lengths = lengths or [(37 * b) % T + 1 for b in range(B)]
    for b, n in enumerate(lengths):
        x[n - 1, b, ::3], x[n - 1, b, 1::3] = INF, -INF
    cut = lambda t, b, n: None if t is None else t[:n, b:b + 1]
    out, state, _, _ = sgr.gated_scan_forward(
        x, f, i, zt, state0=state0, lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    assert (state[:, ::3] == INF).all() and (state[:, 1::3] == -INF).all()
    assert torch.isfinite(state[:, 2::3]).all()
    for b, n in list(enumerate(lengths))[:5]:
        assert not out[n:, b].any()
        if not z:
            assert (out[n - 1, b, ::3] == INF).all()
        alone = sgr.gated_scan_forward(*(cut(t, b, n) for t in (x, f, i, zt)),
                                       state0=state0[b:b + 1].clone())
        assert torch.equal(alone[1], state[b:b + 1])
        assert torch.equal(alone[0][:, 0], out[:n, b])


def test_a_row_without_text_passes_an_infinite_state():
    for T, B, D in ((40, 2, 33), (300, 2, 33), (40, 70, 300)):
        x, f, i, z, state0 = make(T, B, D, "bf16", True, True)
        state0[::2, 5], state0[::2, 6] = INF, -INF
        lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
        out, state, _, _ = sgr.gated_scan_forward(x, f, i, z, state0=state0, lengths=lengths)
        assert torch.equal(state, state0) and not out.any()


@pytest.mark.parametrize("T,B,D", [(300, 2, 65), (40, 3, 33), (300, 40, 420)])
@pytest.mark.parametrize("bad", [INF, -INF, float("nan")])
def test_other_channels_and_steps_are_not_reached(T, B, D, bad):
    """One channel of a row is not finite from a step on; all else has the bits of a call
    without it."""
    x, f, i, z, state0 = make(T, B, D, "bf16", True, True)
    good = sgr.gated_scan_forward(x, f, i, z, state0=state0)
    at, b, d = 21, B - 1, D // 2
    x[at, b, d] = bad
    got = sgr.gated_scan_forward(x, f, i, z, state0=state0)
    assert not torch.isfinite(got[0][at:, b, d].float()).any()
    assert not torch.isfinite(got[1][b, d])
    for g, w in zip(got[:2], good[:2]):
        g, w = g.clone(), w.clone()
        for t in (g, w):
            (t[at:] if t.dim() == 3 else t)[..., b, d] = 0
        assert torch.equal(g, w)
