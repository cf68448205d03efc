"""Bias gradients of the gated scan over many steps and rows.  They are sums of the
gradients of f and i, which fp32 calls hand out as they are added up, so that each can be
held to the sum of those in 64 bits:

    |g_bias - sum g| <= 10 2^-24 sum |g|

a window's eight steps are added in fp32 (7 roundings), and a workgroup's part and the
result are rounded to fp32 (2); sums between them are in 64 bits (less than 2^-30 of
sum |g| for any number of terms here)."""
import pytest
import torch

import sparse_graph_recurrent_amd as sgr
from gpu_helpers import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sgr.lib()


CASES = [  # T, B, D: a column a CU, windows of their own, many rows of few steps
    (16384, 8, 1024), (262144, 1, 33), (8, 40000, 32), (129, 3000, 40), (1, 70000, 1)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("alike", [True, False])
def test_bias_gradients_do_not_lose_steps(case, alike):
    """`alike`: all steps' gradients nearly the same, whose sum rounds the same way each time."""
    log(f"gated bias sums {case} alike={alike}")
    T, B, D = case
    gen = torch.Generator(device="cuda").manual_seed(4)
    if alike:
        x, f, i, go = (torch.full((T, B, D), v, device="cuda") for v in (0.7, 0.3, -0.2, 1.1))
    else:
        x, f, i, go = (torch.rand(T, B, D, generator=gen, device="cuda") for _ in range(4))
    _, _, saved, _ = sgr.gated_scan_forward(x, f, i)
    g = sgr.gated_scan_backward(x, f, saved, go, i)
    for part, total in (("g_f", "g_f_bias"), ("g_i", "g_i_bias")):
        each = g[part].double()
        want, size = each.sum((0, 1)), each.abs().sum((0, 1))
        assert (size > 0).all() or T == 1
        off = (g[total].double() - want).abs()
        assert (off <= 10 * 2.0 ** -24 * size).all(), \
            f"{total}: {(off / size.clamp_min(1e-30)).max().item() * 2 ** 24:.1f} 2^-24 of the terms"


def test_lengths_and_gates_without_sums():
    """Rows of no text, windows behind the text, a tied input gate; buffers that held NaN."""
    T, B, D = 700, 5, 70
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, f, go = (torch.rand(T, B, D, generator=gen, device="cuda") for _ in range(3))
    for lens in ([700, 0, 1, 129, 640], [0] * 5):
        lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
        _, _, saved, _ = sgr.gated_scan_forward(x, f, lengths=lengths)
        grads = {"g_x": torch.empty_like(x), "g_f": torch.empty_like(x),
                 "g_f_bias": torch.full((D,), float("nan"), device="cuda")}
        ws = torch.full((4 << 20,), 255, dtype=torch.uint8, device="cuda")
        g = sgr.gated_scan_backward(x, f, saved, go, lengths=lengths, grads=grads, workspace=ws)
        each = g["g_f"].double()
        off = (g["g_f_bias"].double() - each.sum((0, 1))).abs()
        assert (off <= 10 * 2.0 ** -24 * each.abs().sum((0, 1))).all()
