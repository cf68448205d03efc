"""The gradients' norm and scaling over thousands of tensors: many tables of them, whose
time grows as their number does.

Tolerances as for fewer tensors: sums are in 64 bits, the norm is rounded once to fp32
(2^-24; 2^-23 for what the sums lose), outputs once (2^-24, of a factor in 64 bits)."""
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


def split(flat, n):
    """n tensors of sizes 1, 2, 3, 4, 1, .. that lie one behind the other."""
    sizes = [k % 4 + 1 for k in range(n)]
    assert sum(sizes) <= flat.numel()
    return list(flat[:sum(sizes)].split(sizes))


@pytest.mark.parametrize("n", [96, 97, 193, 5000, 60_000])
@pytest.mark.parametrize("part", [0.5, 2.0])
def test_many_tensors(n, part):
    log(f"clip of {n} tensors")
    gen = torch.Generator(device="cuda").manual_seed(n)
    flat = torch.randn(4 * n, generator=gen, device="cuda")
    grads = split(flat, n)
    used = sum(t.numel() for t in grads)
    before = flat.clone()
    want = before[:used].double().norm()
    limit = part * want.item()
    norm, outs = sgr.clip_grad_norm(grads, limit)
    assert abs(norm.item() - want.item()) <= 2.0 ** -23 * want.item()
    scaled = before[:used].double() * min(1.0, part)
    # (the limit was rounded to its 64 bits with the norm's own sum: nothing beside 2^-24)
    assert ((flat[:used].double() - scaled).abs() <= 2.0 ** -23 * scaled.abs()).all()
    assert torch.equal(flat[used:], before[used:])
    again = split(before, n)
    assert torch.equal(sgr.grad_norm(again), norm)
    outs = split(torch.full_like(flat, 9.0), n)
    sgr.clip_grad_norm(again, limit, out=outs)
    assert torch.equal(torch.cat(outs), flat[:used])


def test_large_tensors_over_several_tables():
    """Each launch leaves as many sums as it has workgroups."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    grads = list(torch.randn(250, 60_011, generator=gen, device="cuda"))
    want = torch.stack(grads).double()
    norm, outs = sgr.clip_grad_norm(grads, 10.0)
    n = want.norm()
    assert abs(norm.item() - n.item()) <= 2.0 ** -23 * n.item()
    want *= 10.0 / n
    assert ((torch.stack(list(outs)).double() - want).abs() <= 2.0 ** -23 * want.abs()).all()


def test_time_grows_as_the_number_of_tensors():
    """16 times as many tensors: 16 times as many launches, not 256 times the work."""
    flat = torch.randn(400_000, device="cuda")
    took = []
    for n in (6_000, 96_000):
        log(f"clip of {n} tensors in a graph")
        grads = split(flat, n)
        outs = split(torch.empty_like(flat), n)
        run = lambda: sgr.clip_grad_norm(grads, 1.0, out=outs)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graph.replay()
        best = float("inf")
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        took.append(best)
        replayed = torch.cat(outs)
        run()
        assert torch.equal(replayed, torch.cat(outs))
    log(f"clip: {took[0]:.3f} and {took[1]:.3f} ms")
    # (the fold of the sums is one workgroup's: it may take a part of its own)
    assert took[1] <= 2 * 16 * took[0], took
