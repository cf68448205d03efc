"""The norm of a model's gradients and their scaling, against sums in 64 bits.

Tolerances: squares and their sum are in fp64 (n additions: n 2^-53, less than a
2^-25 for every size here), the norm is rounded once to fp32, the factor c is fp64;
outputs are rounded once, 16-bit ones from a product that was rounded to fp32 (2^-24
more)."""
import numpy as np
import pytest
import torch

import sparse_graph_recurrent_amd as sgr

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sgr.lib()


def make(seed, sizes, dtypes, scale=1.0):
    r = np.random.default_rng(seed)
    return [torch.from_numpy(scale * r.standard_normal(n)).to(DT[d]).cuda()
            for n, d in zip(sizes, dtypes)]


def norm_of(ts):
    return float(np.sqrt(sum((t.double().cpu().numpy() ** 2).sum() for t in ts)))


def check(grads, max_norm, norm, outs, before):
    n = norm_of(before)
    assert norm.shape == (1,) and norm.dtype == torch.float32
    assert abs(norm.item() - n) <= 2.0 ** -23 * n
    c = max_norm / n if n > max_norm else 1.0
    for b, o in zip(before, outs):
        want = b.double().cpu().numpy() * c
        fi = torch.finfo(o.dtype)
        tol = (fi.eps / 2 + 2.0 ** -22) * np.abs(want) + fi.smallest_normal * fi.eps / 2
        if n <= max_norm:
            assert torch.equal(b, o)
        assert (np.abs(o.double().cpu().numpy() - want) <= tol).all()


CASES = [
    ([1], ["fp32"]), ([7, 1, 0, 8], ["fp32", "bf16", "fp16", "bf16"]),
    ([2047, 2048, 2049], ["bf16"] * 3), ([5, 100_001, 64, 9], ["fp32", "fp16", "bf16", "fp32"]),
    ([300_000, 17], ["fp32", "fp32"]), ([3_000_001], ["bf16"]), ([9_000_003, 5], ["fp32", "fp16"]),
    ([k % 37 for k in range(300)], ["fp32", "bf16", "fp16"] * 100),   # several tables
    ([100_000] * 97, ["bf16"] * 97)]


@pytest.mark.parametrize("sizes,dtypes", CASES, ids=lambda c: str(len(c)))
@pytest.mark.parametrize("part", [0.5, 2.0])
@pytest.mark.parametrize("in_place", [True, False])
def test_clip(sizes, dtypes, part, in_place):
    grads = make(1, sizes, dtypes)
    before = [t.clone() for t in grads]
    limit = part * max(norm_of(before), 1e-3)
    out = None if in_place else [torch.full_like(t, 9.0) for t in grads]
    norm, outs = sgr.clip_grad_norm(grads, limit, out=out)
    check(grads, limit, norm, outs, before)
    if in_place:
        assert all(a is b for a, b in zip(grads, outs))
    else:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    assert torch.equal(sgr.grad_norm(before), norm)


def test_unaligned_and_permuted_tensors():
    base = make(2, [10_007], ["bf16"])[0]
    grads = [base[1:4002], base[5003:10_004],
             torch.randn(33, 40, device="cuda").t(), torch.randn(3, 5, 7, device="cuda").permute(2, 0, 1)]
    before = [t.clone() for t in grads]
    rest = base[4002:5003].clone(), base[:1].clone(), base[10_004:].clone()
    norm, _ = sgr.clip_grad_norm(grads, 1.0)
    check(grads, 1.0, norm, grads, before)
    assert torch.equal(rest[0], base[4002:5003]) and torch.equal(rest[1], base[:1])
    assert torch.equal(rest[2], base[10_004:])


def test_values_whose_squares_leave_fp32():
    for scale in (1e30, 1e-30):
        grads = make(3, [1000, 50], ["fp32", "bf16"], scale)
        before = [t.clone() for t in grads]
        norm, outs = sgr.clip_grad_norm(grads, 0.25 * norm_of(before))
        check(grads, 0.25 * norm_of(before), norm, outs, before)


def test_a_factor_below_the_range_of_fp32():
    """c = 1e-7 / 8e37 or so has no bits left in fp32; what it gives has."""
    grads = make(6, [64, 40], ["bf16", "fp32"], 1e37)
    before = [t.clone() for t in grads]
    norm, outs = sgr.clip_grad_norm(grads, 1e-7)
    check(grads, 1e-7, norm, outs, before)


def test_limits():
    grads = make(4, [100], ["fp32"])
    before = grads[0].clone()
    norm, _ = sgr.clip_grad_norm(grads, float("inf"))
    assert torch.equal(before, grads[0])
    sgr.clip_grad_norm(grads, norm.item() * 1.001)
    assert torch.equal(before, grads[0])
    sgr.clip_grad_norm(grads, 0.0)
    assert not grads[0].any()
    norm, _ = sgr.clip_grad_norm(grads, 0.0)
    assert norm.item() == 0.0 and not grads[0].any()
    norm, outs = sgr.clip_grad_norm([], 1.0)
    assert norm.item() == 0.0 and outs == ()


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), -float("inf")])
def test_a_norm_that_is_not_finite_scales_nothing(bad):
    grads = make(5, [5000, 30], ["fp32", "bf16"])
    grads[1][7] = bad
    before = [t.clone() for t in grads]
    norm, _ = sgr.clip_grad_norm(grads, 1.0)
    assert not torch.isfinite(norm).item()
    for a, b in zip(grads, before):
        assert torch.equal(torch.nan_to_num(a.float(), 1.5), torch.nan_to_num(b.float(), 1.5))
    big = [torch.full((4,), 3e38, device="cuda")]       # its norm is beyond fp32
    norm, _ = sgr.clip_grad_norm(big, 1.0)
    assert norm.item() == float("inf") and (big[0] == 3e38).all()


def test_same_bits_on_another_stream_and_in_a_graph():
    grads = make(6, [70_001, 300, 5], ["fp32", "bf16", "fp16"])
    want_norm, want = sgr.clip_grad_norm(grads, 3.0, out=[torch.empty_like(t) for t in grads])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(t) for t in grads]
    norm, _ = sgr.clip_grad_norm(grads, 3.0, out=outs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(norm, want_norm) and all(map(torch.equal, outs, want))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sgr.clip_grad_norm(grads, 3.0, out=outs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    work = [t.clone() for t in grads]
    with torch.cuda.graph(graph):
        held, _ = sgr.clip_grad_norm(work, 3.0)
    for k in range(4):
        for w, t in zip(work, grads):
            w.copy_(t * (0.5 * k + 0.001))
        plain = [w.clone() for w in work]
        graph.replay()
        again, scaled = sgr.clip_grad_norm(plain, 3.0)
        torch.cuda.synchronize()
        assert torch.equal(held, again) and all(map(torch.equal, work, scaled)), k


def test_a_write_into_a_saved_tensor_is_seen():
    w = torch.randn(8, device="cuda", requires_grad=True)
    t = torch.randn(8, device="cuda")
    y = (w * t).sum()
    sgr.clip_grad_norm([t], 0.1)
    with pytest.raises(RuntimeError, match="modified"):
        y.backward()


def test_binding_refusals():
    a, b = make(7, [64, 64], ["fp32", "fp32"])
    for bad in ([a.cpu()], [a.double()], [a[::2]], [a.expand(3, 64)], [None], [a, a], [a, a[3:]],
                [a.view(8, 8)[:, :4]]):
        with pytest.raises((TypeError, ValueError, sgr.CkError)):
            sgr.clip_grad_norm(bad, 1.0)
    for out in ([b[:4]], [b.bfloat16()], [b.cpu()], [], [b, b], [a[:63]]):
        with pytest.raises((TypeError, ValueError, sgr.CkError)):
            sgr.clip_grad_norm([a], 1.0, out=out)
    for limit in (-1.0, float("nan")):
        with pytest.raises(sgr.CkError):
            sgr.clip_grad_norm([a], limit)
    with pytest.raises(ValueError):
        sgr.clip_grad_norm([a], 1.0, norm=torch.empty(2, device="cuda"))
    assert torch.equal(sgr.grad_norm([a, a]), sgr.grad_norm([a, a.clone()]))  # read only: allowed
