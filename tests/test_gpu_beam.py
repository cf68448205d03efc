"""Beam search's selection and reordering against plain definitions in 64 bits.
Places (parents, tokens) have to be equal; scores may be off by the rounding of the
result (2^-24 of it) and by what the sum of exponentials loses in 32 bits: an
exponent of up to 60 is rounded twice (60 log2(e) 2^-23 of a term that is e^-60 of
the sum; 4 2^-24 of one at its top), the sum of up to 64 adds a lane and six more:
together below 80 2^-24 of the sum, which is that much of a nat."""
import numpy as np
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


def select(x, scores, finished=None, eos=None):
    """The definition: (scores, parents, tokens, finished) in fp64.  Of equal scores the
    lower beam is first, and in one beam the larger logit, then the lower token."""
    B, K, V = x.shape
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    top = x.max(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = np.log(np.exp(x - top).sum(-1, keepdims=True))
        s = scores.astype(np.float64)[..., None] + ((x - top) - lse)
    s = np.where(x == -np.inf, -np.inf, s)
    if finished is not None:
        end = np.full(s.shape, -np.inf)
        end[:, :, eos] = scores
        s = np.where(finished[..., None], end, s)
    s = np.where(~(scores > -np.inf)[..., None], -np.inf, s)
    x = np.where(s == -np.inf, -np.inf, x)
    if finished is not None:
        x = np.where(finished[..., None] & (s > -np.inf), 0.0, x)
    s, x = s.reshape(B, K * V), x.reshape(B, K * V)
    beam = np.repeat(np.arange(K), V)
    order = np.stack([np.lexsort((-x[b], beam, -s[b])) for b in range(B)])[:, :K]
    got = np.take_along_axis(s, order, 1)
    parents, tokens = order // V, order % V
    done = None if eos is None else tokens == eos
    if finished is not None:
        done = done | np.take_along_axis(finished, parents, 1)
    return got, parents, tokens, done


def check(got, want):
    torch.cuda.synchronize()
    s, parents, tokens, done = got
    assert parents.dtype == tokens.dtype == torch.int64
    np.testing.assert_array_equal(parents.cpu().numpy(), want[1])
    np.testing.assert_array_equal(tokens.cpu().numpy(), want[2])
    g, w = s.double().cpu().numpy(), want[0]
    with np.errstate(invalid="ignore"):
        ok = (g == w) | (np.abs(g - w) <= 2.0 ** -24 * np.abs(w) + 80 * 2.0 ** -24)
    assert ok.all(), (g[~ok], w[~ok])
    if want[3] is None:
        assert done is None
    else:
        np.testing.assert_array_equal(done.cpu().numpy(), want[3])


def make(seed, B, K, V, dtype, layout="time", scale=3.0):
    r = np.random.default_rng(seed)
    t = torch.from_numpy(scale * r.standard_normal((B, K, V))).to(DT[dtype])
    if layout == "slice":
        d = torch.full((B, K, V + 5), 99.0, dtype=t.dtype, device="cuda")[:, :, 3:3 + V]
    elif layout == "beams":     # beams outermost
        d = torch.empty((K, B, V), dtype=t.dtype, device="cuda").transpose(0, 1)
    else:
        d = torch.empty(t.shape, dtype=t.dtype, device="cuda")
    d.copy_(t)
    scores = torch.from_numpy(-20 * r.random((B, K))).float()
    return d, t.double().numpy(), scores.cuda(), scores.numpy()


CASES = [  # B, K, V, dtype, layout
    (1, 1, 1, "fp32", "time"), (1, 1, 9, "bf16", "slice"), (2, 4, 3, "fp16", "time"),
    (3, 5, 28, "fp32", "beams"), (1, 8, 511, "bf16", "slice"), (2, 3, 512, "fp16", "time"),
    (2, 2, 513, "fp32", "slice"), (2, 8, 4095, "bf16", "beams"), (2, 4, 4096, "fp32", "time"),
    (3, 16, 4097, "fp16", "slice"), (2, 32, 1000, "bf16", "time"), (1, 32, 20_001, "fp32", "beams"),
    (5, 17, 9000, "fp32", "slice"), (2, 7, 100_003, "bf16", "slice"), (40, 4, 300, "bf16", "time"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("ends", [False, True])
def test_select(case, ends):
    log(f"beam_select {case} ends={ends}")
    x, xv, scores, sv = make(1, *case)
    B, K, V = x.shape
    if not ends:
        return check(sgr.beam_select(x, scores), select(xv, sv))
    eos = V // 2
    done = np.arange(B * K).reshape(B, K) % 3 == 1
    check(sgr.beam_select(x, scores, torch.from_numpy(done).cuda(), eos),
          select(xv, sv, done, eos))
    check(sgr.beam_select(x, scores, eos=eos), select(xv, sv, None, eos))


@pytest.mark.parametrize("K,V", [(4, 28), (8, 5000), (32, 9000)])
def test_equal_logits_go_by_their_place(K, V):
    r = np.random.default_rng(2)
    for levels in (1, 2, 5):
        xv = r.integers(0, levels, (2, K, V)).astype(np.float32)
        x = torch.from_numpy(xv).cuda()
        # whole numbers and equal rows: scores that are equal are so exactly
        xv[:] = xv[:, :1]
        x = torch.from_numpy(xv).cuda()
        sv = np.repeat(-np.arange(2, dtype=np.float32)[:, None], K, 1)
        check(sgr.beam_select(x, torch.from_numpy(sv).cuda()), select(xv.astype(np.float64), sv))


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("K", [3, 32])
def test_sorted_logits(rising, K):
    """Every candidate in a few lanes: the most that a wave can have above its limit."""
    V = 9000
    xv = np.linspace(-4, 4, V).astype(np.float32)
    xv = np.stack([np.stack([(xv if rising else xv[::-1]) + 0.01 * k for k in range(K)])])
    sv = -np.linspace(0, 0.3, K, dtype=np.float32)[None]
    check(sgr.beam_select(torch.from_numpy(xv.copy()).cuda(), torch.from_numpy(sv).cuda()),
          select(xv.astype(np.float64), sv))


def test_columns_of_a_lane():
    """All large logits where one lane reads them (8 adjacent in every 512)."""
    V, K = 4096, 32
    r = np.random.default_rng(3)
    xv = r.standard_normal((1, K, V)).astype(np.float32)
    hot = (np.arange(V) // 8) % 64 == 17
    xv[:, :, hot] += 20
    sv = -r.random((1, K)).astype(np.float32)
    check(sgr.beam_select(torch.from_numpy(xv).cuda(), torch.from_numpy(sv).cuda()),
          select(xv.astype(np.float64), sv))


def test_first_step_from_one_beam():
    x, xv, _, _ = make(4, 3, 6, 40, "bf16")
    sv = np.full((3, 6), -np.inf, np.float32)
    sv[:, 0] = 0
    check(sgr.beam_select(x, torch.from_numpy(sv).cuda()), select(xv, sv))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_masked_rows_infinities_and_nan(dtype):
    x, xv, scores, sv = make(5, 6, 4, 5000, dtype)
    inf = float("inf")

    def put(b, k, at, v):
        x[b, k, at] = v
        xv[b, k, at] = v

    put(0, slice(None), slice(None), -inf)              # nothing anywhere: the lowest places
    put(1, 0, slice(None), -inf)                        # one beam without anything
    put(2, slice(None), slice(3, None), -inf)           # fewer candidates than places
    put(2, slice(1, None), slice(None), -inf)
    put(3, 1, 77, float("nan"))
    put(3, 2, slice(0, 4990), float("nan"))
    put(4, 1, 4999, inf)
    put(4, 2, slice(10, 13), inf)
    put(4, 3, 5, torch.finfo(DT[dtype]).min)
    put(4, 0, slice(100, None), torch.finfo(DT[dtype]).min)
    scores[5, 1], sv[5, 1] = float("nan"), np.nan
    scores[5, 2], sv[5, 2] = -inf, -np.inf
    check(sgr.beam_select(x, scores), select(xv, sv))
    done = np.zeros((6, 4), bool)
    done[0, 1] = done[1, 0] = done[5, 2] = done[5, 3] = True
    check(sgr.beam_select(x, scores, torch.from_numpy(done).cuda(), 4999),
          select(xv, sv, done, 4999))


@pytest.mark.parametrize("scale", [1e38, 3.3e38, 1e-39])
def test_logits_near_the_ends_of_fp32(scale):
    """Differences beyond fp32's range; and all alike to it but in their order."""
    r = np.random.default_rng(11)
    xv = (scale * r.uniform(-1, 1, (3, 4, 700))).astype(np.float32)
    xv[1] = -np.abs(xv[1]) - np.float32(scale * 0.01)
    xv[2, 1, 5], xv[2, 2, 9] = np.inf, -np.inf
    sv = -20 * r.random((3, 4)).astype(np.float32)
    check(sgr.beam_select(torch.from_numpy(xv).cuda(), torch.from_numpy(sv).cuda()),
          select(xv.astype(np.float64), sv))


def test_all_beams_finished():
    x, xv, scores, sv = make(6, 2, 5, 3, "fp32")
    x.fill_(float("nan"))                               # not looked at
    done = np.ones((2, 5), bool)
    for eos in (0, 2):
        check(sgr.beam_select(x, scores, torch.from_numpy(done).cuda(), eos),
              select(xv, sv, done, eos))


def test_scores_in_place_streams_and_graphs():
    x, xv, scores, sv = make(7, 4, 8, 9001, "bf16")
    done = torch.zeros(4, 8, dtype=torch.bool, device="cuda")
    want = sgr.beam_select(x, scores, done, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sgr.beam_select(x, scores, done, 5, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(map(torch.equal, want, got))
    s, d = scores.clone(), done.clone()
    out = (s, torch.empty_like(want[1]), torch.empty_like(want[2]), d)
    got = sgr.beam_select(x, s, d, 5, out=out)
    assert got[0] is s and got[3] is d and all(map(torch.equal, want, got))
    # a graph of three steps with the scores carried, replayed on new logits
    states = [torch.randn(32, 30, device="cuda"), torch.randn(3, 32, 8, device="cuda").bfloat16()]

    def steps(s, d, st):
        for _ in range(3):
            _, parents, _, _ = sgr.beam_select(x, s, d, 5, out=(
                s, torch.empty_like(want[1]), torch.empty_like(want[2]), d))
            sgr.beam_reorder([st[0], st[1].transpose(0, 1)], parents)

    with torch.cuda.stream(side):
        steps(scores.clone(), done.clone(), [t.clone() for t in states])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    s, d, st = scores.clone(), done.clone(), [t.clone() for t in states]
    with torch.cuda.graph(graph):
        steps(s, d, st)
    for k in range(4):
        x.copy_(x.flip(-1))
        s.copy_(scores), d.copy_(done)
        for a, b in zip(st, states):
            a.copy_(b)
        graph.replay()
        s2, d2, st2 = scores.clone(), done.clone(), [t.clone() for t in states]
        steps(s2, d2, st2)
        torch.cuda.synchronize()
        assert torch.equal(s, s2) and torch.equal(d, d2) and all(map(torch.equal, st, st2)), k


@pytest.mark.parametrize("K,V", [(1, 28), (4, 28), (8, 4000), (16, 50), (3, 9000), (32, 4096)])
def test_scores_and_ends_in_place(K, V):
    """Rows of one part and of more, few beams and many."""
    log(f"beam_select in place K={K} V={V}")
    x, _, scores, _ = make(11, 3, K, V, "bf16")
    done = torch.zeros(3, K, dtype=torch.bool, device="cuda")
    done[1, K // 2] = True
    want = sgr.beam_select(x, scores, done, 2)
    out = (scores, torch.empty_like(want[1]), torch.empty_like(want[2]), done)
    assert all(map(torch.equal, want, sgr.beam_select(x, scores, done, 2, out=out)))


def test_offsets_past_32_bits():
    """Texts 2^31 elements apart."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    V = 5000
    far = torch.empty((1 << 31) + 2 * V, dtype=torch.float32, device="cuda")
    x, xv, scores, sv = make(8, 2, 2, V, "fp32")
    y = far.as_strided((2, 2, V), (1 << 31, V, 1))
    y.copy_(x)
    check(sgr.beam_select(y, scores), select(xv, sv))


REORDER = [(1, 1), (1, 4), (3, 5), (2, 8), (2, 9), (3, 16), (2, 17), (1, 32)]


@pytest.mark.parametrize("B,K", REORDER)
@pytest.mark.parametrize("in_place", [True, False])
def test_reorder(B, K, in_place):
    log(f"beam_reorder {B} {K} in_place={in_place}")
    r = np.random.default_rng(9)
    rows = B * K
    new = lambda *s, dtype=torch.float32: torch.randint(-120, 120, s, device="cuda").to(dtype)
    wide = new(rows, 50, dtype=torch.float16)
    states = [new(rows, 6, 4), new(3, rows, 33, dtype=torch.bfloat16).transpose(0, 1),
              wide[:, 1:18], wide[:, 18:49], new(rows, 1, dtype=torch.uint8), new(rows, 300),
              new(rows, dtype=torch.int64), new(rows, 4, 5, 6).transpose(1, 2).contiguous()[:, :, 1:3],
              new(rows, 0), new(rows, 1031, dtype=torch.int8)]
    edges = wide[:, :1].clone(), wide[:, 49:].clone()
    parents = torch.from_numpy(r.integers(0, K, (B, K))).cuda()
    at = (parents + K * torch.arange(B, device="cuda")[:, None]).view(-1)
    want = [t[at].clone() for t in states]
    before = [t.clone() for t in states]
    outs = None
    if not in_place:
        outs = [torch.full_like(t, 1) for t in states]
        outs[1] = torch.full((3, rows, 33), 1, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        outs[5] = torch.full((300, rows), 1.0, device="cuda").t().contiguous()
    got = sgr.beam_reorder(states, parents, out=outs)
    torch.cuda.synchronize()
    for n, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), n
    assert torch.equal(edges[0], wide[:, :1]) and torch.equal(edges[1], wide[:, 49:])
    if in_place:
        assert all(a is b for a, b in zip(got, states))
    else:
        assert all(map(torch.equal, states, before))


def test_reorder_every_number_of_beams():
    for K in range(1, 33):
        log(f"beam_reorder K={K}")
        t = torch.arange(2 * K * 37, dtype=torch.int16, device="cuda").view(2 * K, 37)
        parents = torch.stack([torch.arange(K - 1, -1, -1, device="cuda"),
                               torch.arange(K, device="cuda") * 7 % K])
        want = t[(parents + K * torch.arange(2, device="cuda")[:, None]).view(-1)].clone()
        assert torch.equal(sgr.beam_reorder([t], parents)[0], want), K


def test_reorder_many_states_bad_parents_and_other_streams():
    states = [torch.randn(6, k + 1, device="cuda") for k in range(70)]   # several tables
    parents = torch.tensor([[0, -5, 99], [2, 1, 1 << 40]], device="cuda")   # the nearer bound
    at = torch.tensor([0, 0, 2, 5, 4, 5], device="cuda")
    want = [t[at] for t in states]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sgr.beam_reorder(states, parents, out=[torch.empty_like(t) for t in states], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(map(torch.equal, got, want))
    assert all(map(torch.equal, sgr.beam_reorder(states, parents), want))


def test_a_write_into_a_saved_tensor_is_seen():
    w = torch.randn(4, 3, device="cuda", requires_grad=True)
    t = torch.randn(4, 3, device="cuda")
    y = (w * t).sum()
    sgr.beam_reorder([t], torch.tensor([[1, 0, 3, 2]], device="cuda"))
    with pytest.raises(RuntimeError, match="modified"):
        y.backward()


def test_binding_refusals():
    x, _, scores, _ = make(10, 2, 4, 20, "fp32")
    done = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    for bad in (dict(logits=x.cpu()), dict(logits=x.double()), dict(logits=x[0]),
                dict(logits=x.transpose(1, 2)), dict(scores=scores[:1]), dict(scores=None),
                dict(scores=scores.double()), dict(finished=done), dict(finished=done.int(), eos=1),
                dict(eos=20), dict(eos=-1), dict(logits=x.repeat(1, 9, 1)),
                dict(out=(scores, None, None, None))):
        with pytest.raises((TypeError, ValueError, sgr.CkError)):
            sgr.beam_select(**{**dict(logits=x, scores=scores), **bad})
    parents = torch.zeros(2, 4, dtype=torch.int64, device="cuda")
    t = torch.randn(8, 6, device="cuda")
    for states, par, out in (
            ([t], parents.int(), None), ([t], parents.cpu(), None), ([t[:7]], parents, None),
            ([t.cpu()], parents, None), ([t, t], parents, None), ([t], parents, []),
            ([t], parents, [t[:, :3]]), ([t], parents, [t.half()]),
            ([t], parents, [torch.zeros(1, 6, device="cuda").expand(8, 6)]),
            ([torch.randn(8, 4, 6, 5, device="cuda")[:, :3, :4, :2]], parents, None)):
        with pytest.raises((TypeError, ValueError, sgr.CkError)):
            sgr.beam_reorder(states, par, out=out)
