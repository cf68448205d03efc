"""Beam search's calls whose outputs lie over what they read, or over one another, are
refused before any device work, where addresses, sizes and strides show it."""
import ctypes
import os

import pytest

import sparse_graph_recurrent_amd as sgr
from sparse_graph_recurrent_amd.beam import BeamShape, BeamState
from sparse_graph_recurrent_amd.sequence import CkSeq

BAD_VALUE = 12
B, K = 2, 4
ROWS = B * K
A = 1 << 24     # addresses that are never read or written: every call fails
PARENTS = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(sgr.LIB_PATH):
        from sparse_graph_recurrent_amd import build
        build.build()
    return sgr.lib()


def reorder(L, *rows, parents=PARENTS):
    states = (BeamState * len(rows))(*[BeamState(*r) for r in rows])
    assert L.ck_beam_reorder(states, len(rows), parents, B, K, None) == BAD_VALUE
    return L.ck_last_error().decode()


def dense(at, out=None, size=64):
    """A state of rows without gaps; in place without `out`."""
    return at, at if out is None else out, 1, size, size, 0, size, 0


def slices(at, out, size=64, row=256):
    """Rows of `size` bytes, slices of wider ones."""
    return at, out, 1, size, row, 0, row, 0


def test_reorder_output_over_its_state_with_gaps(L):
    for by in (1, 63, -63, 256, -256, 256 * (ROWS - 1) + 63):
        assert "lies over it" in reorder(L, slices(A, A + by))
    # strides that are not alike: without gaps over slices, pieces over rows
    assert "lies over it" in reorder(L, (A, A + 256 * 3, 1, 64, 256, 0, 64, 0))
    assert "lies over it" in reorder(L, (A, A + 16, 2, 32, 256, 128, 256, 64))


def test_reorder_states_over_one_another(L):
    last = 64 * ROWS - 1
    for a, b in ((dense(A), dense(A + 64)), (dense(A), dense(A + last)),
                 (dense(A + last), dense(A)), (dense(A), dense(4 * A, A + 8)),
                 (dense(4 * A, A + 8), dense(A)), (dense(A, 2 * A), dense(2 * A + 64, 3 * A)),
                 (dense(2 * A, 3 * A), dense(4 * A, 3 * A + last)),
                 (slices(A, A), slices(A + 63, A + 63)), (slices(A, A), dense(A + 256 * 7, 2 * A))):
        assert "share memory" in reorder(L, a, b)
        assert "share memory" in reorder(L, a, dense(8 * A, 9 * A), b)


def test_reorder_output_over_the_parents(L):
    for par in (A, A + 64, A + 64 * ROWS - 8, A - 8 * (ROWS - 1)):
        assert "parents" in reorder(L, dense(2 * A, A), parents=par)
        assert "parents" in reorder(L, dense(A), parents=par)


V = 100
PLACES = {n: (k + 2) * A for k, n in enumerate(
    ("logits", "scores", "finished", "out_scores", "parents", "tokens", "out_finished",
     "workspace"))}


def select(L, name, **kw):
    a = {**PLACES, **kw}
    x = a["logits"]
    x = x if isinstance(x, CkSeq) else CkSeq(x, K * V, V)
    shape = ctypes.byref(BeamShape(B, K, V, 3, 1))
    assert L.ck_beam_select(shape, x, a["scores"], a["finished"], a["out_scores"], a["parents"],
                            a["tokens"], a["out_finished"], a["workspace"], 2**40, None) == BAD_VALUE
    text = L.ck_last_error().decode()
    assert "must not lie over" in text and name in text, text


def test_select_outputs_over_what_is_read(L):
    p = PLACES
    for out in ("out_scores", "parents", "tokens", "out_finished", "workspace"):
        select(L, "logits", **{out: p["logits"]})
        select(L, "logits", **{out: p["logits"] + 2 * V * ROWS // 256 * 256 - 256})
    for at in (p["scores"] + 4, p["scores"] - 4, p["scores"] + 4 * (ROWS - 1)):
        select(L, "scores", out_scores=at)
    select(L, "scores", parents=p["scores"])
    select(L, "scores", out_finished=p["scores"] + 4 * ROWS - 1)
    select(L, "finished", out_finished=p["finished"] + 1)
    select(L, "finished", tokens=p["finished"])
    # a padded projection's rows: the last of them, and the next beam's first logit
    select(L, "logits", logits=CkSeq(p["logits"], K * 128, 128),
           out_scores=p["logits"] + 2 * (7 * 128 + V) - 4)
    select(L, "logits", logits=CkSeq(p["logits"], K * 128, 128), out_scores=p["logits"] + 2 * 128 - 4)
    select(L, "logits", logits=CkSeq(p["logits"], 0, 0), out_scores=p["logits"] + 2 * V - 4)


def test_select_outputs_over_one_another(L):
    p = PLACES
    select(L, "tokens", parents=p["tokens"])
    select(L, "tokens", parents=p["tokens"] + 8 * (ROWS - 1))
    select(L, "parents", out_scores=p["parents"] + 8)
    select(L, "out_finished", out_finished=p["out_scores"] + 31)
    select(L, "workspace", tokens=p["workspace"])
