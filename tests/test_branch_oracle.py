"""Pins of oracle/branch_oracle.py: examples worked by hand and identities with other parts of
the oracle."""

import numpy as np

from oracle import attn_oracle as attn
from oracle import branch_oracle as ora


def test_fork_and_reserve_by_hand():
    # one prompt of 40 tokens in pages 5, 2, 7 of 16 tokens; page 0 is another's
    table, refs = np.array([[5, 2, 7, -1]]), np.array([1, 0, 1, 0, 0, 1, 0, 1])
    t, n, refs = ora.fork(table, [40], [[0, 0, 3]], refs, 16)
    assert t.tolist() == [[5, 2, 7, -1], [5, 2, 7, -1], [-1] * 4] and n.tolist() == [40, 40, 0]
    assert refs.tolist() == [1, 0, 2, 0, 0, 2, 0, 2]
    # the first child leaves page 7 for a copy in page 1, the second keeps it; the third starts in page 3
    t, refs, src, dst, info = ora.reserve(t, n, refs, 1, 16)
    assert t.tolist() == [[5, 2, 1, -1], [5, 2, 7, -1], [3, -1, -1, -1]]
    assert src.tolist() == [7, -1, -1] and dst.tolist() == [1, -1, -1] and info.tolist() == [0, 2]
    assert refs.tolist() == [1, 1, 2, 1, 0, 2, 0, 1]
    # again: nothing changes
    assert ora.reserve(t, n, refs, 1, 16)[0].tolist() == t.tolist()
    # 30 tokens more: two pages for the first two, one for the third, four of two are there
    t, refs, src, dst, info = ora.reserve(t, n, refs, 30, 16)
    assert t.tolist() == [[5, 2, 1, 4], [5, 2, 7, 6], [3, -1, -1, -1]] and info.tolist() == [1, 0]
    t, refs = ora.free(t, refs, 16, [0, 33, 0], [20, 48, 0])
    assert t.tolist() == [[5, 2, -1, -1], [-1, -1, 7, -1], [-1] * 4] and refs.tolist() == [1, 0, 1, 0, 0, 1, 0, 1]
    t, refs, remap, pairs = ora.compact(t, refs)
    assert pairs == [(5, 1), (7, 3)] and t.tolist() == [[1, 2, -1, -1], [-1, -1, 3, -1], [-1] * 4]
    assert refs.tolist() == [1, 1, 1, 1, 0, 0, 0, 0] and remap.tolist() == [0, -1, 2, -1, -1, 1, -1, 3]


def test_references_count_the_entries_of_all_tables():
    rng = np.random.default_rng(0)
    page, n_pages, width = 16, 60, 5
    table, lens, refs = np.full((3, width), -1), np.array([0, 0, 0]), np.zeros(n_pages, int)
    count = lambda *ts: np.bincount(np.concatenate([t[t >= 0] for t in ts]), minlength=n_pages)  # noqa: E731
    for step in range(30):
        T = int(rng.integers(0, 20))
        table, refs, src, dst, info = ora.reserve(table, lens, refs, T, page)
        assert (refs == count(table)).all() and info[1] == (refs == 0).sum() and info[0] == 0
        # nobody shares a page that is written
        for b, n in enumerate(lens):
            for j in range(n // page, min(-(-(n + T) // page), width) if T else 0):
                assert refs[table[b, j]] == 1
        lens = np.minimum(lens + T, page * width)
        table, lens, refs = ora.fork(table, lens, [rng.integers(0, 3, 3)], refs, page)
        assert (refs == count(table)).all()
        if lens.max() > 50:
            table, refs = ora.free(table, refs, page, None, lens := lens // 2)
            assert (refs == count(table)).all()


def test_attn_shared_is_attn_step_where_rows_agree():
    rng = np.random.default_rng(1)
    K, V = attn.Cache(10, 2, 16, 16), attn.Cache(10, 2, 16, 16)
    for c in (K, V):
        c.val[:] = attn.e4m3(rng.normal(size=c.val.shape) * 50)
        c.scale[:] = 2.0 ** rng.integers(-7, -4, c.scale.shape)
    table = np.array([[3, 1, 5], [3, 1, 6], [3, 1, 7], [0, 2, 4]])
    q = rng.normal(size=(4, 2, 4, 16))
    for window in (0, 20):
        a = ora.attn_shared(q, K, V, table, [40, 33, 32, 9], [0, 3], [32], 0.25, None, window)
        assert np.array_equal(a, attn.attn_step(q, K, V, table, [40, 33, 32, 9], 0.25, None, window))


def test_beam_select_by_hand():
    x = np.log(np.array([[[0.5, 0.25, 0.25], [0.125, 0.375, 0.5]]]))
    s, b, w = ora.beam_select(x, np.log([[0.5, 0.5]]), 5)
    assert b.tolist() == [[0, 1, 1, 0, 0]] and w.tolist() == [[0, 2, 1, 1, 2]]
    assert np.allclose(np.exp(s), [[0.25, 0.25, 0.1875, 0.125, 0.125]])
    s, b, w = ora.beam_select(x, np.log([[0.5, 0.5]]), 3, [[0, 1]], 2)
    assert b.tolist() == [[1, 0, 0]] and w.tolist() == [[2, 0, 1]] and np.allclose(np.exp(s), [[0.5, 0.25, 0.125]])
    s, b, w = ora.beam_select(np.where(np.arange(3) < 1, x, -np.inf), [[0.0, -np.inf]], 2)
    assert s.tolist() == [[0.0, -np.inf]] and b.tolist() == [[0, -1]] and w.tolist() == [[0, -1]]


def test_state_reorder_by_hand():
    s = np.arange(8).reshape(4, 2)
    assert ora.state_reorder(s, [[1, 1, 0], [0, -1, 2]]).tolist() == [[2, 3], [2, 3], [0, 1], [4, 5], [0, 0], [0, 0]]
