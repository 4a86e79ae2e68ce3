"""The oracle of the calls around the decode step, pinned on hand-made states,
invariants and closed forms (CPU only)."""
import numpy as np
import pytest

import gen
from oracle import dsa as O
from oracle import serving as S


def _state(lens, shared_pages=0, num_pages=40, width=8, seed=0):
    rng = np.random.default_rng(seed)
    perm = rng.permutation(num_pages).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    refs = np.zeros(num_pages, np.int32)
    at = shared_pages
    for b, n in enumerate(lens):
        k = S.pages_of(n)
        s = min(shared_pages, k)
        table[b, :s] = perm[:s]
        table[b, s:k] = perm[at:at + k - s]
        at += k - s
        np.add.at(refs, table[b, :k], 1)
    pools = [rng.integers(0, 255, (num_pages, 32), dtype=np.uint8)]
    return table, np.array(lens, np.int32), refs, pools


def _check(table, ctx, refs):
    """The counts are what the tables hold, and no entry is used twice in a row."""
    held = np.zeros_like(refs)
    for b, n in enumerate(ctx):
        row = table[b, :S.pages_of(int(n))]
        assert (row >= 0).all() and len(set(row.tolist())) == len(row)
        np.add.at(held, row, 1)
    assert np.array_equal(held, refs)


def _text(table, ctx, pools, b):
    """The bytes that request b sees."""
    return [pools[0][table[b, s // 64], s % 32] for s in range(int(ctx[b]))]


def test_resize_grows_trims_frees_and_copies():
    table, ctx, refs, pools = _state([100, 130, 64, 0], shared_pages=1)
    S.pages_fork(table, ctx, refs, [1], [3])
    _check(table, ctx, refs)
    seen = [_text(table, ctx, pools, b) for b in range(4)]
    shared = table[1, 2]
    assert refs[shared] == 2
    free = [p for p in range(40) if refs[p] == 0]
    assert S.pages_resize(table, ctx, refs, [0, 200, -1, 135], pools) == 0
    _check(table, ctx, refs)
    assert ctx.tolist() == [0, 200, 64, 135]
    # a copy first, then the appended page; the next request's copy after it
    assert table[1, 2] == free[0] and table[1, 3] == free[1] and table[3, 2] == free[2]
    assert refs[shared] == 0
    for b, n in ((1, 130), (2, 64), (3, 130)):
        assert _text(table, ctx, pools, b)[:n] == seen[b][:n]


def test_resize_without_enough_pages_serves_a_prefix_of_the_requests():
    table, ctx, refs, pools = _state([64, 64, 64], num_pages=5, width=4)
    assert S.pages_resize(table, ctx, refs, [128, 256, 65], pools) == S.ERR_NO_PAGES
    assert ctx.tolist() == [128, 64, 64]
    _check(table, ctx, refs)


def test_resize_leaves_pages_without_references_alone():
    # request 0's open page has no references: it is free, and another request may get it
    table, ctx, refs, pools = _state([100, 64, 64], num_pages=8)
    lost = table[0, 1]
    refs[lost] = 0
    first = min(p for p in range(8) if refs[p] == 0)
    assert S.pages_resize(table, ctx, refs, [101, 65, 0], pools) == S.ERR_PAGES
    assert ctx.tolist() == [100, 65, 0] and table[1, 1] == first and refs[first] == 1
    # released, and handed out by the same call: the new holder keeps it, in either order
    for lens, new in (([64, 100], [65, 0]), ([100, 64], [0, 65])):
        table, ctx, refs, pools = _state(lens, num_pages=3)
        lost = table[lens.index(100), 1]
        refs[lost] = 0
        assert S.pages_resize(table, ctx, refs, new, pools) == S.ERR_PAGES
        assert table[lens.index(64), 1] == lost and refs[lost] == 1


def test_fork_refuses_taken_slots():
    table, ctx, refs, pools = _state([100, 0, 0, 50])
    err = S.pages_fork(table, ctx, refs, [0, 0, 3, 0, 9], [1, 1, 2, 3, 2])
    assert err == S.ERR_PAGES
    assert ctx.tolist() == [100, 100, 50, 50]
    _check(table, ctx, refs)


@pytest.mark.parametrize("seed", range(4))
def test_compact_keeps_what_every_request_sees(seed):
    table, ctx, refs, pools = _state([100, 130, 0, 300], shared_pages=1, seed=seed)
    seen = [_text(table, ctx, pools, b) for b in range(4)]
    old = table.copy()
    where, live, err = S.pages_compact(table, ctx, refs, pools)
    assert err == 0 and live == 1 + 1 + 2 + 4 and (refs[:live] > 0).all() and (refs[live:] == 0).all()
    _check(table, ctx, refs)
    assert [_text(table, ctx, pools, b) for b in range(4)] == seen
    assert (where[old[old >= 0]] == table[old >= 0]).all()


def test_verified_tokens_follow_the_target():
    """One draft over five tokens: the first token out is distributed as the target,
    whatever the draft (checked by integrating over a grid of uniform numbers)."""
    p = np.array([0.1, 0.4, 0.2, 0.05, 0.25])
    q = np.array([0.3, 0.1, 0.2, 0.35, 0.05])
    got = np.zeros(5)
    grid = (np.arange(64) + 0.5) / 64
    for x in range(5):
        for u0 in grid:
            u = np.array([[u0, g] for g in grid], np.float32)
            n = len(grid)
            _, out, _, err = S.verify_draft(np.tile(p, (n, 2, 1)), np.tile(q, (n, 1, 1)), np.full((n, 1), x), None, u, None)
            assert err == 0
            got += q[x] * np.bincount(out[:, 0], minlength=5) / n / len(grid)
    # each threshold cuts a grid of 64 off by at most one half cell
    assert np.abs(got - p).max() < 2 / 64


def test_verify_edges():
    one = np.float32(1) - np.float32(2) ** -24
    t = np.zeros((1, 2, 4))
    t[0, 0], t[0, 1] = [0.5, 0.5, 0, 0], [0, 0, 0.25, 0.75]
    d = np.array([[[0.0, 1.0, 0, 0]]])
    # accepted: the bonus token from the last row; rejected: what p has beyond q
    assert S.verify_draft(t, d, [[1]], None, [[0.25, 0.0]], [70])[1].tolist() == [[1, 2]]
    assert S.verify_draft(t, d, [[1]], None, [[0.25, one]], [70])[1].tolist() == [[1, 3]]
    assert S.verify_draft(t, d, [[1]], None, [[0.5, one]], [70])[1].tolist() == [[0, -1]]
    assert S.verify_draft(t, None, [[2]], None, [[0.0, 0.0]], [70])[1].tolist() == [[0, -1]]
    assert S.verify_draft(t, d, [[1]], [0], [[0.0, 0.6]], [70])[1].tolist() == [[1, -1]]
    # equal rows: a rejected draft (u * q = p) leaves no mass beyond q, so p itself is drawn from
    t[0, 0] = d[0, 0] = [0, 0.25, 0.75, 0]
    assert S.verify_draft(t, d, [[0]], None, [[0.5, 0.5]], [70])[1].tolist() == [[2, -1]]


def test_entries_that_are_no_probabilities_count_as_zero_in_the_draft_tests():
    for bad in (np.inf, 1.5, np.nan, -0.25):
        t, d = np.full((1, 2, 4), 0.25), np.full((1, 1, 4), 0.25)
        t[0, 0, 2] = bad  # p(x) counts as 0: the draft does not pass
        acc, out, _, err = S.verify_draft(t, d, [[2]], None, [[0.0, 0.5]], [70])
        assert acc[0] == 0 and err == S.ERR_PROB and out[0, 0] in (0, 1, 3)
        t, d = np.full((1, 2, 4), 0.25), np.full((1, 1, 4), 0.25)
        d[0, 0, 2] = bad  # q(x) counts as 0: u q < p holds
        acc, out, _, err = S.verify_draft(t, d, [[2]], None, [[0.9375, 0.5]], [70])
        assert acc[0] == 1 and err == S.ERR_PROB and out[0].tolist() == [2, 2]


def test_prefix_mla_is_dense_attention():
    inp = gen.make_inputs(2, 2, [200, 150], seed=3, bt_mode="permuted")
    pages = inp.block_table[0, :1].copy()
    inp.block_table[1, 0] = pages[0]
    for b in range(2):
        for t in range(2):
            out, lse, mass, bulk = S.prefix_mla(inp, pages, 64, b, t)
            ref = O.dense_mla(inp, b, t)
            assert np.allclose(out, ref[0]) and np.allclose(lse, ref[1])
            assert (np.abs(out) <= mass + 1e-12).all() and (bulk > 0).all()
