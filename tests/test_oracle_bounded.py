"""The oracle of the bounded cache's operators, against hand-worked cases and identities."""
import numpy as np
import pytest

import gen
from oracle import bounded as B
from oracle import serving as S


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_is_a_rotation_by_the_position(interleaved):
    rng = np.random.default_rng(0)
    x, f = rng.standard_normal((3, 64)), 10000.0 ** (-np.arange(32) / 32)
    one = B.rotate(x, 1 * f, interleaved)
    assert np.allclose(np.linalg.norm(one, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.allclose(B.rotate(one, 6 * f, interleaved), B.rotate(x, 7 * f, interleaved))
    assert np.allclose(B.rotate(x, 0 * f, interleaved), x)
    # pairs: dim 0 goes with 1 or with 32
    e = np.zeros(64)
    e[0] = 1
    hit = np.nonzero(B.rotate(e, np.full(32, 0.5), interleaved))[0].tolist()
    assert hit == ([0, 1] if interleaved else [0, 32])


def test_front_row_norms():
    x = np.arange(1.0, 513.0)
    q, lat = B.front_row(np.ones((96, 512)) * 3, np.zeros((96, 64)), None, x, np.zeros(64), np.full(512, 2.0),
                         np.ones(32), 5, 0.0 + 1e-30, True)
    assert (q[:, :512] == 3).all() and np.isclose((lat[:512] ** 2).mean(), 4.0)
    q, _ = B.front_row(np.ones((96, 512)) * 3, np.zeros((96, 64)), np.full(512, 0.5), x, np.zeros(64), np.ones(512), np.ones(32),
                       5, 1e-30, True)
    assert np.allclose(q[:, :512], 0.5)


def test_visible_tokens():
    assert B.visible(10, 2, 3).tolist() == [0, 1, 7, 8, 9]
    assert B.visible(4, 2, 3).tolist() == [0, 1, 2, 3]
    assert B.visible(5, 0, 1).tolist() == [4]
    assert B.visible(3, 9, 1).tolist() == [0, 1, 2]


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
def test_a_wide_window_is_dense_attention(lat_fmt):
    inp = gen.make_inputs(2, 2, [90, 131], seed=1, lat_fmt=lat_fmt, bt_mode="permuted")
    none = lambda q: np.zeros_like(q)
    for b in range(2):
        lse = np.stack([B.window_mla(inp, 0, 1 << 20, b, t, none)[1] for t in range(2)])
        for t in range(2):
            out, l = S.prefix_mla(inp, [], 0, b, t)[:2]
            got = B.window_mla(inp, 7, 131, b, t, none)
            assert np.allclose(got[0], out) and np.allclose(got[1], l)
        # every row hands out a weight of 1 a head
        tok, w, _ = B.attention_mass(inp, 0, 1 << 20, lse, b, none)
        assert tok.tolist() == list(range(inp.ctx[b])) and np.isclose(w.sum(), 2 * 96)


def test_window_mass_sums_to_one_a_head():
    inp = gen.make_inputs(1, 3, [300], seed=2, bt_mode="permuted")
    none = lambda q: np.zeros_like(q)
    lse = np.stack([B.window_mla(inp, 5, 70, 0, t, none)[1] for t in range(3)])
    tok, w, _ = B.attention_mass(inp, 5, 70, lse, 0, none)
    assert tok.tolist() == [0, 1, 2, 3, 4] + list(range(298 - 70, 300)) and np.isclose(w.sum(), 3 * 96)
    lse[1, 4] = -np.inf  # an empty head adds nothing
    assert np.isclose(B.attention_mass(inp, 5, 70, lse, 0, none)[1].sum(), 3 * 96 - 1)


def test_chosen_tokens():
    m = np.array([0, 5, 1, 5, np.nan, 5, -0.0, 0.0, 2], np.float32)
    assert B.chosen(m, 9, 4, 0, 0) == [1, 3, 5, 8]
    assert B.chosen(m, 9, 3, 1, 1) == [0, 1, 8]
    assert B.chosen(m, 9, 2, 0, 0) == [1, 3]
    assert B.chosen(m, 9, 7, 0, 0) == [0, 1, 2, 3, 5, 6, 8]  # 0 at 0 and 6 (-0 ties with 0: the lower index), not 7
    assert B.chosen(m, 9, 8, 0, 0) == [0, 1, 2, 3, 5, 6, 7, 8]  # the NaN goes first
    assert B.chosen(m, 9, 1, 4, 4) == [0] and B.chosen(m, 9, 0, 4, 4) == []


def test_evict_by_hand():
    """Two requests share their first page; the first is cut within it, the second behind it."""
    table = np.array([[3, 1, -1], [3, 2, 5]], np.int32)
    ctx, refs = np.array([100, 140], np.int32), np.array([0, 1, 1, 2, 0, 1], np.int32)
    pool = np.arange(6 * 64, dtype=np.int64).astype(np.uint8).reshape(6, 64, 1).repeat(576, 2).reshape(6, -1)
    mass = np.ones((2, 192), np.float32)
    mass[0, 10] = 0.5
    mass[1, 70:] = 2
    kept = np.full((2, 192), -9, np.int32)
    first = pool[3].copy()
    err = B.tokens_evict(table, ctx, refs, mass, [99, -1], 0, 0, [("lat_fp8", [pool])], kept)
    assert err == 0 and ctx.tolist() == [99, 140] and table[0].tolist() == [0, 1, -1] and refs.tolist() == [1, 1, 1, 1, 0, 1]
    rows = pool.reshape(6, 64, 576)[:, :, 0]
    was = np.arange(6 * 64).astype(np.uint8).reshape(6, 64)
    want = np.delete(np.concatenate([was[3], was[1]])[:100], 10)
    assert (np.concatenate([rows[0], rows[1]])[:99] == want).all() and (pool[3] == first).all()
    assert kept[0, :99].tolist() == [i for i in range(100) if i != 10] and (kept[0, 99:] == -9).all()
    assert kept[1, :140].tolist() == list(range(140)) and mass[0, 99] == 0 and mass[0, 98] == 1
    # 64 tokens of the second: those from 70 on stay, from 76 on by the tie; no page of it is free of change
    err = B.tokens_evict(table, ctx, refs, mass, [-1, 64], 0, 0, [("lat_fp8", [pool])], kept)
    assert err == 0 and table[1].tolist() == [3, -1, -1] and refs.tolist() == [1, 1, 0, 1, 0, 0]
    assert kept[1, :64].tolist() == list(range(70, 134))


def test_evict_without_fresh_pages_leaves_the_request():
    table = np.array([[0], [0]], np.int32)
    ctx, refs, mass = np.array([60, 60], np.int32), np.array([2], np.int32), np.ones((2, 64), np.float32)
    err = B.tokens_evict(table, ctx, refs, mass, [30, 60], 0, 30, [])
    assert err == S.ERR_NO_PAGES and ctx.tolist() == [60, 60] and refs.tolist() == [2]
    # the first tokens alone: nothing moves, no page is needed
    assert B.tokens_evict(table, ctx, refs, mass, [30, 0], 30, 0, []) == 0 and ctx.tolist() == [30, 0] and refs.tolist() == [1]
