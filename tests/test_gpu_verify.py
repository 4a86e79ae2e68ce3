"""dsa_verify_draft against the oracle's integer arithmetic: accepted counts, tokens,
remaining lengths and error bits, all exact."""
import numpy as np
import pytest

import dsa_sparse_mla_paged_gb300 as dsa
from oracle import serving as S

pytestmark = pytest.mark.gpu
NAMES = ("float32", "bfloat16", "float16")


@pytest.fixture(scope="module", autouse=True)
def _need(lib, cuda_ok):
    yield


def _rows(rng, B, n, V, dtype, sharp=2.0, near=0.7):
    import torch

    z = rng.standard_normal((B, n, V)) * sharp
    e = lambda x: torch.from_numpy(np.exp(x) / np.exp(x).sum(-1, keepdims=True)).to(getattr(torch, dtype))
    q = e(z[:, :-1] + near * rng.standard_normal((B, n - 1, V)))
    tok = np.array([[rng.choice(V, p=q[b, i].double().numpy() / q[b, i].double().sum().item()) for i in range(n - 1)]
                    for b in range(B)], np.int32).reshape(B, n - 1)
    return e(z), q, tok


def _run(target, draft, tokens, counts, u, ctx, p=None, ws=None):
    import torch

    B, n, _ = target.shape
    p = p or dsa.make_params(batch=B, n_q=n, max_pages_per_req=100, num_pages=1, key_page_stride=8448, lat_page_stride=36864)
    ws = torch.zeros(dsa.workspace_size(p), dtype=torch.uint8, device="cuda") if ws is None else ws
    i32 = lambda a: None if a is None else torch.tensor(np.asarray(a, np.int32), device="cuda")
    acc, out, new = i32(np.full(B, -9)), i32(np.full((B, n), -9)), i32(np.full(B, -9))
    dsa.verify_draft(p, target.cuda(), None if draft is None else draft.cuda(), i32(tokens), i32(counts),
                     torch.tensor(np.asarray(u, np.float32), device="cuda"), i32(ctx), acc, out, new if ctx is not None else None,
                     ws)
    bits = dsa.get_device_error(ws)
    return acc.cpu().numpy(), out.cpu().numpy(), new.cpu().numpy() if ctx is not None else None, bits


def _check(target, draft, tokens, counts, u, ctx):
    got = _run(target, draft, tokens, counts, u, ctx)
    ref = S.verify_draft(target.double().numpy(), None if draft is None else draft.double().numpy(), tokens, counts, u, ctx)
    assert np.array_equal(got[0], ref[0]), "accepted"
    assert np.array_equal(got[1], ref[1]), "tokens"
    if ctx is not None:
        assert np.array_equal(got[2], ref[2]), "new lengths"
    assert got[3] == ref[3]
    return got


@pytest.mark.parametrize("dtype", NAMES)
@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (1, 2, 2), (3, 4, 31), (2, 3, 257), (5, 8, 4099), (2, 6, 9000), (2, 2, 33001)])
def test_matches_oracle(dtype, B, n, V):
    rng = np.random.default_rng(B * 100 + n + V)
    target, draft, tokens = _rows(rng, B, n, V, dtype)
    u = rng.random((B, n), dtype=np.float32)
    _check(target, draft, tokens, None, u, rng.integers(n, 500, B))
    _check(target, draft, tokens, rng.integers(0, n, B), rng.random((B, n), dtype=np.float32), None)
    _check(target, None, tokens, None, rng.random((B, n), dtype=np.float32), rng.integers(n, 500, B))


def test_many_draws():
    """256 requests: accepted counts from 0 to all, draws over the whole row."""
    rng = np.random.default_rng(4)
    target, draft, tokens = _rows(rng, 256, 5, 300, "float32", near=0.9)
    acc, out, _, bits = _check(target, draft, tokens, None, rng.random((256, 5), dtype=np.float32), np.full(256, 70))
    assert bits == 0 and set(acc.tolist()) == {0, 1, 2, 3, 4}


@pytest.mark.parametrize("u", [0.0, 2.0 ** -30, 0.5, 1 - 2.0 ** -24])
def test_threshold_at_the_edges(u):
    """Weights that are powers of two put thresholds exactly on borders between tokens."""
    import torch

    V = 6000
    t = torch.zeros(4, 1, V)
    t[0, 0, 17] = 1.0
    t[1, 0, :4096] = 2.0 ** -12
    t[2, 0, [0, V - 1]] = 0.5
    t[3, 0, 4096:4096 + 1024] = 2.0 ** -10
    _check(t, None, np.zeros((4, 0)), None, np.full((4, 1), u), np.full(4, 3))


def test_acceptance_at_equality_and_no_mass_beyond_the_draft():
    import torch

    t = torch.tensor([[[0.25, 0.75, 0.0], [0.0, 0.0, 1.0]]]).repeat(3, 1, 1)
    d = torch.tensor([[[0.5, 0.5, 0.0]], [[0.25, 0.75, 0.0]], [[0.25, 0.75, 0.0]]])
    # u * q == p does not pass; equal rows pass below 1 and fall back to p at 1 (an out-of-range test number)
    u = np.array([[0.5, 0.3], [1 - 2.0 ** -24, 0.0], [1.0, 0.5]], np.float32)
    acc, out, _, _ = _check(t, d, [[0], [0], [0]], None, u, [9, 9, 9])
    assert acc.tolist() == [0, 1, 0] and out.tolist() == [[1, -1], [0, 2], [1, -1]]


def test_bad_inputs_are_reported():
    import torch

    rng = np.random.default_rng(8)
    target, draft, tokens = _rows(rng, 6, 3, 500, "float32")
    u = rng.random((6, 3), dtype=np.float32)
    ctx = np.full(6, 50)
    zero = np.zeros_like(u)
    bad = tokens.copy()
    bad[0, 0], bad[1, 1], bad[2, 0] = -1, 500, 2 ** 31 - 1
    assert _check(target, draft, bad, None, zero, ctx)[3] == S.ERR_DRAFT
    assert _check(target, None, bad, None, zero, ctx)[3] == S.ERR_DRAFT
    assert _check(target, draft, tokens, [0, 1, 2, 3, -1, 2], u, ctx)[3] == S.ERR_DRAFT
    assert _check(target, draft, tokens, None, u, [2, 3, 50, 0, -4, 3])[3] == S.ERR_CTX
    worse = target.clone()
    worse[0, :, 7], worse[1, :, 7], worse[2, :, 7], worse[3] = float("nan"), -0.5, float("inf"), 0.0
    worse[4] = 0.9  # sums to 450
    got = _check(worse, None, tokens, np.zeros(6), u, ctx)
    assert got[3] == S.ERR_PROB and got[1][3, 0] == -1 and got[1][4, 0] == -1
    d = draft.clone()
    d[5, 0, 3] = float("nan")
    one = u.copy()
    one[:, 0] = 1.0
    assert _check(target, d, tokens, None, one, ctx)[3] == S.ERR_PROB
    for v in (-1.0, 1.0, 7.5, float("nan")):
        last = zero.copy()
        last[:, 2] = v
        _check(target, draft, tokens, np.zeros(6), last, ctx)


def test_sums_that_would_wrap_the_integers():
    """Rows of ones sum far past 2^4 (where 2^-60 units leave 64 bits): no token, an error, nothing else."""
    import torch

    for V in (5, 16, 17, 40, 4096, 70000):
        t = torch.ones(1, 1, V)
        got = _run(t, None, np.zeros((1, 0)), None, [[0.4]], [5])
        assert got[1].tolist() == [[-1]] and got[3] == S.ERR_PROB, V


def test_strided_and_misaligned_rows():
    import torch

    rng = np.random.default_rng(11)
    for dtype in NAMES:
        target, draft, tokens = _rows(rng, 2, 3, 1001, dtype)
        wide_t = torch.full((2, 3, 1013), float("nan")).to(target.dtype)
        wide_t[:, :, 5:1006] = target
        wide_d = torch.full((2, 2, 1007), float("nan")).to(target.dtype)
        wide_d[:, :, 3:1004] = draft
        u = rng.random((2, 3), dtype=np.float32)
        ref = S.verify_draft(target.double().numpy(), draft.double().numpy(), tokens, None, u, [9, 9])
        got = _run(wide_t.cuda()[:, :, 5:1006], wide_d.cuda()[:, :, 3:1004], tokens, None, u, [9, 9])
        assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1]) and got[3] == 0


def test_forty_drafts():
    """More drafts than a warp has lanes."""
    import torch

    rng = np.random.default_rng(12)
    target, draft, tokens = _rows(rng, 3, 41, 50, "float32", sharp=0.3, near=0.02)
    u = rng.random((3, 41), dtype=np.float32) * 0.9
    acc = _check(target, draft, tokens, [40, 35, 33], u, np.full(3, 60))[0]
    assert acc.max() > 32


def test_captured_twice_with_one_workspace():
    import torch

    rng = np.random.default_rng(13)
    cases = []
    p = dsa.make_params(batch=4, n_q=3, max_pages_per_req=10, num_pages=1, key_page_stride=8448, lat_page_stride=36864)
    ws = torch.zeros(dsa.workspace_size(p), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        target, draft, tokens = _rows(rng, 4, 3, 5000, "float32")
        u = rng.random((4, 3), dtype=np.float32)
        ref = S.verify_draft(target.double().numpy(), draft.double().numpy(), tokens, None, u, None)
        args = (target.cuda(), draft.cuda(), torch.tensor(tokens, device="cuda"), None, torch.tensor(u, device="cuda"), None,
                torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(4, 3, dtype=torch.int32, device="cuda"), None, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dsa.verify_draft(p, *args)
        cases.append((g, args, ref))
    for g, args, ref in cases + cases[::-1]:
        args[6].fill_(-9), args[7].fill_(-9)
        g.replay()
        assert np.array_equal(args[6].cpu().numpy(), ref[0]) and np.array_equal(args[7].cpu().numpy(), ref[1])


@pytest.mark.parametrize("dtype", NAMES)
@pytest.mark.parametrize("V", [9, 255, 5003, 20011])
def test_rows_on_every_boundary(dtype, V):
    """Row strides of 8k + 1 and 8k + 3 elements: p's and q's rows differ by every shift. NaN lies between rows."""
    import torch

    rng = np.random.default_rng(V)
    B, n = 17, 2
    target, draft, _ = _rows(rng, B, n, V, dtype)
    tokens = (draft.double() - target[:, :1].double()).argmax(-1).numpy().astype(np.int32)
    u = np.stack([np.full(B, 0.999), rng.random(B)], 1).astype(np.float32)

    def spread(x, residue):
        rows, stride = x.reshape(-1, V), (V + 15) // 8 * 8 + residue
        buf = torch.full((len(rows) * stride,), float("nan"), dtype=x.dtype, device="cuda")
        view = buf.as_strided((x.shape[0], x.shape[1], V), (x.shape[1] * stride, stride, 1))
        view.copy_(x)
        return view

    for src in (draft, None):
        got = _run(spread(target, 1), None if src is None else spread(src, 3), tokens, None, u, np.full(B, 70))
        ref = S.verify_draft(target.double().numpy(), None if src is None else src.double().numpy(), tokens, None, u, np.full(B, 70))
        for g, r in zip(got[:3], ref):
            assert np.array_equal(g, r)
        assert got[3] == ref[3] == 0
        assert (got[0] == 0).sum() >= B // 2


def test_rows_beyond_four_gigabytes():
    import torch

    rng = np.random.default_rng(21)
    target, draft, tokens = _rows(rng, 5, 4, 3001, "bfloat16")
    far = 1 << 28  # elements between rows
    wide = lambda x: torch.empty(x.shape[0] * x.shape[1] * far, dtype=x.dtype, device="cuda").as_strided(
        x.shape, (x.shape[1] * far, far, 1)).copy_(x)
    u = rng.random((5, 4), dtype=np.float32)
    got = _run(wide(target), wide(draft), tokens, None, u, np.full(5, 70))
    ref = S.verify_draft(target.double().numpy(), draft.double().numpy(), tokens, None, u, np.full(5, 70))
    for g, r in zip(got, ref):
        assert np.array_equal(g, r)


@pytest.mark.parametrize("dtype", NAMES)
def test_entries_that_are_no_probabilities_in_the_draft_tests(dtype):
    """What a draft is tested with counts as 0 like any other entry outside [0, 1]: in p it does not pass, in q it
    does, and both are reported."""
    import torch

    rng = np.random.default_rng(31)
    for bad in (float("inf"), 1.5, float("nan"), -0.25):
        for where in ("p", "q"):
            target, draft, tokens = _rows(rng, 4, 4, 200, dtype)
            t, d = target.clone(), draft.clone()
            for b, i in ((0, 0), (1, 1), (2, 2)):
                (t if where == "p" else d)[b, i, int(tokens[b, i])] = bad
            u = np.full((4, 4), 2.0 ** -10, np.float32)
            acc, _, _, bits = _check(t, d, tokens, None, u, np.full(4, 60))
            assert bits == S.ERR_PROB
            if where == "p":
                assert acc[0] == 0 and acc[1] <= 1 and acc[2] <= 2
            if where == "p":
                assert _check(t, None, tokens, None, u, np.full(4, 60))[3] == S.ERR_PROB
