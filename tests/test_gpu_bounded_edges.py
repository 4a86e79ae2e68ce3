"""The bounded cache's calls where the other tests do not go: two calls at once, the choice by clusters of eight, rows that far
outnumber their tiles, and pages past 4 GB that do move."""
import numpy as np
import pytest

import dsa_sparse_mla_paged_gb300 as dsa
from oracle import bounded as B

from dsa_testlib import Dev
from test_gpu_evict import FMT, PAGE_BYTES, State
from test_gpu_window import check_mass, launch, make, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need(lib, cuda_ok):
    yield


@pytest.mark.parametrize("n", [65537, 99999, 131072])
@pytest.mark.parametrize("values", [1, 3, 1000])
def test_a_choice_by_clusters_of_eight(n, values):
    """Tables of more than 65,536 and at most 131,072 tokens; equal weights in every CTA's slice, so that the last tie that stays
    lies in any of them."""
    s = State([n], ("key_mxfp4",), seed=21)
    assert 65536 < s.width * 64 <= 131072
    s.mass[:] = np.random.default_rng(values).integers(0, values, s.mass.shape)
    s.check([n // 2 + 77], 4, 1000)


def test_choices_of_several_requests_by_clusters():
    s = State([70000, 300, 66000], ("key_mxfp4",), seed=22)
    s.mass[:] = np.random.default_rng(4).integers(0, 2, s.mass.shape)
    s.check([41000, 299, 12345], 4, 100)


def test_pages_that_move_past_four_gigabytes():
    """A pool of 9 GB: rows are read from and written to pages that begin past 2^32 bytes."""
    import torch

    s = State([500, 400], ("lat_fp8",), seed=15, spare=3)
    n = s.num_pages
    gap = (9 << 30) // n // 16 * 16
    s.to_device()
    pool = torch.empty(n * gap, dtype=torch.uint8, device="cuda")
    view = pool.as_strided((n, PAGE_BYTES["lat_fp8"]), (gap, 1))
    view.copy_(s.d_raw[0][:, 0])
    s.d_pools = dsa.make_token_pools([(pool, FMT["lat_fp8"], 1, 0, gap)])
    before = s.raw[0].copy()
    s.call([300, 350], 3, 50)
    assert dsa.get_device_error(s.ws) == 0
    assert B.tokens_evict(s.table, s.ctx, s.refs, s.mass, [300, 350], 3, 50, s.pools(), s.kept) == 0
    changed = np.nonzero((s.raw[0] != before).any(axis=(1, 2)))[0]
    assert (changed * gap >= 1 << 32).sum() >= 2 and (changed * gap < 1 << 32).any()
    s.d_raw[0][:, 0] = view
    s.same()


def test_two_evictions_at_once():
    """Two grids whose CTAs meet, on two streams, each on its own pools and workspace."""
    import torch

    states = [State([30000, 17000, 500], ("key_fp8", "lat_fp8"), seed=31), State([900, 41000], ("lat_nvfp4",), 2, seed=32)]
    cuts = [([20000, 16999, 100], [12000, 8000, 99], [700, 7999, 0]), ([899, 30000], [400, 29990], [-1, 3000])]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in states:
        s.to_device()
    budgets = [[torch.tensor(b, dtype=torch.int32, device="cuda") for b in c] for c in cuts]
    torch.cuda.synchronize()
    for i in range(3):
        for s, b, stream in zip(states, budgets, streams):
            s.call(b[i], 4, 60, stream=stream)
    torch.cuda.synchronize()
    for s, c in zip(states, cuts):
        assert dsa.get_device_error(s.ws) == 0
        for b in c:
            assert B.tokens_evict(s.table, s.ctx, s.refs, s.mass, b, 4, 60, s.pools(), s.kept) == 0
        s.same()


def test_an_eviction_beside_other_streams_attention():
    """Its CTAs meet although another stream's kernels keep the SMs busy; each call on a workspace of its own."""
    import torch

    inp = make([9000 + 100 * i for i in range(40)], 2, 10, 6000, seed=36)
    d = Dev(inp)
    ref, ref_lse = launch(d, 10, 6000)
    s = State([30000, 17000, 500], ("key_fp8", "lat_fp8"), seed=37)
    s.to_device()
    cuts = [[20000, 16999, 100], [12000, 8000, 99], [700, 7999, 0]]
    budgets = [torch.tensor(c, dtype=torch.int32, device="cuda") for c in cuts]
    start = torch.rand(inp.batch, inp.max_pages * 64, device="cuda")
    masses, ws = start.clone(), torch.zeros_like(d.ws)
    a, b, c = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for i in range(12):
        with torch.cuda.stream(a):
            outs.append(launch(d, 10, 6000)[0])
        dsa.attention_mass(d.p, d.q, d.lat_pool, 10, 6000, d.block_table, d.ctx, ref_lse, 0, masses, ws, c)
        if i % 4 == 1:
            s.call(budgets[i // 4], 4, 60, stream=b)
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    for w in (s.ws, d.ws, ws):
        assert dsa.get_device_error(w) == 0
    for _ in range(12):
        dsa.attention_mass(d.p, d.q, d.lat_pool, 10, 6000, d.block_table, d.ctx, ref_lse, 0, start, ws)
    assert torch.equal(masses, start)
    for cut in cuts:
        assert B.tokens_evict(s.table, s.ctx, s.refs, s.mass, cut, 4, 60, s.pools(), s.kept) == 0
    s.same()


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
def test_two_sums_of_weights_at_once(lat_fmt):
    import torch

    inp = make([5000, 900, 3100], 2, 10, 4000, seed=33, lat_fmt=lat_fmt)
    d = Dev(inp)
    _, lse = launch(d, 10, 4000)
    start = torch.rand(3, inp.max_pages * 64, device="cuda")
    call = lambda m, ws, stream=None: dsa.attention_mass(d.p, d.q, d.lat_pool, 10, 4000, d.block_table, d.ctx, lse, 2, m, ws, stream)
    ref = start.clone()
    for _ in range(4):
        call(ref, d.ws)
    masses, ws = [start.clone(), start.clone()], [torch.zeros_like(d.ws), torch.zeros_like(d.ws)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for m, w, s in zip(masses, ws, streams):
            call(m, w, s)
    torch.cuda.synchronize()
    assert all(torch.equal(m, ref) for m in masses)
    assert all(dsa.get_device_error(w) == 0 for w in ws)


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("sinks,window", [(3, 70), (0, 1 << 30)])
def test_weights_of_far_more_rows_than_tiles(lat_fmt, sinks, window):
    """One request's 333 rows on four tiles, beside one whose rows are all its tokens."""
    inp = make([400, 333], 333, sinks, window, seed=34, lat_fmt=lat_fmt)
    d = Dev(inp)
    _, lse = launch(d, sinks, window)
    check_mass(inp, sinks, window, *weights(inp, sinks, window, lse=lse.cpu().numpy(), d=d, fresh=333), fresh=333)
    assert dsa.get_device_error(d.ws) == 0


def test_fresh_tokens_that_no_row_sees_are_the_callers():
    """`fresh` sets what some row sees: a slot's new owner clears the rest, or the eviction ranks it by what lay there."""
    import torch

    sinks, window, n = 4, 60, 700
    inp = make([n], 2, sinks, window, seed=35, release=False)
    d = Dev(inp)
    _, lse = launch(d, sinks, window)
    left = np.full((1, inp.max_pages * 64), 5000, np.float32)  # the slot's last owner's
    got, _, ls = weights(inp, sinks, window, lse=lse.cpu().numpy(), start=left, d=d, fresh=n)
    check_mass(inp, sinks, window, got, left, ls, fresh=n)
    unseen = np.arange(sinks, n - 1 - window)
    assert (got[0, unseen] == 5000).all()
    cleared = np.zeros_like(left)
    got, _, _ = weights(inp, sinks, window, lse=lse.cpu().numpy(), start=cleared, d=d, fresh=n)
    mass = torch.from_numpy(got).cuda()
    table = torch.arange(inp.max_pages, dtype=torch.int32, device="cuda").view(1, -1)
    ctx, refs = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.ones(inp.num_pages, dtype=torch.int32, device="cuda")
    kept = torch.full(mass.shape, -1, dtype=torch.int32, device="cuda")
    dsa.tokens_evict(d.p, torch.tensor([30], dtype=torch.int32, device="cuda"), 0, 0, mass, dsa.make_token_pools([]), table, ctx, refs, kept,
                     d.ws)
    assert dsa.get_device_error(d.ws) == 0 and ctx.tolist() == [30]
    stay = kept[0, :30].cpu().numpy()
    assert stay.tolist() == B.chosen(got[0], n, 30, 0, 0) and not np.isin(stay, unseen).any()
