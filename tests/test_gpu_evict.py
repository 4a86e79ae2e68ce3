"""dsa_tokens_evict against the oracle: tables, counts, lengths, weights, kept tokens and every byte of the pools, exactly."""
import numpy as np
import pytest

import dsa_sparse_mla_paged_gb300 as dsa
from oracle import bounded as B

pytestmark = pytest.mark.gpu
FMT = {"key_fp8": 0, "key_mxfp4": 1, "lat_fp8": 2, "lat_nvfp4": 3}
PAGE_BYTES = {"key_fp8": 8448, "key_mxfp4": 4352, "lat_fp8": 36864, "lat_nvfp4": 22528}


@pytest.fixture(scope="module", autouse=True)
def _need(lib, cuda_ok):
    yield


class State:
    """Requests of the lengths `lens`, the first `shared` pages of the first `sharers` of them held together."""

    def __init__(self, lens, fmts=("key_fp8", "lat_fp8"), layers=1, outer=False, shared=0, sharers=0, spare=4, seed=0, ties=True,
                 width=None, pad=0):
        rng = np.random.default_rng(seed)
        self.batch, pages = len(lens), [-(-int(n) // 64) for n in lens]
        self.width = width or max(max(pages), 1)
        own = [p - (shared if b < sharers else 0) for b, p in enumerate(pages)]
        self.num_pages = shared + sum(own) + spare
        perm = rng.permutation(self.num_pages).astype(np.int32)
        self.table, self.refs = np.full((self.batch, self.width), -1, np.int32), np.zeros(self.num_pages, np.int32)
        at = shared
        for b, p in enumerate(pages):
            k = shared if b < sharers else 0
            self.table[b, :k], self.table[b, k:p] = perm[:k], perm[at:at + own[b]]
            at += own[b]
            np.add.at(self.refs, self.table[b, :p], 1)
        self.ctx = np.array(lens, np.int32)
        self.stride = self.width * 64 + 3
        m = rng.lognormal(0, 2, (self.batch, self.stride))
        if ties:
            m = np.where(rng.random(m.shape) < 0.6, np.floor(m), m)
        self.mass, self.kept = m.astype(np.float32), np.full((self.batch, self.stride), -7, np.int32)
        # pools: a page's layers side by side, or each layer's pages
        self.raw, self.plan, self.fmts = [], [], fmts
        for f in fmts:
            size = PAGE_BYTES[f] + pad
            shape = (layers, self.num_pages, size) if outer else (self.num_pages, layers, size)
            self.raw.append(rng.integers(0, 256, shape, dtype=np.uint8))
            self.plan.append((FMT[f], layers, self.num_pages * size if outer else size, size if outer else layers * size))
        self.outer = outer

    def pools(self):
        return [(f, [r[l] if self.outer else r[:, l] for l in range(r.shape[0 if self.outer else 1])]) for f, r in zip(self.fmts, self.raw)]

    def to_device(self):
        import torch

        t = lambda a: torch.from_numpy(a.copy()).cuda()
        self.d = {k: t(getattr(self, k)) for k in ("table", "ctx", "refs", "mass", "kept")}
        self.d_raw = [t(r) for r in self.raw]
        self.p = dsa.make_params(batch=self.batch, n_q=1, max_pages_per_req=self.width, num_pages=self.num_pages, key_page_stride=8448,
                                 lat_page_stride=36864, topk=1)
        self.ws = torch.full((dsa.workspace_size(self.p),), 0, dtype=torch.uint8, device="cuda")
        self.ws[256:] = 0xFF  # whatever another call left there
        self.d_pools = dsa.make_token_pools([(r, *plan) for r, plan in zip(self.d_raw, self.plan)])

    def call(self, budgets, sinks, recent, kept=True, stream=None):
        import torch

        b = budgets if isinstance(budgets, torch.Tensor) else torch.tensor(budgets, dtype=torch.int32, device="cuda")
        d = self.d
        dsa.tokens_evict(self.p, b, sinks, recent, d["mass"], self.d_pools, d["table"], d["ctx"], d["refs"], d["kept"] if kept else None,
                         self.ws, stream)

    def same(self):
        for k in ("ctx", "table", "refs", "kept"):
            got, ref = self.d[k].cpu().numpy(), getattr(self, k)
            assert (got == ref).all(), (k, np.argwhere(got != ref)[:5])
        assert (self.d["mass"].cpu().numpy().view(np.int32) == self.mass.view(np.int32)).all()
        for d, r in zip(self.d_raw, self.raw):
            got = d.cpu().numpy()
            assert (got == r).all(), np.argwhere(got != r)[:5]

    def check(self, budgets, sinks, recent, bits=0, device=True):
        if device:
            self.to_device()
        self.call(budgets, sinks, recent)
        err = dsa.get_device_error(self.ws)
        ref = B.tokens_evict(self.table, self.ctx, self.refs, self.mass, budgets, sinks, recent, self.pools(), self.kept)
        assert err == ref == bits, (err, ref)
        self.same()
        return self


@pytest.mark.parametrize("lens,budgets,sinks,recent", [
    ([1], [0], 0, 0), ([1], [1], 0, 0), ([2], [1], 0, 0), ([64], [63], 0, 0), ([65], [64], 1, 1), ([65, 64], [1, 0], 0, 0),
    ([200], [100], 0, 0), ([200], [100], 100, 0), ([200], [100], 0, 100), ([200], [100], 70, 70), ([200], [100], 1000, 5),
    ([200], [130], 64, 64), ([700, 0, 333, 64, 5], [300, 0, 332, 64, 4], 4, 30), ([700, 640, 333], [-1, 639, 500], 4, 30),
    ([1500, 1300, 4000], [700, 1299, 17], 3, 9)])
def test_matches_oracle(lens, budgets, sinks, recent):
    State(lens, seed=len(lens) + sinks).check(budgets, sinks, recent)


@pytest.mark.parametrize("outer", [False, True])
@pytest.mark.parametrize("fmts", [("key_fp8",), ("key_mxfp4", "lat_nvfp4"), ("lat_nvfp4", "key_fp8", "lat_fp8", "key_mxfp4"), ()])
def test_formats_and_layers(fmts, outer):
    State([500, 130, 900], fmts, 3, outer, seed=2, pad=32).check([200, 128, 899], 5, 40)


def test_pages_before_the_first_evicted_token_are_not_copied():
    """A shared prompt under the sinks stays shared; the shared page that changes is copied for each."""
    s = State([600, 500, 400, 300], shared=3, sharers=4, seed=3, spare=9)
    before = s.table[:, :2].copy()
    s.check([300, 200, 250, -1], 130, 20)
    assert (s.table[:, :2] == before).all() and s.refs[before[0]].tolist() == [4, 4]
    assert len(set(s.table[:, 2].tolist())) == 4


def test_every_holder_may_leave_a_shared_page():
    s = State([300, 300], shared=4, sharers=2, seed=4, spare=10)
    old = s.table[0, :4].copy()
    s.check([100, 90], 0, 0)
    assert (s.refs[old] == 0).all()


def test_fresh_pages_run_out():
    """The requests in order: the second does not fit, the third needs a page, too, and waits; the fourth needs none."""
    s = State([300, 320, 310, 200], shared=4, sharers=3, seed=5, spare=3)
    s.check([100, 200, 60, 90], 0, 0, bits=dsa.DSA_DEVERR_NO_PAGES)
    assert s.ctx.tolist() == [100, 320, 310, 90]


@pytest.mark.parametrize("spare", [0, 5, 40, 2000, 70001])
def test_fresh_pages_from_pools_of_any_size(spare):
    """The lowest free pages, wherever they lie, and none handed out twice."""
    s = State([700 + 3 * i for i in range(30)], ("key_mxfp4",), shared=9, sharers=20, seed=17, spare=spare)
    s.check([400 + i for i in range(30)], 3, 9, bits=0 if spare > 150 else dsa.DSA_DEVERR_NO_PAGES)
    live = np.concatenate([s.table[b, :-(-int(n) // 64)] for b, n in enumerate(s.ctx)])
    assert (np.bincount(live, minlength=s.num_pages) == s.refs).all()


def test_bad_requests_are_left_alone():
    s = State([300, 320, 310, 200, 100], seed=6, width=6)
    s.table[0, 2], s.refs[s.table[1, 4]] = s.num_pages, 0
    s.ctx[2], s.ctx[4] = 6 * 64 + 1, -5
    s.check([100, 100, 100, 100, 50], 3, 3, bits=dsa.DSA_DEVERR_CTX | dsa.DSA_DEVERR_BLOCK_TABLE | dsa.DSA_DEVERR_PAGES)
    assert s.ctx.tolist() == [300, 320, 385, 100, -5]


def test_weights_of_every_kind():
    """Ties, zeros of either sign, NaN, infinities, negative and subnormal weights."""
    s = State([900] * 9, seed=7)
    rng = np.random.default_rng(1)
    s.mass[0] = 0
    s.mass[1] = 1
    s.mass[2] = np.where(rng.random(s.stride) < 0.5, 0.0, -0.0)
    s.mass[3] = rng.choice([np.nan, np.inf, -np.inf, 0, -1, 1e-44, 1e-45, 3e38], s.stride)
    s.mass[4] = np.nan
    s.mass[5] = rng.standard_normal(s.stride)
    s.mass[6] = np.arange(s.stride)
    s.mass[7] = -np.arange(s.stride)
    s.mass[8] = np.float32(1) + np.arange(s.stride) * np.float32(2.0 ** -23)
    s.check([300, 301, 302, 450, 100, 299, 64, 65, 500], 4, 33)


def test_many_requests():
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 500, 1100).tolist()
    budgets = [int(rng.integers(-1, max(1, n + 20))) for n in lens]
    State(lens, ("key_mxfp4",), seed=8).check(budgets, 2, 5)


@pytest.mark.parametrize("batch,width", [(3, 5000), (40, 3000), (300, 700)])
def test_a_table_far_wider_than_its_contexts(batch, width):
    rng = np.random.default_rng(16)
    lens = rng.integers(1, 400, batch).tolist()
    lens[0] = 2500
    State(lens, ("key_mxfp4",), seed=16, width=width).check([n - 1 - n // 3 for n in lens], 3, 9)


def test_many_batches_of_moves():
    """More units than all CTAs gather at once, several times over, for one request and for several."""
    State([150000], seed=9).check([110000], 0, 100)
    State([30000, 41000, 29999], ("key_fp8", "lat_fp8"), 2, seed=10).check([20000, 12000, 29998], 16, 1000)


def test_a_long_context_is_chosen_from_exactly():
    State([1000001], ("key_mxfp4",), seed=11, ties=False).check([333333], 4, 1000)
    s = State([700001], ("key_mxfp4",), seed=12)
    s.mass[:] = np.random.default_rng(2).integers(0, 3, s.mass.shape)
    s.check([400000], 4, 1000)


def test_repeated_and_replayed():
    """The same state cut again and again, eager and as a graph with changing budgets."""
    import torch

    s = State([900, 800, 1000], shared=2, sharers=2, spare=12, seed=13)
    s.check([800, 790, 900], 3, 50)
    s.check([800, 790, 900], 3, 50, device=False)  # nothing left to do: kept is the identity
    budgets = torch.tensor([700, -1, 899], dtype=torch.int32, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.call(budgets, 3, 50)
    for new in ([700, -1, 899], [650, 100, 0], [-1, 99, 5]):
        budgets.copy_(torch.tensor(new, dtype=torch.int32))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        assert dsa.get_device_error(s.ws) == 0
        assert B.tokens_evict(s.table, s.ctx, s.refs, s.mass, new, 3, 50, s.pools(), s.kept) == 0
        s.same()


def test_without_kept_and_on_another_stream():
    import torch

    s = State([500, 400], seed=14)
    s.to_device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.call(torch.tensor([200, 300], dtype=torch.int32, device="cuda"), 3, 50, kept=False, stream=side)
    torch.cuda.synchronize()
    assert dsa.get_device_error(s.ws) == 0
    assert B.tokens_evict(s.table, s.ctx, s.refs, s.mass, [200, 300], 3, 50, s.pools()) == 0
    s.same()


def test_pages_beyond_four_gigabytes():
    import torch

    s = State([300, 200], ("lat_fp8",), seed=15)
    n, gap = s.num_pages, 1 << 30  # 5 pages a GB apart reach past 4 GB
    s.to_device()
    pool = torch.empty(9 << 30, dtype=torch.uint8, device="cuda")
    assert n * gap > 9 << 30 or n <= 9
    gap = (9 << 30) // n // 16 * 16
    view = pool.as_strided((n, PAGE_BYTES["lat_fp8"]), (gap, 1))
    view.copy_(s.d_raw[0][:, 0])
    s.d_pools = dsa.make_token_pools([(pool, FMT["lat_fp8"], 1, 0, gap)])
    s.call([100, 150], 3, 50)
    assert dsa.get_device_error(s.ws) == 0
    assert B.tokens_evict(s.table, s.ctx, s.refs, s.mass, [100, 150], 3, 50, s.pools(), s.kept) == 0
    s.d_raw[0][:, 0] = view
    s.same()
