"""The page operations on the GPU against the oracle, one request and one page at
a time: tables, lengths, counts, page contents and error bits, all exact."""
import numpy as np
import pytest

import dsa_sparse_mla_paged_gb300 as dsa
from oracle import serving as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need(lib, cuda_ok):
    yield


class State:
    """A random consistent state: requests of the given lengths, the first `shared`
    tokens held by all (their open page too, where a request ends in it)."""

    def __init__(self, lens, shared=0, num_pages=None, width=None, pools=((64, 64),), seed=0, spare=9):
        rng = np.random.default_rng(seed)
        whole, need = shared // 64, shared // 64 + (shared % 64 != 0)
        counts = [need if n == shared else whole + S.pages_of(n) - whole for n in lens]
        total = need + sum(max(0, S.pages_of(n) - whole) for n in lens if n != shared)
        self.num_pages = num_pages or total + spare
        self.width = width or max(counts) + 4
        perm = rng.permutation(self.num_pages).astype(np.int32)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = need
        for b, n in enumerate(lens):
            k = min(need, S.pages_of(n)) if n == shared else min(whole, S.pages_of(n))
            self.table[b, :k] = perm[:k]
            rest = S.pages_of(n) - k
            self.table[b, k:k + rest] = perm[at:at + rest]
            at += rest
        self.ctx = np.array(lens, np.int32)
        self.refs = np.zeros(self.num_pages, np.int32)
        for b, n in enumerate(lens):
            np.add.at(self.refs, self.table[b, :S.pages_of(n)], 1)
        self.pools = [rng.integers(0, 256, (self.num_pages, stride), dtype=np.uint8) for _, stride in pools]
        self.sizes = [size for size, _ in pools]

    def params(self):
        return dsa.make_params(batch=len(self.ctx), n_q=1, max_pages_per_req=self.width, num_pages=self.num_pages,
                               key_page_stride=8448, lat_page_stride=36864)

    def upload(self):
        import torch

        t = lambda a: torch.from_numpy(a.copy()).cuda()
        self.p = self.params()
        self.d = dict(table=t(self.table), ctx=t(self.ctx), refs=t(self.refs), pools=[t(x) for x in self.pools])
        self.ws = torch.zeros(dsa.workspace_size(self.p), dtype=torch.uint8, device="cuda")
        self.plan = dsa.make_pools([(x, n, x.shape[1]) for x, n in zip(self.d["pools"], self.sizes)])
        return self

    def views(self):
        """The pools as the oracle copies them: the page bytes, not what lies between pages."""
        return [x[:, :n] for x, n in zip(self.pools, self.sizes)]

    def check(self, bits=0):
        import torch

        torch.cuda.synchronize()
        assert dsa.get_device_error(self.ws) == bits
        for name in ("table", "ctx", "refs"):
            assert np.array_equal(self.d[name].cpu().numpy(), getattr(self, name)), name
        for i, (x, y) in enumerate(zip(self.d["pools"], self.pools)):
            assert np.array_equal(x.cpu().numpy(), y), f"pool {i}"


def _dev(a):
    import torch

    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def _resize(s, new):
    dsa.pages_resize(s.p, _dev(new), s.plan, s.d["table"], s.d["ctx"], s.d["refs"], s.ws)
    s.check(S.pages_resize(s.table, s.ctx, s.refs, list(new), s.views()))


def _fork(s, src, dst):
    dsa.pages_fork(s.p, _dev(src), _dev(dst), s.d["table"], s.d["ctx"], s.d["refs"], s.ws)
    s.check(S.pages_fork(s.table, s.ctx, s.refs, src, dst))


def _compact(s, outputs=True):
    import torch

    m = torch.full((s.num_pages,), -7, dtype=torch.int32, device="cuda") if outputs else None
    n = torch.full((1,), -7, dtype=torch.int32, device="cuda") if outputs else None
    dsa.pages_compact(s.p, s.plan, s.d["table"], s.d["ctx"], s.d["refs"], m, n, s.ws)
    where, live, bits = S.pages_compact(s.table, s.ctx, s.refs, s.views())
    s.check(bits)
    if outputs:
        assert np.array_equal(m.cpu().numpy(), where) and n.item() == live


POOLS = ((8448, 8448), (36864, 36864 + 48), (16, 32))


@pytest.mark.parametrize("lens,new,shared", [
    ([0], [1], 0), ([0], [0], 0), ([1], [0], 0), ([64], [65], 0), ([64], [64], 0), ([63], [64], 0), ([65], [64], 0),
    ([100, 100, 100], [101, 128, 129], 100),        # every holder of the open page grows: each gets a copy
    ([100, 100, 40], [130, -1, 0], 100),            # one grows, one stays, one (that holds none of it) ends
    ([128, 128], [129, 200], 128),                  # a full last page is shared, not copied
    ([300, 10, 0, 200, 64], [0, 500, 64, 130, -1], 0),
])
def test_resize(lens, new, shared):
    s = State(lens, shared, pools=POOLS, seed=len(lens) + shared, spare=30, width=10).upload()
    _resize(s, new)


@pytest.mark.parametrize("seed", range(3))
def test_resize_many_requests_over_several_plan_blocks(seed):
    rng = np.random.default_rng(100 + seed)
    lens = rng.integers(0, 400, 1500)
    lens[rng.random(1500) < 0.3] = 90
    s = State([int(x) for x in lens], 90 if seed else 0, pools=((32, 32),), seed=seed, spare=[20000, 2500, 300][seed], width=12).upload()
    new = np.where(rng.random(1500) < 0.2, -1, rng.integers(0, 700, 1500))
    _resize(s, [int(x) for x in new])               # seeds 1 and 2 run out of pages


def test_resize_exact_fit_and_one_page_short():
    s = State([64, 64], pools=POOLS, num_pages=4).upload()
    _resize(s, [128, 128])
    s = State([64, 64, 0], pools=POOLS, num_pages=4).upload()
    _resize(s, [128, 129, 0])
    s = State([64, 64, 64], pools=POOLS, num_pages=4).upload()
    _resize(s, [192, 128, 64])                      # the first does not fit: nobody after it is served


def test_resize_bad_state_and_arguments():
    s = State([100, 100, 200, 64, 10], pools=POOLS, spare=20, width=6)
    s.table[0, 1] = -1                              # the open page is a bad entry
    s.table[2, 3] = 10 ** 6                         # a bad entry that is released
    s.refs[s.table[3, 0]] = 0                       # held by nobody: the count stays at 0
    s.ctx[4] = 6 * 64 + 1                           # longer than a row
    s.upload()
    new = [101, 6 * 64 + 1, 100, 0, 0]
    dsa.pages_resize(s.p, _dev(new), s.plan, s.d["table"], s.d["ctx"], s.d["refs"], s.ws)
    bits = S.pages_resize(s.table, s.ctx, s.refs, new, s.views())
    assert bits == S.ERR_BLOCK_TABLE | S.ERR_CTX | S.ERR_PAGES
    s.check(bits)


def test_resize_leaves_pages_without_references_alone():
    s = State([100, 64, 64], pools=POOLS, spare=5)
    s.refs[s.table[0, 1]] = 0                       # an open page that is free: nothing is appended to it
    s.upload()
    _resize(s, [101, 65, 0])
    assert s.ctx.tolist() == [100, 65, 0]
    for lens, new in (([64, 100], [65, 0]), ([100, 64], [0, 65])):
        s = State(lens, pools=POOLS, num_pages=3)
        s.refs[s.table[lens.index(100), 1]] = -2    # released, and handed out by the same call
        s.upload()
        _resize(s, new)
        assert sorted(s.refs.tolist()) == [0, 1, 1]


def test_resize_without_pools_and_with_negative_length():
    s = State([100, 70], 64, pools=(), spare=10).upload()
    _resize(s, [200, 0])
    s = State([100, 70], 64, pools=(), spare=10)
    s.ctx[0] = -5
    s.upload()
    _resize(s, [200, 0])


@pytest.mark.parametrize("src,dst", [([0], [1]), ([0, 0, 0], [1, 3, 4]), ([2, 0], [1, 3]), ([1], [3])])
def test_fork(src, dst):
    s = State([130, 0, 64, 0, 0], pools=POOLS, spare=20).upload()
    _fork(s, src, dst)
    _resize(s, [140, 150, -1, 160, 0])


def test_fork_refusals():
    s = State([130, 0, 64, 0, 0, 0], pools=POOLS, spare=20).upload()
    # out of the batch, onto itself, onto a held slot, a destination named before, from a slot that is filled in this call
    _fork(s, [0, 9, 2, 0, 2, 1], [1, 3, 2, 0, 1, 4])
    _fork(s, [-1, 0], [5, -1])
    s = State([130, 0], pools=POOLS, spare=20)
    s.ctx[0] = 10 ** 6
    s.upload()
    _fork(s, [0], [1])
    s = State([130, 0], pools=POOLS, spare=20)
    s.table[0, 1] = s.num_pages
    s.upload()
    _fork(s, [0], [1])


def test_fork_wide_rows_and_many_pairs():
    s = State([64 * 700 + 5] + [0] * 1100, pools=((16, 16),), spare=5, width=1000).upload()
    _fork(s, [0] * 1100, list(range(1100, 0, -1)))


@pytest.mark.parametrize("num_pages", [None, 40, 4096 + 3, 20011])
def test_compact(num_pages):
    s = State([300, 100, 0, 64, 100], 100, pools=POOLS if num_pages != 20011 else ((16, 16),), num_pages=num_pages, seed=7).upload()
    _compact(s)
    _compact(s, outputs=False)                      # nothing left to move


def test_compact_full_empty_and_held_pages():
    s = State([256, 256], pools=POOLS, num_pages=8).upload()
    _compact(s)
    s = State([0, 0], pools=POOLS, num_pages=7).upload()
    _compact(s)
    s = State([100, 64], pools=POOLS, num_pages=30, seed=1)
    s.refs[29] += 3                                 # a page that only the caller holds
    s.upload()
    _compact(s)


def test_compact_bad_state():
    s = State([100, 200, 64, 70], pools=POOLS, num_pages=30, seed=5)
    s.table[0, 0] = -1
    s.table[1, 2] = 30
    s.refs[s.table[2, 0]] = 0
    s.ctx[3] = -1
    s.upload()
    _compact(s)


def test_random_life_of_a_cache():
    """Rounds of fork, growth, trimming and packing; the workspace is reused throughout."""
    rng = np.random.default_rng(9)
    s = State([500, 90, 0, 0, 0, 0, 0, 0], pools=((48, 64), (112, 112)), num_pages=90, width=16).upload()
    for step in range(25):
        empty = [b for b in range(8) if s.ctx[b] == 0]
        if empty and step % 3 == 0:
            k = int(rng.integers(1, len(empty) + 1))
            _fork(s, [int(x) for x in rng.integers(0, 8, k)], empty[:k])
        new = [int(min(16 * 64, max(0, n + rng.integers(-100, 130)))) if rng.random() < 0.8 else -1 for n in s.ctx]
        _resize(s, new)
        if step % 4 == 3:
            _compact(s)


def test_captured_and_replayed_on_another_stream():
    import torch

    s = State([500, 90, 0, 0], pools=POOLS, num_pages=60, width=12).upload()
    new = _dev([510, 91, 505, 0])
    src, dst = _dev([0]), _dev([2])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def step():
        dsa.pages_fork(s.p, src, dst, s.d["table"], s.d["ctx"], s.d["refs"], s.ws)
        dsa.pages_resize(s.p, new, s.plan, s.d["table"], s.d["ctx"], s.d["refs"], s.ws)
        dsa.pages_compact(s.p, s.plan, s.d["table"], s.d["ctx"], s.d["refs"], None, None, s.ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        step()
    torch.cuda.synchronize()
    bits = 0
    for _ in range(2):  # the second replay finds the slots taken: the fork is refused
        g.replay()
        bits |= S.pages_fork(s.table, s.ctx, s.refs, [0], [2])
        bits |= S.pages_resize(s.table, s.ctx, s.refs, [510, 91, 505, 0], s.views())
        bits |= S.pages_compact(s.table, s.ctx, s.refs, s.views())[2]
    assert bits == S.ERR_PAGES
    s.check(bits)


def test_pages_beyond_four_gigabytes():
    """A pool whose pages lie 96 MB apart (offsets pass 32 bits): copied on write, then packed."""
    import torch

    s = State([500, 90, 4000, 0], shared=0, pools=((4096, 4096),), num_pages=90, width=70).upload()
    far = 96 << 20
    pool = torch.empty(90 * far, dtype=torch.uint8, device="cuda").view(90, far)
    pool[:, :4096] = s.d["pools"][0]
    s.plan = dsa.make_pools([(pool, 4096, far)])
    dsa.pages_fork(s.p, _dev([0]), _dev([3]), s.d["table"], s.d["ctx"], s.d["refs"], s.ws)
    dsa.pages_resize(s.p, _dev([510, 0, 4001, 501]), s.plan, s.d["table"], s.d["ctx"], s.d["refs"], s.ws)
    dsa.pages_compact(s.p, s.plan, s.d["table"], s.d["ctx"], s.d["refs"], None, None, s.ws)
    views = s.views()
    assert S.pages_fork(s.table, s.ctx, s.refs, [0], [3]) == 0
    assert S.pages_resize(s.table, s.ctx, s.refs, [510, 0, 4001, 501], views) == 0
    live = S.pages_compact(s.table, s.ctx, s.refs, views)[1]
    assert dsa.get_device_error(s.ws) == 0
    assert np.array_equal(s.d["table"].cpu().numpy(), s.table) and np.array_equal(s.d["refs"].cpu().numpy(), s.refs)
    held = [s.table[b, j] for b in range(4) for j in range(S.pages_of(int(s.ctx[b])))]
    assert max(held) < live
    whole = [s.table[b, j] for b in range(4) for j in range(int(s.ctx[b]) // 64)]  # the rest may be unspecified
    assert np.array_equal(pool[:, :4096].cpu().numpy()[whole], views[0][whole])
