"""dsa_prefix_mla_decode against the float64 oracle.

Bounds, derived from the arithmetic that include/dsa.h states:
- a logit is a sum of 576 products in fp32: at most 64 roundings of a partial
  sum no larger than bulk = scale * sum |q c|, 2^-23 of it each (a factor of two
  for accumulators that truncate), and 2^-22 for scaling: 66 * 2^-23 * bulk. With FP8
  latents the query is E4M3(x) + E5M2(x - E4M3(x)), x scaled so that the head's largest
  value is in [2^7, 2^8). x has 8 significant bits and E4M3 keeps the first 4 of them (rounded) down
  to 2^-6; the rest is then at most 8 units in x's last place, and 0..8 have at most three
  significant bits, as E5M2 has: exact. Below 2^-6 (2^-13 of a largest value of 2^7), E4M3 is a multiple of
  2^-9, the rest at most 2^-10, and E5M2 rounds it by at most 2^-3 of itself: 2^-13, or 2^-20 of the
  largest. So a query value under 2^-13 of its head's largest may be off by 2^-20 of
  that largest, and d adds scale * sum over those values of 2^-20 max |q| |c|;
- a weight exp(z) is off by a factor 1 + d, by 2^-21 in the exponential, and
  rounded to w. NVFP4 latents: fp16's 11 bits, w = 2^-11. FP8 latents: to fp16 (2^-11) and then to
  hi + lo, hi = E5M2(P) and lo = E4M3(P - hi), of P = 2^6 exp(z - m) with a running maximum m, raised
  when it is passed by a factor of 2^6 (so P <= 2^12). P in [2^e, 2^(e + 1)): hi has steps of 2^(e - 2),
  so |P - hi| <= 2^(e - 3) (at most 2^8; E4M3 ends at 448), which is 2^(e - 3) itself, exact in E4M3, or
  below it, where E4M3's half step is at most 2^(e - 4 - 4): 2^-8 of P. Where P - hi is under 2^-6, E4M3's
  half step is 2^-10. m is at most the row's final maximum, so that is at most 2^-16 of the row's largest
  weight: w = 2^-8 + 2^-11, and out adds 2^-16 (1 + 2^-10) * tail with tail = max p * sum |c|;
- the normaliser is off by d + 2^-21 and the rounding of its fp32 sum (it adds weights before they
  are rounded); splitting and merging adds a few 2^-22 on either;
- so lse is off by d + 2^-19 + 2^-22 |lse|, and out by (w + 2 d + 2^-18) * mass with
  mass = sum p |c|, plus the bf16 rounding, 2^-8 |out| (2^-133 among subnormals).
Nothing here is measured first."""
import numpy as np
import pytest

import dsa_sparse_mla_paged_gb300 as dsa
import gen
from oracle import serving as S

from dsa_testlib import Dev, bf16_to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need(lib, cuda_ok):
    yield


def make(batch, n_q, prefix, tails, seed=1, **kw):
    """Inputs whose requests share `prefix` tokens (request 0's pages; the other rows'
    entries there are left bad, as they are not read) and add `tails` of their own."""
    inp = gen.make_inputs(batch, n_q, [prefix + t for t in tails], seed=seed, bt_mode="permuted", **kw)
    inp.latent_scale = 0.75
    pages = inp.block_table[0, :prefix // 64].copy()
    inp.block_table[:, :prefix // 64] = 10 ** 8
    return inp, pages


def launch(d, pages, prefix, ws=None, stream=None, lse=True):
    import torch

    out = torch.full((d.rows, 96, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full((d.rows, 96), float("nan"), dtype=torch.float32, device="cuda") if lse else None
    pg = torch.from_numpy(pages).cuda() if prefix else None
    dsa.prefix_mla_decode(d.p, d.q, d.lat_pool, pg, prefix, d.block_table, d.ctx, out, ls, d.ws if ws is None else ws, stream)
    return out, ls


def check_row(inp, pages, prefix, b, t, out, lse):
    def off(q):
        top = np.abs(q).max(axis=1, keepdims=True)
        return np.where(np.abs(q) < 2.0 ** -13 * top, 2.0 ** -20 * top, 0.0) * (inp.lat_fmt == "fp8")

    ref, ref_lse, mass, bulk, extra, tail = S.prefix_mla(inp, pages, prefix, b, t, off)
    d = (66 * 2.0 ** -23 * bulk + extra)[:, None]
    w, floor = (2.0 ** -8 + 2.0 ** -11, 2.0 ** -16 + 2.0 ** -26) if inp.lat_fmt == "fp8" else (2.0 ** -11, 0.0)
    bound = (w + 2 * d + 2.0 ** -18) * mass + floor * tail + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
    err = np.abs(out.astype(np.float64) - ref)
    assert np.isfinite(out).all()
    assert (err <= bound).all(), f"({b}, {t}): {(err / bound).max():.2f} of the bound at {np.unravel_index((err / bound).argmax(), err.shape)}"
    if lse is not None:
        assert (np.abs(lse - ref_lse) <= d[:, 0] + 2.0 ** -19 + 2.0 ** -22 * np.abs(ref_lse)).all(), (b, t, np.abs(lse - ref_lse).max())


def check(inp, pages, prefix, rows=None, bits=0):
    d = Dev(inp)
    out, lse = launch(d, pages, prefix)
    assert dsa.get_device_error(d.ws) == bits
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for b in range(inp.batch):
        for t in range(inp.n_q):
            r = b * inp.n_q + t
            if rows is None or r in rows:
                check_row(inp, pages, prefix, b, t, o[r], l[r])
    return d, out, lse


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("batch,n_q,prefix,tails", [
    (1, 1, 0, [1]), (1, 1, 0, [63]), (1, 1, 64, [1]), (1, 1, 4096, [50]),
    (2, 1, 128, [64, 65]), (3, 1, 640, [1, 200, 129]), (4, 1, 1024, [3, 70, 500, 64]),
    (1, 4, 64, [4]), (2, 3, 192, [3, 67]), (2, 8, 0, [8, 700]), (5, 2, 2048, [2, 9, 66, 130, 1000]),
])
def test_matches_oracle(lat_fmt, batch, n_q, prefix, tails):
    inp, pages = make(batch, n_q, prefix, tails, seed=batch + prefix, lat_fmt=lat_fmt)
    check(inp, pages, prefix)


def test_long_prefix_and_many_rows():
    inp, pages = make(40, 1, 16384, [1 + 13 * i for i in range(40)], seed=5)
    check(inp, pages, 16384, rows={0, 1, 17, 38, 39})


def test_long_private_contexts():
    inp, pages = make(3, 2, 0, [9000, 2, 20001], seed=6)
    check(inp, pages, 0, rows={0, 2, 3, 5})


def test_more_rows_than_a_wave_of_jobs():
    inp, pages = make(150, 2, 128, [2 + i % 90 for i in range(150)], seed=7)
    check(inp, pages, 128, rows={0, 1, 99, 201, 298, 299})


@pytest.mark.parametrize("prefix", [0, 64])
def test_more_rows_than_threads_of_a_block(prefix):
    inp, pages = make(700, 2, prefix, [2 + (i * 7) % 200 for i in range(700)], seed=8)
    check(inp, pages, prefix, rows={0, 639, 640, 641, 1279, 1280, 1398, 1399})


def test_a_prompt_chunk():
    inp, pages = make(1, 130, 256, [200], seed=8)
    check(inp, pages, 256, rows={0, 64, 128, 129})


def test_page_strides_and_holes():
    inp, pages = make(2, 2, 320, [40, 300], seed=9, lat_page_pad=4096, holes=True)
    check(inp, pages, 320)


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
def test_nan_in_hidden_tokens_stays_out(lat_fmt):
    """NaN latents behind a context's end, and in a later new token that an earlier row must not see."""
    inp, pages = make(2, 3, 64, [70, 10], seed=10, lat_fmt=lat_fmt)
    size = 576 if lat_fmt == "fp8" else 352
    for b, c in enumerate(inp.ctx):
        page = inp.lat_pool[inp.block_table[b, (c - 1) // 64]]
        page[((c - 1) % 64) * size:] = 0x7F
    d = Dev(inp)
    out, lse = launch(d, pages, 64)
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for b in range(2):
        for t in range(2):  # the last row sees the token
            check_row(inp, pages, 64, b, t, o[b * 3 + t], l[b * 3 + t])


@pytest.mark.parametrize("exps", [(-100, -60), (-20, 20), (60, 90)])
def test_query_magnitudes(exps):
    """Queries far outside fp16's range (each head's own size), with logits kept moderate by one small
    scale per call: a head's largest value decides its scaling."""
    inp, pages = make(2, 1, 64, [30, 100], seed=11)
    rng = np.random.default_rng(0)
    e = rng.integers(exps[0], exps[1], (2, 1, 96, 1))
    q = rng.standard_normal((2, 1, 96, 576)) * 2.0 ** e
    inp.q = gen.f32_to_bf16_bits(q.astype(np.float32))
    inp.softmax_scale = 2.0 ** -(exps[1] + 3)
    check(inp, pages, 64)


def test_query_with_outliers_and_zeros():
    inp, pages = make(1, 1, 64, [90], seed=12)
    rng = np.random.default_rng(1)
    q = rng.standard_normal((1, 1, 96, 576)) * 2.0 ** rng.integers(-12, 1, (1, 1, 96, 576))
    q[0, 0, 5] = 0.0
    q[0, 0, 6, 3] = 700.0
    inp.q = gen.f32_to_bf16_bits(q.astype(np.float32))
    check(inp, pages, 64)


def test_sharp_and_rising_scores():
    """Scores that rise along the context (every tile raises the running maximum), fall along it, or have
    one token far above the others first, last or in between."""
    inp, pages = make(4, 1, 1024, [300, 300, 300, 300], seed=13)
    inp.softmax_scale = 1.0
    rng = np.random.default_rng(2)
    from oracle.formats import bf16_decode
    direction = np.sign(bf16_decode(inp.q[0, 0, 0]))
    q = rng.standard_normal((4, 1, 96, 576)) * 0.05 + direction * rng.choice([-0.06, 0.06], (4, 1, 96, 1))
    inp.q = gen.f32_to_bf16_bits(q.astype(np.float32))
    rows = inp.lat_pool.reshape(-1, 576)

    def put(page, slot, level):  # latent = direction * level, as E4M3 codes
        rows[page * 64 + slot] = gen.encode_e4m3(direction * level)

    for i, pg in enumerate(pages):
        for s in range(64):
            put(pg, s, 0.05 * i)
    for b, order in enumerate((1, -1, 0, 0)):
        for s in range(300):
            j = 1024 + s
            level = {1: 0.8 + s / 400, -1: 1.6 - s / 400, 0: 0.1}[order]
            put(inp.block_table[b, j // 64], j % 64, level)
    put(inp.block_table[2, 1024 // 64], 0, 4.0)
    put(inp.block_table[3, 1323 // 64], 1323 % 64, 4.0)
    check(inp, pages, 1024)


def test_a_heavy_first_token_and_a_long_light_rest():
    """One token outweighs each of 60,000 others by about e^12: the rest still holds a fair share of the mass."""
    inp, pages = make(1, 1, 60032, [20], seed=14)
    rng = np.random.default_rng(3)
    inp.softmax_scale = 1.0
    q = np.full((1, 1, 96, 576), 0.0)
    q[..., 0] = 1.5
    q[..., 1:] = rng.standard_normal((1, 1, 96, 575)) * 0.01
    inp.q = gen.f32_to_bf16_bits(q.astype(np.float32))
    rows = inp.lat_pool.reshape(-1, 576)
    rows[:, 0] = 0x80
    rows[pages[0] * 64, 0] = gen.encode_e4m3(np.array([11.0]))[0]
    check(inp, pages, 60032)


def test_bad_data_is_skipped_and_reported():
    import torch

    inp, pages = make(4, 2, 128, [90, 70, 2, 300], seed=15)
    good_ctx = inp.ctx.copy()
    inp.ctx[1] = 128 + 1                      # no room for its two new tokens
    inp.ctx[2] = inp.max_pages * 64 + 1
    d = Dev(inp)
    out, lse = launch(d, pages, 128)
    assert dsa.get_device_error(d.ws) == dsa.DSA_DEVERR_CTX
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for r in (2, 3, 4, 5):
        assert (o[r] == 0).all() and np.isneginf(l[r]).all()
    for b in (0, 3):
        for t in range(2):
            check_row(inp, pages, 128, b, t, o[b * 2 + t], l[b * 2 + t])
    # a bad prefix page and a bad page of a request: their tokens are left out
    inp.ctx[:] = good_ctx
    d = Dev(inp)
    bad = pages.copy()
    bad[1] = -1
    d.block_table[3, 3] = inp.num_pages
    out, lse = launch(d, bad, 128)
    assert dsa.get_device_error(d.ws) == dsa.DSA_DEVERR_BLOCK_TABLE
    o, l = bf16_to_np(out), lse.cpu().numpy()
    ref = S.O.sparse_mla
    inp.block_table[:, :2] = pages
    for b, t, keep in ((0, 0, list(range(64)) + list(range(128, 128 + 89))),
                       (3, 1, list(range(64)) + list(range(128, 192)) + list(range(256, 428)))):
        want, want_lse = ref(inp, b, t, np.array(keep))
        assert np.abs(l[b * 2 + t] - want_lse).max() < 1e-4
        assert np.abs(o[b * 2 + t] - want).max() < 2.0 ** -8 * np.abs(want).max() + 2.0 ** -9
    # a request whose every page is bad, without a prefix: nothing to attend to
    inp, pages = make(2, 1, 0, [64, 30], seed=16)
    d = Dev(inp)
    d.block_table[0, 0] = -1
    out, lse = launch(d, pages, 0)
    assert dsa.get_device_error(d.ws) == dsa.DSA_DEVERR_BLOCK_TABLE
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    check_row(inp, pages, 0, 1, 0, bf16_to_np(out)[1], lse.cpu().numpy()[1])


def test_without_lse_and_again():
    import torch

    inp, pages = make(6, 1, 512, [5, 60, 64, 200, 1, 33], seed=17)
    d, out, lse = check(inp, pages, 512)
    again, _ = launch(d, pages, 512, lse=False)
    assert torch.equal(again, out)


def test_agrees_with_sparse_attention_over_all_tokens():
    """The same step through dsa_sparse_mla_decode with every visible token in its list. Both bounds apply."""
    inp, pages = make(3, 2, 320, [100, 64, 700], seed=18)
    d, out, lse = check(inp, pages, 320)
    table = inp.block_table.copy()
    table[:, :5] = pages
    inp.block_table = table
    d2 = Dev(inp)
    import torch

    idx = torch.full((6, 2048), -1, dtype=torch.int32)
    for r in range(6):
        L = int(inp.ctx[r // 2]) - 2 + r % 2 + 1
        idx[r, :L] = torch.arange(L)
    o2, l2 = d2.mla(idx.cuda())
    assert (lse - l2).abs().max() < 1e-3
    assert (out.float() - o2.float()).abs().max() < 2e-2


def test_captured_graphs_share_a_workspace():
    import torch

    cases = []
    for seed, (prefix, tails) in enumerate([(512, [3, 100, 64]), (0, [300, 20, 65]), (1024, [1, 1, 200])]):
        inp, pages = make(3, 1, prefix, tails, seed=20 + seed)
        d = Dev(inp)
        cases.append((inp, pages, prefix, d))
    big = max((c[3].ws for c in cases), key=lambda w: w.numel())
    graphs = []
    for inp, pages, prefix, d in cases:
        pg = torch.from_numpy(pages).cuda() if prefix else None
        out = torch.empty(3, 96, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(3, 96, dtype=torch.float32, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dsa.prefix_mla_decode(d.p, d.q, d.lat_pool, pg, prefix, d.block_table, d.ctx, out, lse, big)
        graphs.append((g, out, lse, pg))
    for i in (0, 1, 2, 1, 0):
        g, out, lse, _ = graphs[i]
        inp, pages, prefix, d = cases[i]
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        o, l = bf16_to_np(out), lse.cpu().numpy()
        for b in range(3):
            check_row(inp, pages, prefix, b, 0, o[b], l[b])


def test_decode_after_it_on_the_same_workspace():
    """The fused step keeps its results when the prefix attention has used the same workspace."""
    import torch

    inp = gen.make_inputs(2, 2, [3000, 700], seed=30, bt_mode="permuted")
    d = Dev(inp)
    first = d.decode()
    again = d.decode()
    out, lse = launch(d, inp.block_table[0, :0], 0)
    after = d.decode()
    assert dsa.get_device_error(d.ws) == 0
    for x, y, z in zip(first, again, after):
        assert torch.equal(x, y) and torch.equal(x, z)
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for r in range(4):
        check_row(inp, inp.block_table[0, :0], 0, r // 2, r % 2, o[r], l[r])


def test_on_a_side_stream():
    import torch

    inp, pages = make(4, 1, 256, [5, 60, 64, 200], seed=31)
    d = Dev(inp)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out, lse = launch(d, pages, 256)
    st.synchronize()
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for b in range(4):
        check_row(inp, pages, 256, b, 0, o[b], l[b])


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
def test_pages_beyond_four_gigabytes(lat_fmt):
    """Pages 64 MB apart: offsets pass 32 bits within the pool."""
    import torch

    inp, pages = make(3, 2, 1024, [2, 600, 1500], seed=32, lat_fmt=lat_fmt)
    d = Dev(inp)
    far = 1 << 26
    assert inp.num_pages > 64
    pool = torch.empty(inp.num_pages * far, dtype=torch.uint8, device="cuda").view(-1, far)
    pool[:, :inp.lat_page_stride] = d.lat_pool
    d.lat_pool = pool
    d.p.lat_page_stride = far
    out, lse = launch(d, pages, 1024)
    assert dsa.get_device_error(d.ws) == 0
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for r in range(6):
        check_row(inp, pages, 1024, r // 2, r % 2, o[r], l[r])


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams, over one another, beside the fused decode."""
    import torch

    cases = [make(6, 2, 512, [2, 70, 400, 1300, 64, 9], seed=33), make(20, 1, 2048, [1 + 31 * i for i in range(20)], seed=34, lat_fmt="nvfp4")]
    devs = [Dev(inp) for inp, _ in cases]
    other = Dev(gen.make_inputs(2, 1, [5000, 300], seed=35))
    alone = [launch(d, pages, prefix) for d, (_, pages), prefix in zip(devs, cases, (512, 2048))]
    step = [x.clone() for x in other.decode()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got, steps = ([], []), []
    for _ in range(12):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(launch(devs[i], cases[i][1], (512, 2048)[i]))
        with torch.cuda.stream(streams[2]):
            steps.append([x.clone() for x in other.decode()])
    torch.cuda.synchronize()
    for i in range(2):
        assert dsa.get_device_error(devs[i].ws) == 0
        for out, lse in got[i]:
            assert torch.equal(out.view(torch.int16), alone[i][0].view(torch.int16)) and torch.equal(lse, alone[i][1])
    assert dsa.get_device_error(other.ws) == 0
    for s in steps:
        for x, y in zip(s, step):
            assert torch.equal(x, y)


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_queries_that_are_not_finite(lat_fmt, value):
    """Such a head is NaN (an infinite logit makes the softmax NaN), beside small and large other values;
    the other heads, in its tile and its row, are what they were."""
    inp, pages = make(3, 2, 192, [70, 3, 130], seed=36, lat_fmt=lat_fmt)
    d = Dev(inp)
    hit = [(0, 0, 3, 0), (0, 1, 95, 575), (2, 0, 31, 300), (2, 1, 64, 511)]
    for b, t, h, i in hit:
        d.q.view(3, 2, 96, 576)[b, t, h, i] = value
    d.q.view(3, 2, 96, 576)[2, 0, 31, 7] = 1e30
    out, lse = launch(d, pages, 192)
    assert dsa.get_device_error(d.ws) == 0
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for b, t, h, _ in hit:
        assert np.isnan(o[2 * b + t, h]).all() and np.isnan(l[2 * b + t, h]), (b, t, h)
        # the head's own values of the oracle stand in, so that the row's others can be checked as they are
        ref, ref_lse = S.prefix_mla(inp, pages, 192, b, t)[:2]
        o[2 * b + t, h], l[2 * b + t, h] = ref[h], ref_lse[h]
    for b in range(3):
        for t in range(2):
            check_row(inp, pages, 192, b, t, o[2 * b + t], l[2 * b + t])


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
def test_runs_of_forty_thousand_tiles(lat_fmt):
    """64 rows on 4 M shared tokens (64 pages, 1,024 times): waits that last for a pair's whole run do not give up.
    Against the distinct tokens with 1,024 times the weight; 8 products a tile are added to an output,
    each off by at most 2^-23 of it."""
    import torch

    from oracle.formats import bf16_decode

    n, times = 64, 1024
    inp, pages = make(64, 1, n * 64, [1] * 64, seed=37, lat_fmt=lat_fmt)
    own = inp.block_table[:, n].copy()
    prefix = n * 64 * times
    d = Dev(inp)
    p = dsa.make_params(batch=64, n_q=1, max_pages_per_req=n * times + 1, num_pages=inp.num_pages, key_page_stride=8448,
                        lat_page_stride=inp.lat_page_stride, lat_fmt=d.p.lat_fmt, softmax_scale=inp.softmax_scale,
                        latent_scale=inp.latent_scale, topk=1)
    ws = torch.zeros(dsa.workspace_size(p), dtype=torch.uint8, device="cuda")
    table = torch.zeros(64, n * times + 1, dtype=torch.int32, device="cuda")
    table[:, -1] = torch.from_numpy(own).cuda()
    ctx = torch.full((64,), prefix + 1, dtype=torch.int32, device="cuda")
    out = torch.empty(64, 96, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(64, 96, dtype=torch.float32, device="cuda")
    dsa.prefix_mla_decode(p, d.q, d.lat_pool, torch.from_numpy(np.tile(pages, times)).cuda(), prefix, table, ctx, out, lse, ws)
    assert dsa.get_device_error(ws) == 0
    o, l = bf16_to_np(out), lse.cpu().numpy()
    inp.block_table[:, :n] = pages
    adds = 8 * (48 * n * times / 76 + 64) * 2.0 ** -23
    for b in (0, 31, 63):
        c = S.O.dequant_latents(inp, b, np.arange(n * 64 + 1))
        q = bf16_decode(inp.q[b, 0])
        z = inp.softmax_scale * (q @ c.T) + np.log(np.append(np.full(n * 64, times), 1))
        top = z.max(axis=1, keepdims=True)
        want_lse = top[:, 0] + np.log(np.exp(z - top).sum(axis=1))
        w = np.exp(z - want_lse[:, None])
        want, mass = w @ c[:, :512], w @ np.abs(c[:, :512])
        bulk = inp.softmax_scale * (np.abs(q) @ np.abs(c).T).max(axis=1)
        dz = (66 * 2.0 ** -23 + 2.0 ** -20) * bulk
        assert (np.abs(l[b] - want_lse) <= dz + adds / 8 + 2.0 ** -19 + 2.0 ** -22 * np.abs(want_lse)).all()
        assert (np.abs(o[b] - want) <= (2.0 ** -7 + 2 * dz[:, None] + adds) * mass + 2.0 ** -8 * np.abs(want)).all()


def check_row_by_tiles(inp, pages, prefix, b, t, out, lse):
    """As check_row, with a bound that is relative to sum p |c| of each dim and says what a weight may lose tile by tile.
    A weight P = 2^(z - ref) is split as follows (FP8). Rows whose largest in the tile is at most 2^8: E4M3(P) is off by half a
    step, 2^(e - 4) for P in [2^e, 2^(e + 1)) or 2^-10 for P under 2^-6, and E5M2 of that by an eighth of it at most (half
    of a step of a quarter), or of a part of it: 2^-8 of P, or 2^-14. Rows above, up to 2^12: E5M2 first, 2^(e - 3), then E4M3: 2^-8
    of P, or 2^-10. ref is chosen so that a tile's largest is 2^2 or more in a segment's first tile, 2^-4 or more in every
    other, and a tile's largest above 2^12 brings itself to 2^8; and it is lowered where that is broken, except by more than
    2^40 in all. So what is not within 2^-8 (and 2^-11, from fp16) of a weight is within 2^-14 / 2^-4 (or 2^-10 / 2^8) of the
    largest in its tile and 2^-14 / 2^2 of the row's largest, or, past the limit, 2^-14 / 2^42 of it. NVFP4: fp16 leaves 2^-11, or
    2^-25 with a tile's largest at 2^-5 or more, and 2^7 or more in a segment's first. The fp32 sums: 8 products a tile,
    each off by at most 2^-23 of the sum so far, and sums are at most sum p |c|."""
    from oracle.formats import bf16_decode

    table = inp.block_table[b].copy()
    inp.block_table[b, :prefix // 64] = pages
    L = S.O.visible_len(inp.ctx[b], inp.n_q, t)
    c = S.O.dequant_latents(inp, b, np.arange(L))
    inp.block_table[b] = table
    q = bf16_decode(inp.q[b, t])
    z = inp.softmax_scale * (q @ c.T)
    top = z.max(axis=1, keepdims=True)
    want_lse = top[:, 0] + np.log(np.exp(z - top).sum(axis=1))
    p, size = np.exp(z - want_lse[:, None]), np.abs(c[:, :512])
    want, mass = p @ c[:, :512], p @ size
    starts = np.arange(0, L, 64)
    peak, tiles = np.maximum.reduceat(p, starts, axis=1), np.add.reduceat(size, starts, axis=0)
    low, far, w = (2.0 ** -10, 2.0 ** -16, 2.0 ** -8 + 2.0 ** -11) if inp.lat_fmt == "fp8" else (2.0 ** -20, 2.0 ** -32, 2.0 ** -11)
    lost = np.minimum(low * peak, far * p.max(axis=1, keepdims=True)) @ tiles + 2.0 ** -56 * p.max(axis=1, keepdims=True) * size.sum(axis=0)
    dz = (66 * 2.0 ** -23 * inp.softmax_scale * (np.abs(q) @ np.abs(c).T).max(axis=1))[:, None]
    if inp.lat_fmt == "fp8":  # query values far below their head's largest
        big = np.abs(q).max(axis=1, keepdims=True)
        dz += inp.softmax_scale * (np.where(np.abs(q) < 2.0 ** -13 * big, 2.0 ** -20 * big, 0.0) @ np.abs(c).T).max(axis=1)[:, None]
    adds = 8 * len(starts) * 2.0 ** -23
    bound = (w + 2 * dz + adds + 2.0 ** -18) * mass + (1 + 2.0 ** -6) * lost + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    err = np.abs(out.astype(np.float64) - want)
    assert np.isfinite(out).all()
    assert (err <= bound).all(), f"({b}, {t}): {(err / bound).max():.2f} of the bound at {np.unravel_index((err / bound).argmax(), err.shape)}, err/mass {(err / mass).max():.2e}"
    assert (np.abs(lse - want_lse) <= dz[:, 0] + adds / 8 + 2.0 ** -19 + 2.0 ** -22 * np.abs(want_lse)).all()


def put_tokens(inp, pages_of_tokens, slots, level, rows=None):
    """Latents whose dim 575 (of the logits alone) is `level`, all other values zero, or left as they are with rows."""
    size = 576 if inp.lat_fmt == "fp8" else 352
    pool = inp.lat_pool.reshape(-1, inp.lat_page_stride)[:, :64 * size].reshape(-1, 64, size)
    level = np.broadcast_to(np.asarray(level, np.float64), np.shape(slots))
    for pg, s, v in zip(np.ravel(pages_of_tokens), np.ravel(slots), np.ravel(level)):
        row = pool[pg, s]
        if rows is None:
            row[:] = 0
        row[size - 1] = gen.encode_e4m3(np.array([v]))[0]


def plain_light(inp, rng, equal):
    """Every latent: dim 575 zero; equal: the same values for all tokens."""
    size = 576 if inp.lat_fmt == "fp8" else 352
    pool = inp.lat_pool.reshape(-1, inp.lat_page_stride)[:, :64 * size].reshape(-1, size)
    assert np.shares_memory(pool, inp.lat_pool)
    if equal:
        pool[:] = pool[int(rng.integers(len(pool)))]
    pool[:, size - 1] = 0


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("equal", [True, False])
@pytest.mark.parametrize("gap", [3, 5, 8, 11, 14, 18, 30, 60])
def test_a_heavy_first_token_whose_own_values_are_zero(lat_fmt, equal, gap):
    """Attention sinks: one token outweighs each of 16,000 others by e^gap to e^(1.75 gap) (by head), and adds nothing to the
    output, which is the others' sum. Many rows, so that it shares its segment with thousands of them."""
    inp, pages = make(40, 1, 16384, [1 + 5 * i for i in range(40)], seed=60 + gap, lat_fmt=lat_fmt)
    rng = np.random.default_rng(gap)
    plain_light(inp, rng, equal)
    put_tokens(inp, pages[:1], [0], 2.0 * gap)
    inp.softmax_scale = 0.5
    q = np.zeros((40, 1, 96, 576)) if equal else rng.standard_normal((40, 1, 96, 576)) * 2.0 / 24
    q[..., 575] = 1 + np.arange(96) / 128
    inp.q = gen.f32_to_bf16_bits(q.astype(np.float32))
    d = Dev(inp)
    out, lse = launch(d, pages, 16384)
    assert dsa.get_device_error(d.ws) == 0
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for b in (0, 7, 39):
        check_row_by_tiles(inp, pages, 16384, b, 0, o[b], l[b])


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("every", [1, 40, 64, 333])
def test_heavy_tokens_here_and_there(lat_fmt, every):
    """Heavy tokens without values of their own, of random heights, again and again along each row's own tokens: the
    weights' reference goes up and down."""
    inp, pages = make(3, 2, 64, [700, 5000, 1300], seed=80 + every, lat_fmt=lat_fmt)
    rng = np.random.default_rng(every)
    plain_light(inp, rng, False)
    inp.softmax_scale = 0.5
    for b in range(3):
        at = np.arange(64, int(inp.ctx[b]))[::every]
        put_tokens(inp, inp.block_table[b, at // 64], at % 64, rng.uniform(0, 60, len(at)), rows=True if every == 1 else None)
    q = rng.standard_normal((3, 2, 96, 576)) / 24
    q[..., 575] = 1 + np.arange(96) / 128
    inp.q = gen.f32_to_bf16_bits(q.astype(np.float32))
    d = Dev(inp)
    out, lse = launch(d, pages, 64)
    assert dsa.get_device_error(d.ws) == 0
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for b in range(3):
        for t in range(2):
            check_row_by_tiles(inp, pages, 64, b, t, o[2 * b + t], l[2 * b + t])


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("step", [-30.0, -4.0, -0.7, 0.7, 4.0, 30.0])
def test_stairs(lat_fmt, step):
    """Logits that fall or rise by `step` nats from tile to tile, over up to 800: through every threshold, and past the
    limit of how far the reference is lowered; then one more tile as at the start."""
    inp, pages = make(2, 1, 64 * 26, [64, 130], seed=90, lat_fmt=lat_fmt)
    rng = np.random.default_rng(1)
    plain_light(inp, rng, False)
    inp.softmax_scale = 1.0
    levels = step * (np.arange(26) - 13)
    levels[-1] = levels[0]
    for pg, v in zip(pages, levels):
        put_tokens(inp, np.full(64, pg), np.arange(64), v, rows=True)
    q = rng.standard_normal((2, 1, 96, 576)) / 24
    q[..., 575] = 1.0
    inp.q = gen.f32_to_bf16_bits(q.astype(np.float32))
    d = Dev(inp)
    out, lse = launch(d, pages, 64 * 26)
    assert dsa.get_device_error(d.ws) == 0
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for b in range(2):
        check_row_by_tiles(inp, pages, 64 * 26, b, 0, o[b], l[b])
