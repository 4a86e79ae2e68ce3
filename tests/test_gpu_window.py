"""dsa_window_mla_decode against the float64 oracle, within the bounds that tests/test_gpu_prefix.py derives (the
arithmetic is that call's), and dsa_attention_mass within the bound that oracle/bounded.py states."""
import numpy as np
import pytest

import dsa_sparse_mla_paged_gb300 as dsa
import gen
from oracle import bounded as B

from dsa_testlib import Dev, bf16_to_np

pytestmark = pytest.mark.gpu
ALL = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _need(lib, cuda_ok):
    yield


def make(lens, n_q, sinks, window, seed=1, release=True, **kw):
    """Inputs whose pages that no row sees are released: their entries are -1, or out of range."""
    inp = gen.make_inputs(len(lens), n_q, list(lens), seed=seed, bt_mode="permuted", **kw)
    inp.latent_scale = 0.75
    if release:
        for b, n in enumerate(lens):
            first = max(0, n - n_q + 1 - window)
            for j in range(-(-n // 64)):
                if j * 64 >= sinks and (j + 1) * 64 <= first:
                    inp.block_table[b, j] = -1 if j % 2 else 10 ** 8
    return inp


def off(inp):
    """How far each query value may be off (tests/test_gpu_prefix.py)."""
    def f(q):
        top = np.abs(q).max(axis=1, keepdims=True)
        return np.where(np.abs(q) < 2.0 ** -13 * top, 2.0 ** -20 * top, 0.0) * (inp.lat_fmt == "fp8")
    return f


def launch(d, sinks, window, ws=None, stream=None, lse=True):
    import torch

    out = torch.full((d.rows, 96, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full((d.rows, 96), float("nan"), dtype=torch.float32, device="cuda") if lse else None
    dsa.window_mla_decode(d.p, d.q, d.lat_pool, sinks, window, d.block_table, d.ctx, out, ls, d.ws if ws is None else ws, stream)
    return out, ls


def check_row(inp, sinks, window, b, t, out, lse=None):
    ref, ref_lse, mass, bulk, extra, tail = B.window_mla(inp, sinks, window, b, t, off(inp))
    d = (66 * 2.0 ** -23 * bulk + extra)[:, None]
    w, floor = (2.0 ** -8 + 2.0 ** -11, 2.0 ** -16 + 2.0 ** -26) if inp.lat_fmt == "fp8" else (2.0 ** -11, 0.0)
    bound = (w + 2 * d + 2.0 ** -18) * mass + floor * tail + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
    err = np.abs(out.astype(np.float64) - ref)
    assert np.isfinite(out).all()
    assert (err <= bound).all(), f"({b}, {t}): {(err / bound).max():.2f} of the bound at {np.unravel_index((err / bound).argmax(), err.shape)}"
    if lse is not None:
        assert (np.abs(lse - ref_lse) <= d[:, 0] + 2.0 ** -19 + 2.0 ** -22 * np.abs(ref_lse)).all(), (b, t, np.abs(lse - ref_lse).max())


def check(inp, sinks, window, rows=None, bits=0):
    d = Dev(inp)
    out, lse = launch(d, sinks, window)
    assert dsa.get_device_error(d.ws) == bits
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for b in range(inp.batch):
        for t in range(inp.n_q):
            r = b * inp.n_q + t
            if rows is None or r in rows:
                check_row(inp, sinks, window, b, t, o[r], l[r])
    return d, out, lse


CASES = [  # lens, n_q, sinks, window
    ([1], 1, 0, 1), ([1], 1, 5, 1), ([64], 1, 0, 64), ([65], 1, 0, 64), ([129], 1, 1, 64), ([200], 1, 64, 64), ([200], 1, 65, 1),
    ([500, 64, 3], 1, 4, 100), ([700, 130], 3, 0, 65), ([300, 260], 4, 130, 63), ([1000, 9], 8, 2, 700), ([777, 500], 2, 63, 2),
    ([130], 1, 60, 66), ([130], 1, 60, 67), ([191, 190], 1, 100, 40), ([400, 300], 2, ALL, 1), ([400, 300], 2, 0, ALL),
    ([90], 5, 20, 3), ([70], 6, 66, 2), ([300, 131], 7, 64, 61), ([200], 13, 0, 1), ([160, 70, 65], 4, 70, 5), ([2100, 40, 900, 1500], 1, 128, 1024)]


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("lens,n_q,sinks,window", CASES)
def test_matches_oracle(lat_fmt, lens, n_q, sinks, window):
    check(make(lens, n_q, sinks, window, seed=len(lens) + n_q, lat_fmt=lat_fmt), sinks, window)


@pytest.mark.parametrize("sinks,window", [(0, 2 ** 31 - 1), (2 ** 31 - 1, 1), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_the_largest_counts(sinks, window):
    """More than there can be, in tiles that lie behind a job's first rows: all tokens up to the row's own."""
    inp = make([200, 331], 150, sinks, window, seed=8)
    check(inp, sinks, window, rows={0, 1, 70, 149, 150, 223, 299})


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
def test_a_prompt_chunk(lat_fmt):
    inp = make([900, 150], 140, 10, 200, seed=3, lat_fmt=lat_fmt)
    check(inp, 10, 200, rows={0, 1, 70, 139, 140, 200, 279})


def test_long_contexts_and_many_rows():
    inp = make([30000 + 17 * i for i in range(90)], 2, 70, 500, seed=4)
    check(inp, 70, 500, rows={0, 1, 64, 101, 178, 179})


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("lens,n_q", [([200 + i for i in range(76)], 1), ([300] * 100, 1), ([900] * 24, 4), ([130] * 200, 3), ([64, 5000], 2)])
def test_many_jobs(lat_fmt, lens, n_q):
    """As many jobs as CTA pairs, or several times as many, or one that dwarfs the other, with empty requests and bad pages among
    them; the same call gives the same bits."""
    import torch

    inp = make(lens, n_q, 70, 120, seed=30 + n_q, lat_fmt=lat_fmt, release=False)
    inp.ctx = inp.ctx.copy()
    rows = {r for b in (1, len(lens) // 2, len(lens) - 1) for r in range(b * n_q, (b + 1) * n_q)}
    bits = 0
    if len(lens) > 2:
        inp.ctx[0] = 0  # no job
        inp.block_table[len(lens) - 1, 0] = -1
        bits = dsa.DSA_DEVERR_CTX | dsa.DSA_DEVERR_BLOCK_TABLE
    d, out, lse = check(inp, 70, 120, rows=rows, bits=bits)
    if len(lens) > 2:
        assert (out[:n_q] == 0).all() and (lse[:n_q] == -np.inf).all()
    again, _ = launch(d, 70, 120, lse=False)
    assert (again.view(torch.int16) == out.view(torch.int16)).all()
    assert dsa.get_device_error(d.ws) == bits


def test_a_wide_window_is_the_dense_call():
    """The same bits for single rows (rows of a request share jobs here, and not there)."""
    import torch

    inp = make([700, 64, 333], 1, 0, ALL, seed=5)
    d, out, lse = check(inp, 0, ALL)
    ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
    dsa.prefix_mla_decode(d.p, d.q, d.lat_pool, None, 0, d.block_table, d.ctx, ref, ref_lse, d.ws)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    out, _ = launch(d, 300, 400, lse=False)  # the parts meet
    assert torch.equal(out, ref)


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
def test_nan_in_hidden_tokens_stays_out(lat_fmt):
    """NaN latents between sinks and window, inside the pages that both read, behind the end, and in a later row's tokens."""
    sinks, window, size = 70, 100, 576 if lat_fmt == "fp8" else 352
    inp = make([400, 171], 3, sinks, window, seed=6, lat_fmt=lat_fmt, release=False)
    rows = inp.lat_pool.reshape(-1, size)
    for b, n in enumerate(inp.ctx):
        first = n - 2 - window  # of the first row
        for s in list(range(sinks, first)) + list(range(n, -(-n // 64) * 64)):
            rows[inp.block_table[b, s // 64] * 64 + s % 64] = 0x7F
    check(inp, sinks, window)
    planted = [(n - 1, n - 2 - window) for n in inp.ctx]  # the last token, the first row's oldest
    for b in range(2):
        for s in planted[b]:
            rows[inp.block_table[b, s // 64] * 64 + s % 64] = 0x7F
    d = Dev(inp)
    out, lse = launch(d, sinks, window)
    o, l = bf16_to_np(out), lse.cpu().numpy()
    clean = 0
    for b in range(2):
        for t in range(3):
            if set(planted[b]) & set(B.visible(inp.ctx[b] - 2 + t, sinks, window).tolist()):
                assert np.isnan(o[b * 3 + t]).all() and np.isnan(l[b * 3 + t]).all()
            else:
                check_row(inp, sinks, window, b, t, o[b * 3 + t], l[b * 3 + t])
                clean += 1
    assert clean == 1  # request 0's middle row (request 1's older one is a sink, which every row sees)


def test_bad_data_is_skipped_and_reported():
    inp = make([500, 300, 40, 200], 2, 64, 130, seed=7, release=False)
    inp.block_table[0, 0], inp.block_table[0, 6] = -3, inp.num_pages  # a sink page, one in the window
    inp.block_table[3, 0], inp.block_table[3, 1], inp.block_table[3, 2], inp.block_table[3, 3] = -1, -1, -1, -1
    keep = inp.ctx.copy()
    inp.ctx = np.array([500, 1, 40, 200], np.int32)
    d = Dev(inp)
    out, lse = launch(d, 64, 130)
    assert dsa.get_device_error(d.ws) == dsa.DSA_DEVERR_CTX | dsa.DSA_DEVERR_BLOCK_TABLE
    o, l = bf16_to_np(out), lse.cpu().numpy()
    for r in (0, 1, 4, 5):
        check_row(inp, 64, 130, r // 2, r % 2, o[r], l[r])
    for r in (2, 3, 6, 7):
        assert (o[r] == 0).all() and np.isneginf(l[r]).all()
    inp.ctx = keep


def test_a_query_with_nan_spoils_its_head_alone():
    inp = make([300], 2, 10, 100, seed=8)
    inp.q[0, 1, 7, 30] = 0x7FC0
    inp.q[0, 1, 9, 3] = 0xFF80
    d = Dev(inp)
    out, lse = launch(d, 10, 100)
    o, l = bf16_to_np(out), lse.cpu().numpy()
    check_row(inp, 10, 100, 0, 0, o[0], l[0])
    for h in (7, 9):
        assert np.isnan(o[1, h]).all() and np.isnan(l[1, h])
    rest = np.delete(np.arange(96), [7, 9])
    inp.q[0, 1, [7, 9]] = 0
    assert np.isfinite(o[1, rest]).all()
    out, lse2 = launch(Dev(inp), 10, 100)
    assert (bf16_to_np(out)[1, rest] == o[1, rest]).all()


def test_sharp_scores_at_both_ends():
    """One token far above the others in the sinks, at the window's first token, or just outside of it."""
    sinks, window = 4, 300
    inp = make([1000, 1000, 1000], 1, sinks, window, seed=9, release=False)
    inp.softmax_scale = 1.0
    from oracle.formats import bf16_decode
    direction = np.sign(bf16_decode(inp.q[0, 0, 0]))
    rng = np.random.default_rng(2)
    q = rng.standard_normal((3, 1, 96, 576)) * 0.05 + direction * 0.06
    inp.q = gen.f32_to_bf16_bits(q.astype(np.float32))
    rows = inp.lat_pool.reshape(-1, 576)
    for b, s in ((0, 2), (1, 700), (2, 699)):
        rows[inp.block_table[b, s // 64] * 64 + s % 64] = gen.encode_e4m3(direction * 4.0)
    check(inp, sinks, window)


def test_offsets_past_32_bits():
    """Pages far apart: the pool's last pages lie beyond 4 GB."""
    import torch

    inp = make([500], 1, 64, 200, seed=10)
    d = Dev(inp)
    ref, _ = launch(d, 64, 200)
    n = 130000
    pool = torch.empty(n, 36864, dtype=torch.uint8, device="cuda")
    pool[n - inp.num_pages:] = torch.from_numpy(inp.lat_pool[:, :36864]).cuda()
    p = dsa.make_params(batch=1, n_q=1, max_pages_per_req=inp.max_pages, num_pages=n, key_page_stride=8448, lat_page_stride=36864,
                        softmax_scale=inp.softmax_scale, latent_scale=inp.latent_scale)
    table = torch.where((d.block_table >= 0) & (d.block_table < inp.num_pages), d.block_table + (n - inp.num_pages), -1)
    ws = torch.zeros(dsa.workspace_size(p), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(ref)
    dsa.window_mla_decode(p, d.q, pool, 64, 200, table, d.ctx, out, None, ws)
    assert torch.equal(out, ref)


def test_graph_replay_and_two_streams():
    import torch

    inp = make([900, 400], 2, 10, 250, seed=11, release=False)
    d = Dev(inp)
    out, lse = torch.empty(4, 96, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 96, device="cuda")
    call = lambda: dsa.window_mla_decode(d.p, d.q, d.lat_pool, 10, 250, d.block_table, d.ctx, out, lse, d.ws)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([870, 2], [640, 399]):
        inp.ctx = np.array(lens, np.int32)
        d.ctx.copy_(torch.from_numpy(inp.ctx))
        graph.replay()
        o, l = bf16_to_np(out), lse.cpu().numpy()
        for r in range(4):
            check_row(inp, 10, 250, r // 2, r % 2, o[r], l[r])
    # two calls at once, each with a workspace of its own
    ref, streams = out.clone(), [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [torch.zeros_like(d.ws) for _ in streams]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                outs.append(launch(d, 10, 250, ws=w)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


# ---------------------------------------------------------------- accumulated weights


def weights(inp, sinks, window, lse=None, fresh=0, start=None, d=None, stride=None, stream=None):
    """(mass after, mass before, lse) on the host; lse: the oracle's unless given."""
    import torch

    d = d or Dev(inp)
    if lse is None:
        lse = np.stack([B.window_mla(inp, sinks, window, b, t, off(inp))[1] for b in range(inp.batch) for t in range(inp.n_q)])
    lse = np.asarray(lse, np.float32).reshape(inp.batch, inp.n_q, 96)
    width = inp.max_pages * 64
    rng = np.random.default_rng(0)
    start = rng.random((inp.batch, stride or width)).astype(np.float32) if start is None else start
    mass = torch.from_numpy(start.copy()).cuda()
    dsa.attention_mass(d.p, d.q, d.lat_pool, sinks, window, d.block_table, d.ctx, torch.from_numpy(lse).cuda(), fresh, mass, d.ws, stream)
    return mass.cpu().numpy(), start, lse


def check_mass(inp, sinks, window, got, start, lse, fresh=0, requests=None):
    for b in range(inp.batch) if requests is None else requests:
        tok, add, bound = B.attention_mass(inp, sinks, window, lse[b], b, off(inp))
        new = tok >= inp.ctx[b] - fresh
        ref = np.where(new, 0, start[b, tok].astype(np.float64)) + add
        err = np.abs(got[b, tok] - ref)
        assert (err <= bound + 2.0 ** -23 * ref).all(), (b, tok[err.argmax()], (err / (bound + 2.0 ** -23 * ref)).max())
        rest = np.delete(np.arange(got.shape[1]), tok)
        assert (got[b, rest] == start[b, rest]).all(), b


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("lens,n_q,sinks,window", CASES)
def test_mass_matches_oracle(lat_fmt, lens, n_q, sinks, window):
    inp = make(lens, n_q, sinks, window, seed=20 + len(lens) + n_q, lat_fmt=lat_fmt)
    d = Dev(inp)
    for fresh in (0, n_q, ALL):
        check_mass(inp, sinks, window, *weights(inp, sinks, window, fresh=fresh, d=d), fresh=fresh)
    assert dsa.get_device_error(d.ws) == 0


def test_mass_of_long_contexts_and_many_requests():
    inp = make([9000 + 331 * i for i in range(40)], 2, 70, 5000, seed=21)
    d = Dev(inp)
    _, lse = launch(d, 70, 5000)
    got = weights(inp, 70, 5000, lse=lse.cpu().numpy(), d=d, stride=inp.max_pages * 64 + 5)
    check_mass(inp, 70, 5000, *got, requests=(0, 7, 39))
    inp = make([40001], 7, 0, ALL, seed=22, lat_fmt="nvfp4")
    d = Dev(inp)
    _, lse = launch(d, 0, ALL)
    check_mass(inp, 0, ALL, *weights(inp, 0, ALL, lse=lse.cpu().numpy(), d=d, fresh=7), fresh=7)


def test_mass_of_a_chunk_and_padded_pages():
    inp = make([300, 170], 70, 3, 90, seed=23, lat_page_pad=4096, holes=True)
    check_mass(inp, 3, 90, *weights(inp, 3, 90))


def test_mass_does_not_depend_on_the_batch():
    inp = make([1500, 1111, 800, 64, 1300], 3, 17, 900, seed=24)
    whole, start, lse = weights(inp, 17, 900)
    import dataclasses
    for b in (0, 1, 3, 4):
        one = dataclasses.replace(inp, batch=1, ctx=inp.ctx[b:b + 1], block_table=inp.block_table[b:b + 1], q=inp.q[b:b + 1],
                                  q_idx=inp.q_idx[b:b + 1], w=inp.w[b:b + 1])
        got, _, _ = weights(one, 17, 900, lse=lse[b:b + 1], start=start[b:b + 1])
        assert (got == whole[b:b + 1]).all()


@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
def test_mass_of_nan_and_missing_lse(lat_fmt):
    """Heads without a finite lse add nothing, even where their query is NaN; a NaN latent spoils its token alone; hidden
    tokens and padding may hold anything."""
    sinks, window, size = 70, 100, 576 if lat_fmt == "fp8" else 352
    inp = make([400, 171], 3, sinks, window, seed=25, lat_fmt=lat_fmt, release=False)
    lse = np.stack([B.window_mla(inp, sinks, window, b, t, off(inp))[1] for b in range(2) for t in range(3)]).reshape(2, 3, 96)
    lse = lse.astype(np.float32)
    lse[0, 1, 5], lse[0, 2, 95], lse[1, 0, 0], lse[1, 2] = -np.inf, np.nan, np.inf, -np.inf
    inp.q[0, 2, 95, 7], inp.q[1, 0, 0, 100] = 0x7FC0, 0x7F80
    clean = inp.q.copy()
    clean[0, 2, 95], clean[1, 0, 0] = 0, 0
    rows = inp.lat_pool.reshape(-1, size)
    for b, n in enumerate(inp.ctx):
        for s in list(range(sinks, n - 2 - window)) + list(range(n, -(-n // 64) * 64)):
            rows[inp.block_table[b, s // 64] * 64 + s % 64] = 0x7F
    got = weights(inp, sinks, window, lse=lse)
    inp.q = clean
    check_mass(inp, sinks, window, *got)
    s = 399  # the last row's alone
    rows[inp.block_table[0, s // 64] * 64 + s % 64] = 0x7F
    bad, _, _ = weights(inp, sinks, window, lse=lse)
    assert np.isnan(bad[0, s]) and (np.delete(bad[0], s) == np.delete(got[0][0], s)).all() and (bad[1] == got[0][1]).all()


def test_mass_of_bad_data_changes_nothing():
    inp = make([500, 300, 200], 2, 64, 130, seed=26, release=False)
    lse = np.zeros((3, 2, 96), np.float32) + 3
    inp.block_table[0, 0], inp.block_table[0, 6] = -3, inp.num_pages
    inp.ctx = np.array([500, 1, 200], np.int32)
    d = Dev(inp)
    got, start, lse = weights(inp, 64, 130, lse=lse, d=d)
    assert dsa.get_device_error(d.ws) == dsa.DSA_DEVERR_CTX | dsa.DSA_DEVERR_BLOCK_TABLE
    check_mass(inp, 64, 130, got, start, lse, requests=(0, 2))
    assert (got[1] == start[1]).all()


def test_mass_in_a_graph_on_one_workspace_with_the_attention():
    import torch

    inp = make([900, 400], 2, 10, 250, seed=27, release=False)
    d = Dev(inp)
    out, lse = torch.empty(4, 96, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 96, device="cuda")
    mass = torch.zeros(2, inp.max_pages * 64, device="cuda")

    def step():
        dsa.window_mla_decode(d.p, d.q, d.lat_pool, 10, 250, d.block_table, d.ctx, out, lse, d.ws)
        dsa.attention_mass(d.p, d.q, d.lat_pool, 10, 250, d.block_table, d.ctx, lse, 2, mass, d.ws)

    step()
    first = mass.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    mass.zero_()
    graph.replay()
    assert torch.equal(mass, first)
    lens = np.array([871, 33], np.int32)
    d.ctx.copy_(torch.from_numpy(lens))
    start = mass.cpu().numpy()
    graph.replay()
    inp.ctx = lens
    check_mass(inp, 10, 250, mass.cpu().numpy(), start, lse.cpu().numpy().reshape(2, 2, 96), fresh=2)
    assert dsa.get_device_error(d.ws) == 0
