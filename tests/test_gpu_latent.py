"""dsa_latent_frontend against the float64 oracle.

Bounds, derived from the arithmetic that include/dsa.h states:
- a latent value is ((x * r) * gamma) * (1 / scale) with r rounded from fp64 and 1 / scale to fp32: five roundings of 2^-24,
  2^-21 of it in all; the code must be one of those that the values off by that much either way round to;
- a rotated value x0 cos - x1 sin: cosine and sine are within 2^-24 of themselves rounded, and 2^-33 for the angle (positions to
  2^20, rounded to 53 bits); each product rounds by 2^-24 and their difference by 2^-24 of the sum of both: 4 * 2^-24 of
  |x0| + |x1|, with the scale's two roundings 6 * 2^-24;
- a query value without a norm is copied; rotated 4 * 2^-24 (|x0| + |x1|), and bf16's 2^-8 of itself (2^-134 among subnormals);
- with a norm: a sum of 512 squares by 16 additions a lane and 5 across, 22 * 2^-24 of it, half of that in the root, 2^-22 for the
  reciprocal root, and three roundings: 2^-20 of it, and bf16's 2^-8.
Nothing here is measured first."""
import numpy as np
import pytest

import dsa_sparse_mla_paged_gb300 as dsa
import gen
from oracle import bounded as B
from oracle.formats import E2M1, E4M3, bf16_decode, e4m3_encode_rne_satfinite

from dsa_testlib import LAT_FMT, bf16_to_np

pytestmark = pytest.mark.gpu
ROW = {"fp8": 576, "nvfp4": 352}


@pytest.fixture(scope="module", autouse=True)
def _need(lib, cuda_ok):
    yield


class Case:
    def __init__(self, lens, n_q, fmt="fp8", norm_q=True, positions=False, scale=0.75, seed=0, pad=0, size=3.0, width=None):
        import torch

        rng = np.random.default_rng(seed)
        self.B, self.n_q, self.fmt, self.scale, rows = len(lens), n_q, fmt, scale, len(lens) * n_q
        self.rows, self.lens = rows, np.array(lens, np.int32)
        width = width or max(max(-(-int(x) // 64) for x in lens), 1)
        self.pages = self.B * width + 3
        self.table = rng.permutation(self.pages)[:self.B * width].astype(np.int32).reshape(self.B, width)
        bits = lambda *s: gen.f32_to_bf16_bits((rng.standard_normal(s) * size).astype(np.float32))
        self.q_nope, self.q_rope, self.c_kv, self.k_rope = bits(rows, 96, 512), bits(rows, 96, 64), bits(rows, 512), bits(rows, 64)
        self.gamma_kv, self.gamma_q = bits(512), bits(512) if norm_q else None
        self.inv_freq = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
        self.positions = rng.integers(0, 1 << 20, rows).astype(np.int32) if positions else None
        self.stride = 64 * ROW[fmt] + pad
        self.p = dsa.make_params(batch=self.B, n_q=n_q, max_pages_per_req=width, num_pages=self.pages, key_page_stride=8448,
                                 lat_page_stride=self.stride, lat_fmt=LAT_FMT[fmt], latent_scale=scale)
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def dev(self, a, dtype=None):
        import torch

        if a is None:
            return None
        t = torch.from_numpy(np.ascontiguousarray(a.view(np.int16) if a.dtype == np.uint16 else a)).cuda()
        return t.view(torch.bfloat16) if a.dtype == np.uint16 else t

    def inputs(self):
        return {k: self.dev(getattr(self, k)) for k in ("q_nope", "q_rope", "gamma_q", "c_kv", "k_rope", "gamma_kv", "inv_freq",
                                                        "positions")}

    def run(self, interleaved=True, eps=1e-6, stream=None, **change):
        import torch

        pool = torch.full((self.pages, self.stride), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.full((self.rows, 96, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
        args = {**self.inputs(), "lat_pool": pool, "block_table": self.dev(self.table), "ctx_lens": self.dev(self.lens), "q_out": out,
                **change}
        dsa.latent_frontend(self.p, **args, ws=self.ws, eps=eps, interleaved=interleaved, stream=stream)
        return args["lat_pool"], args["q_out"]

    def check(self, pool, out, interleaved=True, eps=1e-6, rows=None, query=True, cache=True):
        pool, written = pool.cpu().numpy(), np.zeros((self.pages, 64), bool)
        out = bf16_to_np(out) if query else None
        dec = bf16_decode
        for r in range(self.rows):
            b, t = divmod(r, self.n_q)
            slot = self.lens[b] - self.n_q + t
            page, at = self.table[b, slot // 64], slot % 64
            written[page, at] = True
            if rows is not None and r not in rows:
                continue
            pos = slot if self.positions is None else self.positions[r]
            q, lat = B.front_row(dec(self.q_nope[r]), dec(self.q_rope[r]), None if self.gamma_q is None else dec(self.gamma_q),
                                 dec(self.c_kv[r]), dec(self.k_rope[r]), dec(self.gamma_kv), self.inv_freq, pos, eps, interleaved)
            pair = lambda x: np.abs(x) + np.abs(x[..., np.arange(64) ^ 1] if interleaved else np.roll(x, 32, -1))
            if query:
                got = out[r].astype(np.float64)
                if self.gamma_q is None:
                    assert (got[:, :512] == q[:, :512]).all()
                slack = np.concatenate([2.0 ** -20 * np.abs(q[:, :512]), 4 * 2.0 ** -24 * pair(dec(self.q_rope[r]))], 1)
                err = np.abs(got - q)
                assert (err <= 2.0 ** -8 * np.abs(q) + (1 + 2.0 ** -8) * slack + 2.0 ** -134).all(), (r, err.max())
            if cache:
                v = lat / self.scale
                slack = np.concatenate([2.0 ** -21 * np.abs(v[:512]), 6 * 2.0 ** -24 * pair(dec(self.k_rope[r])) / self.scale])
                self.check_row(pool[page, at * ROW[self.fmt]:(at + 1) * ROW[self.fmt]], v, slack, r)
        if cache:  # nothing else was written
            body = pool[:, :64 * ROW[self.fmt]].reshape(self.pages, 64, -1)
            assert (body[~written] == 0xA5).all() and (pool[:, 64 * ROW[self.fmt]:] == 0xA5).all()

    def check_row(self, raw, v, slack, r):
        nope, rope = (raw[:512], raw[512:]) if self.fmt == "fp8" else (raw[:256], raw[288:])
        near(rope, v[512:], slack[512:], r)
        if self.fmt == "fp8":
            return near(nope, v[:512], slack[:512], r)
        amax = np.abs(v[:512]).reshape(32, 16).max(1) / 6
        near(raw[256:288], amax, 2.0 ** -20 * amax, r)
        s = E4M3[raw[256:288]].repeat(16)
        codes = np.empty(512, np.uint8)
        codes[0::2], codes[1::2] = nope & 15, nope >> 4
        assert (codes[s == 0] == 0).all()
        s, codes, v = s[s > 0], codes[s > 0], v[:512][s > 0]
        lo, hi = (np.abs(v) * (1 - 2.0 ** -20) / s, np.abs(v) * (1 + 2.0 ** -20) / s)
        a = E2M1[codes & 7]
        assert ((a >= E2M1[gen.encode_e2m1(lo)]) & (a <= E2M1[gen.encode_e2m1(hi)])).all(), r
        assert ((codes >= 8) == (v < 0)).all(), r  # the sign is kept


def near(codes, v, slack, r):
    """E4M3 codes of values within `slack` of v."""
    got = E4M3[codes]
    lo, hi = (E4M3[gen.encode_e4m3(v - slack)], E4M3[gen.encode_e4m3(v + slack)])
    assert ((got >= lo) & (got <= hi)).all(), (r, np.nonzero((got < lo) | (got > hi))[0][:5])


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("lens,n_q,norm_q,positions", [
    ([1], 1, False, False), ([64], 1, True, True), ([65, 700], 1, True, False), ([130, 9], 3, False, True), ([70, 8, 1000], 8, True, True)])
def test_matches_oracle(fmt, interleaved, lens, n_q, norm_q, positions):
    c = Case(lens, n_q, fmt, norm_q, positions, seed=n_q + len(lens))
    c.check(*c.run(interleaved), interleaved)
    assert dsa.get_device_error(c.ws) == 0


@pytest.mark.parametrize("fmt,norm_q", [("fp8", False), ("nvfp4", True)])
def test_a_chunk_and_many_rows(fmt, norm_q):
    """Enough rows for the other division of the heads; page padding; odd rows."""
    c = Case([333, 300, 1001], 299, fmt, norm_q, True, seed=9, pad=64)
    c.check(*c.run(False), False, rows={0, 1, 298, 299, 598, 600, 895, 896})


def test_sizes_of_values():
    """Tiny and huge values, zeros, a scale that saturates E4M3, blocks that underflow."""
    for fmt in ("fp8", "nvfp4"):
        c = Case([40], 4, fmt, True, False, scale=2.0 ** -6, seed=3)
        f = np.random.default_rng(1)
        c.gamma_kv = gen.f32_to_bf16_bits((2.0 ** f.integers(-40, 12, 512) * f.choice([-1, 1], 512)).astype(np.float32))
        c.c_kv[1] = 0
        c.q_nope[1] = 0
        c.c_kv[2] = gen.f32_to_bf16_bits(np.full(512, 1e18, np.float32))
        c.c_kv[3] = gen.f32_to_bf16_bits(np.full(512, 3e-6, np.float32))  # next to the epsilon
        c.check(*c.run(True), True)
        c.check(*c.run(True, eps=2.5), True, eps=2.5)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_nan_and_infinity_stay_in_their_rows(fmt):
    c = Case([70], 4, fmt, True, False, seed=4)
    c.c_kv[1, 77] = 0x7FC0
    c.c_kv[2, 5] = 0x7F80
    c.q_nope[1, 3, 9] = 0x7FC0
    pool, out = c.run()
    c.check(pool, out, rows={0, 3})
    out, raw = bf16_to_np(out), pool.cpu().numpy()
    assert np.isnan(out[1, 3, :512]).all() and not np.isnan(out[1, 3, 512:]).any() and not np.isnan(np.delete(out[1], 3, 0)).any()
    row = lambda r: raw[c.table[0, (66 + r) // 64], (66 + r) % 64 * ROW[fmt]:][:ROW[fmt]]
    if fmt == "fp8":
        assert np.isnan(E4M3[row(1)[:512]]).all() and np.isnan(E4M3[row(2)[5]]) and (E4M3[np.delete(row(2)[:512], 5)] == 0).all()
    else:
        assert np.isnan(E4M3[row(1)[256:288]]).all() and np.isnan(E4M3[row(2)[256]]) and (E4M3[row(2)[257:288]] == 0).all()


@pytest.mark.parametrize("n_q", [2, 150])
def test_strided_inputs_in_place_and_parts(n_q):
    import torch

    c = Case([180, 170], n_q, "fp8", True, True, seed=5)
    ref_pool, ref = c.run()
    c.check(ref_pool, ref, rows={0, 1, c.rows - 1})
    i = c.inputs()
    # heads of rows, the rotary part behind 128 other values, latent and rotary part side by side, rows [B, n_q]
    up = torch.randn(c.B, n_q, 96, 192, device="cuda").to(torch.bfloat16)
    up[..., 128:] = i["q_rope"].view(c.B, n_q, 96, 64)
    kv = torch.cat([i["c_kv"], i["k_rope"]], 1).view(c.B, n_q, 576)
    pool, out = c.run(q_nope=i["q_nope"].transpose(0, 1).contiguous().transpose(0, 1), q_rope=up[..., 128:], c_kv=kv[..., :512],
                      k_rope=kv[..., 512:])
    assert torch.equal(out, ref) and torch.equal(pool, ref_pool)
    # the query in its own place
    own = torch.cat([i["q_nope"], i["q_rope"]], 2)
    pool, out = c.run(q_nope=own[:, :, :512], q_rope=own[:, :, 512:], q_out=own)
    assert torch.equal(out, ref) and torch.equal(pool, ref_pool)
    # one part alone
    pool, _ = c.run(q_nope=None, q_rope=None, gamma_q=None, q_out=None)
    assert torch.equal(pool, ref_pool)
    pool, out = c.run(c_kv=None, k_rope=None, gamma_kv=None, lat_pool=None, block_table=None)
    assert torch.equal(out, ref)


def test_bad_rows_are_skipped_and_reported():
    c = Case([100, 70, 3, 200], 4, "fp8", True, False, seed=6, width=4)
    c.lens = np.array([100, 70, 3, 300], np.int32)  # the third is shorter than its new tokens, the fourth longer than its row
    c.table[1, 1] = c.pages
    pool, out = c.run()
    assert dsa.get_device_error(c.ws) == dsa.DSA_DEVERR_CTX | dsa.DSA_DEVERR_BLOCK_TABLE
    raw, touched = pool.cpu().numpy(), {(c.table[0, 1], 32 + t) for t in range(4)}
    for pg in range(c.pages):
        for s in range(64):
            assert ((raw[pg, s * 576:(s + 1) * 576] != 0xA5).any()) == ((pg, s) in touched), (pg, s)
    assert np.isfinite(bf16_to_np(out)).all()
    c.table[1, 1] = -1
    c.run()
    assert dsa.get_device_error(c.ws) == dsa.DSA_DEVERR_CTX | dsa.DSA_DEVERR_BLOCK_TABLE


def test_a_graph_replays_with_new_lengths_on_another_stream():
    import torch

    c = Case([70, 200], 2, "nvfp4", True, False, seed=7)
    args = {**c.inputs(), "lat_pool": torch.full((c.pages, c.stride), 0xA5, dtype=torch.uint8, device="cuda"),
            "block_table": c.dev(c.table), "ctx_lens": c.dev(c.lens),
            "q_out": torch.zeros(c.rows, 96, 576, dtype=torch.bfloat16, device="cuda")}
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dsa.latent_frontend(c.p, **args, ws=c.ws)
    for lens in ([66, 130], [5, 249]):
        c.lens = np.array(lens, np.int32)
        args["ctx_lens"].copy_(torch.from_numpy(c.lens))
        args["lat_pool"].fill_(0xA5)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        c.check(args["lat_pool"], args["q_out"])


def test_far_slots_and_positions():
    """A page beyond 4 GB of the pool, positions near 2^31."""
    import torch

    c = Case([64 * 3 + 2], 2, "fp8", False, False, seed=8)
    c.pages = 130000  # 4.8 GB
    c.p = dsa.make_params(batch=1, n_q=2, max_pages_per_req=4, num_pages=c.pages, key_page_stride=8448, lat_page_stride=c.stride)
    c.table[0, 3], c.scale = 129999, 1.0
    pool, out = c.run()
    row = pool[129999].cpu().numpy()[:2 * 576]
    small = Case([2], 2, "fp8", False, False, seed=8)
    for k in ("q_nope", "q_rope", "c_kv", "k_rope", "gamma_kv"):
        setattr(small, k, getattr(c, k))
    small.table[:], small.scale = 0, 1.0
    small.positions = np.array([192, 193], np.int32)
    small.p = dsa.make_params(batch=1, n_q=2, max_pages_per_req=1, num_pages=small.pages, key_page_stride=8448,
                              lat_page_stride=small.stride)
    pool2, out2 = small.run()
    assert (pool2[0].cpu().numpy()[:2 * 576] == row).all() and torch.equal(out, out2)
    # angles of whole turns and quarter turns at far positions: inv_freq 1 at 2^31 - 1 and its negative
    c = Case([4], 2, "fp8", False, False, seed=8)
    c.positions, c.inv_freq = np.array([2 ** 31 - 1, -2 ** 31 + 1], np.int32), np.ones(32, np.float32)
    c.check(*c.run())
