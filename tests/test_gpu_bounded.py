"""The operators of a bounded cache together, as a server of endless conversations runs them: each step grows the
requests, writes the new tokens (index keys and latents), attends through a window with sinks, adds up the weights and cuts
who is over the budget; the sparse decode step runs on what is left. Positions go on as tokens are evicted. Eager and as
one captured graph, every state against the oracle."""
import dataclasses

import numpy as np
import pytest

import dsa_sparse_mla_paged_gb300 as dsa
import gen
from oracle import bounded as B
from oracle import dsa as O
from oracle import serving as S
from oracle.formats import bf16_decode

from dsa_testlib import LAT_FMT, bf16_to_np
from test_gpu_latent import near
from test_gpu_window import check_mass, check_row

pytestmark = pytest.mark.gpu
N, N_Q, SINKS, WINDOW, RECENT, BUDGET, WIDTH, PAGES = 3, 4, 6, 150, 40, 230, 5, 24


@pytest.fixture(scope="module", autouse=True)
def _need(lib, cuda_ok):
    yield


class Server:
    def __init__(self, lat_fmt):
        import torch

        self.rng, self.fmt, self.row = np.random.default_rng(5), lat_fmt, {"fp8": 576, "nvfp4": 352}[lat_fmt]
        self.inp = gen.make_inputs(N, N_Q, WIDTH * 64, seed=6, lat_fmt=lat_fmt, bt_mode="permuted")
        self.inp.latent_scale = 0.75
        self.p = dsa.make_params(batch=N, n_q=N_Q, max_pages_per_req=WIDTH, num_pages=PAGES, key_page_stride=8448, topk=256,
                                 lat_page_stride=64 * self.row, lat_fmt=LAT_FMT[lat_fmt], softmax_scale=self.inp.softmax_scale,
                                 latent_scale=0.75)
        self.table, self.ctx, self.refs = np.full((N, WIDTH), -1, np.int32), np.zeros(N, np.int32), np.zeros(PAGES, np.int32)
        self.seen = np.zeros(N, np.int64)  # tokens so far: the next position
        self.mass, self.kept = np.zeros((N, WIDTH * 64), np.float32), np.full((N, WIDTH * 64), -1, np.int32)
        rng = self.rng
        self.keys, self.lats = rng.integers(0, 100, (PAGES, 8448), dtype=np.uint8), np.full((PAGES, 64 * self.row), 0xFF, np.uint8)
        self.keys.reshape(PAGES, -1)[:, 8192:] = np.ones((PAGES, 64), np.float32).view(np.uint8)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a).copy()).cuda()
        self.d = {k: t(getattr(self, k)) for k in ("table", "ctx", "refs", "mass", "kept", "keys", "lats")}
        z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")
        rows, i32, f32 = N * N_Q, torch.int32, torch.float32
        self.d_in = dict(q_nope=z(rows, 96, 512), q_rope=z(rows, 96, 64), c_kv=z(rows, 512), k_rope=z(rows, 64))
        self.d_seen, self.d_budget = z(N, dtype=i32), torch.full((N,), BUDGET, dtype=i32, device="cuda")
        self.d_q, self.d_out, self.d_lse = z(rows, 96, 576), z(rows, 96, 512), z(rows, 96, dtype=f32)
        self.d_mass = z(N, WIDTH * 64, dtype=f32)  # what the eviction found
        self.d_before = z(N, dtype=i32)
        self.gamma, self.freq = gen.f32_to_bf16_bits(rng.uniform(0.5, 1.5, 512).astype(np.float32)), (1e4 ** (-np.arange(32) / 32)).astype(np.float32)
        self.d_gamma, self.d_freq = t(self.gamma.view(np.int16)).view(torch.bfloat16), t(self.freq)
        self.ws = torch.zeros(dsa.workspace_size(self.p), dtype=torch.uint8, device="cuda")
        self.pools = dsa.make_pools([(self.d["keys"], 8448, 8448), (self.d["lats"], 64 * self.row, 64 * self.row)])
        tok = dsa.DSA_TOKEN_LAT_FP8 if lat_fmt == "fp8" else dsa.DSA_TOKEN_LAT_NVFP4
        self.tokens = dsa.make_token_pools([(self.d["keys"], dsa.DSA_TOKEN_KEY_FP8, 1, 0, 8448), (self.d["lats"], tok, 1, 0, 64 * self.row)])

    def grow_and_write(self):
        import torch

        d = self.d
        dsa.pages_resize(self.p, d["ctx"] + N_Q, self.pools, d["table"], d["ctx"], d["refs"], self.ws)
        pos = (self.d_seen[:, None] + torch.arange(N_Q, device="cuda", dtype=torch.int32)).flatten()
        dsa.latent_frontend(self.p, self.d_in["q_nope"], self.d_in["q_rope"], None, self.d_in["c_kv"], self.d_in["k_rope"], self.d_gamma,
                            self.d_freq, pos, d["lats"], d["table"], d["ctx"], self.d_q, self.ws)
        self.d_seen += N_Q

    def launch(self):
        d = self.d
        self.grow_and_write()
        dsa.window_mla_decode(self.p, self.d_q, d["lats"], SINKS, WINDOW, d["table"], d["ctx"], self.d_out, self.d_lse, self.ws)
        dsa.attention_mass(self.p, self.d_q, d["lats"], SINKS, WINDOW, d["table"], d["ctx"], self.d_lse, N_Q, d["mass"], self.ws)
        self.d_mass.copy_(d["mass"])
        dsa.tokens_evict(self.p, self.d_budget, SINKS, RECENT, d["mass"], self.tokens, d["table"], d["ctx"], d["refs"], d["kept"], self.ws)

    def step(self, run, check=True):
        import torch

        rng, rows = self.rng, N * N_Q
        bits = {k: gen.f32_to_bf16_bits((2 * rng.standard_normal(v.shape)).astype(np.float32)) for k, v in self.d_in.items()}
        for k, v in self.d_in.items():
            v.copy_(torch.from_numpy(bits[k].view(np.int16)).view(torch.bfloat16))
        run()
        assert dsa.get_device_error(self.ws) == 0
        host = {k: v.cpu().numpy() for k, v in self.d.items()}
        # the step's pages, then its latents: the device's bytes where they are what the oracle allows
        assert S.pages_resize(self.table, self.ctx, self.refs, self.ctx + N_Q, [self.keys, self.lats]) == 0
        before, start = self.ctx.copy(), self.mass
        q = self.d_q.view(torch.int16).cpu().numpy().view(np.uint16).reshape(N, N_Q, 96, 576)
        for r in range(rows):
            b, t = divmod(r, N_Q)
            pos, slot = self.seen[b] + t, before[b] - N_Q + t
            x = {k: bf16_decode(v[r]) for k, v in bits.items()}
            want, lat = B.front_row(x["q_nope"], x["q_rope"], None, x["c_kv"], x["k_rope"], bf16_decode(self.gamma), self.freq, pos, 1e-6, True)
            assert np.abs(bf16_decode(q[b, t]) - want).max() <= 2.0 ** -8 * np.abs(want).max() + 2.0 ** -20
            # where the eviction left the token: it is among the last RECENT, which stay
            stay = host["ctx"][b] - (before[b] - slot)
            raw = host["lats"].reshape(-1, self.row)[host["table"][b, stay // 64] * 64 + stay % 64]
            if self.fmt == "fp8":
                near(raw[:512], lat[:512] / 0.75, 2.0 ** -21 * np.abs(lat[:512]) / 0.75, r)
            near(raw[-64:], lat[512:] / 0.75, np.full(64, 2.0 ** -18), r)
            self.lats.reshape(-1, self.row)[self.table[b, slot // 64] * 64 + slot % 64] = raw
        self.seen += N_Q
        inp = dataclasses.replace(self.inp, ctx=before, block_table=self.table.copy(), lat_pool=self.lats.copy(), q=q, num_pages=PAGES,
                                  key_pool=self.keys.copy())
        out, lse, mass = bf16_to_np(self.d_out), self.d_lse.cpu().numpy(), self.d_mass.cpu().numpy()
        if check:
            for r in range(rows):
                check_row(inp, SINKS, WINDOW, r // N_Q, r % N_Q, out[r], lse[r])
            check_mass(inp, SINKS, WINDOW, mass, start, lse.reshape(N, N_Q, 96), fresh=N_Q)
        self.mass = mass.copy()
        pools = [("key_fp8", [self.keys]), ("lat_" + self.fmt, [self.lats])]
        assert B.tokens_evict(self.table, self.ctx, self.refs, self.mass, [BUDGET] * N, SINKS, RECENT, pools, self.kept) == 0
        for k in ("table", "ctx", "refs", "mass", "kept"):
            assert (host[k] == getattr(self, k)).all(), k
        for b in range(N):  # the rows that are in use
            s = np.arange(self.ctx[b])
            at = self.table[b, s // 64] * 64 + s % 64
            assert (host["lats"].reshape(-1, self.row)[at] == self.lats.reshape(-1, self.row)[at]).all()
        assert (host["keys"] == self.keys).all()

    def prompt(self, lens):
        import torch

        # random latents stand for a prompt of the given lengths
        d = self.d
        dsa.pages_resize(self.p, torch.tensor(lens, dtype=torch.int32, device="cuda"), self.pools, d["table"], d["ctx"], d["refs"], self.ws)
        assert S.pages_resize(self.table, self.ctx, self.refs, lens, [self.keys, self.lats]) == 0
        source = self.inp.lat_pool.reshape(-1, self.row)
        for b in range(N):
            s = np.arange(self.ctx[b])
            self.lats.reshape(-1, self.row)[self.table[b, s // 64] * 64 + s % 64] = source[b * 300 + s]
        d["lats"].copy_(torch.from_numpy(self.lats))
        self.seen += self.ctx
        self.d_seen.copy_(torch.from_numpy(self.seen))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
def test_a_server_of_endless_conversations(lat_fmt, captured):
    import torch

    s = Server(lat_fmt)
    s.prompt([225, 100, 218])
    s.step(s.launch)
    run = s.launch
    if captured:
        graph, seen = torch.cuda.CUDAGraph(), s.d_seen.clone()
        with torch.cuda.graph(graph):
            s.launch()
        assert torch.equal(s.d_seen, seen)
        run = graph.replay
    for i in range(8):
        s.step(run, check=i % 3 == 0)
    assert s.ctx.tolist() == [BUDGET, 136, BUDGET] and s.seen.tolist() == [261, 136, 254]
    # the sparse step on the cache that is left: with K above the contexts it is dense attention over them
    rng, rows = np.random.default_rng(7), N * N_Q
    q_idx, w = torch.randn(rows, 32, 128, device="cuda").to(torch.bfloat16), torch.rand(rows, 32, device="cuda")
    idx = torch.zeros(rows, 256, dtype=torch.int32, device="cuda")
    d = s.d
    dsa.decode(s.p, q_idx, w, d["keys"], s.d_q, d["lats"], d["table"], d["ctx"], s.d_out, s.d_lse, idx, s.ws)
    assert dsa.get_device_error(s.ws) == 0
    q = s.d_q.view(torch.int16).cpu().numpy().view(np.uint16).reshape(N, N_Q, 96, 576)
    inp = dataclasses.replace(s.inp, ctx=s.ctx.copy(), block_table=s.table.copy(), lat_pool=d["lats"].cpu().numpy(), q=q, num_pages=PAGES)
    # (the weights and the output are bf16, each off by 2^-8 of itself at most: so many of sum p |c| and of |out|; the
    # fp32 logits are within 2^-13, as the sums of 576 products of at most 100 in all are by 66 * 2^-23 of them)
    out, lse = bf16_to_np(s.d_out), s.d_lse.cpu().numpy()
    for r in range(rows):
        c = O.dequant_latents(inp, r // N_Q, np.arange(s.ctx[r // N_Q] - N_Q + r % N_Q + 1))
        x = bf16_decode(q[r // N_Q, r % N_Q])
        assert (inp.softmax_scale * np.abs(x) @ np.abs(c).T).max() <= 100
        ref, ref_lse = O.mla_attention(x, c, inp.softmax_scale)
        mass = np.exp(inp.softmax_scale * (x @ c.T) - ref_lse[:, None]) @ np.abs(c[:, :512])
        assert (np.abs(out[r] - ref) <= (2.0 ** -8 + 2.0 ** -11) * mass + 2.0 ** -8 * np.abs(ref)).all()
        assert np.abs(lse[r] - ref_lse).max() <= 2.0 ** -12
    # an evicted request forked, and its copy cut: the fork keeps what it had
    one = torch.tensor([0], dtype=torch.int32, device="cuda")
    dsa.pages_resize(s.p, torch.tensor([-1, 0, -1], dtype=torch.int32, device="cuda"), s.pools, d["table"], d["ctx"], d["refs"], s.ws)
    dsa.pages_fork(s.p, one, one + 1, d["table"], d["ctx"], d["refs"], s.ws)
    d["mass"][1] = d["mass"][0]
    rows_of = lambda b: d["lats"].view(-1, s.row)[(d["table"][b].long()[:, None] * 64 + torch.arange(64, device="cuda")).flatten()[:BUDGET]]
    before = rows_of(0).clone()
    dsa.tokens_evict(s.p, torch.tensor([-1, 100, -1], dtype=torch.int32, device="cuda"), SINKS, RECENT, d["mass"], s.tokens, d["table"],
                     d["ctx"], d["refs"], d["kept"], s.ws)
    assert dsa.get_device_error(s.ws) == 0 and d["ctx"].tolist() == [BUDGET, 100, BUDGET]
    assert torch.equal(rows_of(0), before)
    assert torch.equal(rows_of(1)[:100], before[d["kept"][1, :100].long()])
