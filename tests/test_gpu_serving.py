"""The page operations, shared-prefix attention and draft verification together, as a
speculative server runs them: a prompt is written and forked, then each step grows the
requests (copying open pages), writes the new tokens' latents, attends, verifies the
drafts and trims what was rejected; in between a request ends and the pools are packed.
Every table, length and token against the oracle, exactly, and every output within
test_gpu_prefix's bounds; free pages hold NaN bytes throughout."""
import dataclasses

import numpy as np
import pytest

import dsa_sparse_mla_paged_gb300 as dsa
import gen
from oracle import serving as S

from dsa_testlib import LAT_FMT, bf16_to_np
from test_gpu_prefix import check_row

pytestmark = pytest.mark.gpu

B, N_Q, VOCAB, PROMPT, PREFIX = 4, 3, 1003, 200, 192


@pytest.fixture(scope="module", autouse=True)
def _need(lib, cuda_ok):
    yield


class Server:
    def __init__(self, lat_fmt):
        import torch

        self.rng = np.random.default_rng(41)
        self.inp = gen.make_inputs(B, N_Q, 400, seed=40, lat_fmt=lat_fmt, bt_mode="permuted")
        self.inp.latent_scale = 0.75
        self.row = {"fp8": 576, "nvfp4": 352}[lat_fmt]
        self.source = self.inp.lat_pool.reshape(-1, self.row)  # latents of new tokens
        self.taken = 0
        pages, width = self.inp.num_pages, self.inp.max_pages
        self.p = dsa.make_params(batch=B, n_q=N_Q, max_pages_per_req=width, num_pages=pages,
                                 key_page_stride=self.inp.key_page_stride, lat_page_stride=64 * self.row,
                                 lat_fmt=LAT_FMT[lat_fmt], softmax_scale=self.inp.softmax_scale,
                                 latent_scale=self.inp.latent_scale)
        # the host's copy, which the oracle changes
        self.table, self.ctx = np.full((B, width), -1, np.int32), np.zeros(B, np.int32)
        self.refs, self.pool = np.zeros(pages, np.int32), np.full((pages, 64 * self.row), 0xFF, np.uint8)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.d_table, self.d_ctx, self.d_refs, self.d_pool = (t(a.copy()) for a in (self.table, self.ctx, self.refs, self.pool))
        self.pools = dsa.make_pools([(self.d_pool, 64 * self.row, 64 * self.row)])
        self.ws = torch.zeros(dsa.workspace_size(self.p), dtype=torch.uint8, device="cuda")
        z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")
        self.d_new, self.d_grow, self.d_acc = (z(B, dtype=torch.int32) for _ in range(3))
        self.d_latents = z(B * N_Q, self.row, dtype=torch.uint8)
        self.d_q, self.d_target, self.d_draft = z(B, N_Q, 96, 576, dtype=torch.bfloat16), z(B, N_Q, VOCAB), z(B, N_Q - 1, VOCAB)
        self.d_tokens, self.d_uniforms = z(B, N_Q - 1, dtype=torch.int32), z(B, N_Q)
        self.d_out, self.d_lse = z(B * N_Q, 96, 512, dtype=torch.bfloat16), z(B * N_Q, 96)
        self.d_next = z(B, N_Q, dtype=torch.int32)
        self.d_prefix = z(PREFIX // 64, dtype=torch.int32)

    def resize(self, lens):
        import torch

        dsa.pages_resize(self.p, torch.tensor(lens, dtype=torch.int32, device="cuda"), self.pools, self.d_table, self.d_ctx,
                         self.d_refs, self.ws)
        assert S.pages_resize(self.table, self.ctx, self.refs, lens, [self.pool]) == 0

    def fresh(self, n):
        at = (self.taken + np.arange(n)) % len(self.source)
        self.taken += n
        return self.source[at]

    def write(self, b, pos, latents):
        """The host's copy of tokens `pos` of request b."""
        self.pool.reshape(-1, self.row)[self.table[b, pos // 64] * 64 + pos % 64] = latents

    def prompt(self):
        import torch

        self.resize([PROMPT] + [-1] * (B - 1))
        self.write(0, np.arange(PROMPT), self.fresh(PROMPT))
        self.d_pool.copy_(torch.from_numpy(self.pool))
        self.d_prefix.copy_(self.d_table[0, :PREFIX // 64])
        self.d_refs[self.d_prefix.long()] += 1  # the server's own hold of the prefix
        self.refs[self.table[0, :PREFIX // 64]] += 1

    def fork(self, src, dst):
        import torch

        t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        dsa.pages_fork(self.p, t(src), t(dst), self.d_table, self.d_ctx, self.d_refs, self.ws)
        assert S.pages_fork(self.table, self.ctx, self.refs, src, dst) == 0

    def attend(self):
        dsa.prefix_mla_decode(self.p, self.d_q, self.d_pool, self.d_prefix, PREFIX, self.d_table, self.d_ctx, self.d_out,
                              self.d_lse, self.ws)

    def launch(self):
        """A step's calls, all on the device (so that a graph can hold them)."""
        import torch

        torch.add(self.d_ctx, N_Q, out=self.d_grow)
        dsa.pages_resize(self.p, self.d_grow, self.pools, self.d_table, self.d_ctx, self.d_refs, self.ws)
        pos = self.d_ctx[:, None].long() - N_Q + torch.arange(N_Q, device="cuda")
        rows = self.d_table.long().gather(1, pos // 64) * 64 + pos % 64
        self.d_pool.view(-1, self.row).index_copy_(0, rows.flatten(), self.d_latents)
        self.attend()
        dsa.verify_draft(self.p, self.d_target, self.d_draft, self.d_tokens, None, self.d_uniforms, self.d_ctx, self.d_acc,
                         self.d_next, self.d_new, self.ws)
        dsa.pages_resize(self.p, self.d_new, self.pools, self.d_table, self.d_ctx, self.d_refs, self.ws)

    def step(self, run, bold=False):
        """bold: drafts that the draft model prefers to the target, tested against all of [0, 1)."""
        import torch

        rng, soft = self.rng, lambda x: (np.exp(x) / np.exp(x).sum(-1, keepdims=True)).astype(np.float32)
        logits = rng.standard_normal((B, N_Q, VOCAB)) * 2
        target = soft(logits)
        draft = soft(logits[:, :N_Q - 1] + rng.standard_normal((B, N_Q - 1, VOCAB)))
        tokens = rng.integers(0, VOCAB, (B, N_Q - 1)).astype(np.int32)
        tokens[::2] = target[::2, :N_Q - 1].argmax(-1)
        uniforms = rng.random((B, N_Q)).astype(np.float32)
        if bold:
            tokens = (draft - target[:, :N_Q - 1]).argmax(-1).astype(np.int32)
        else:
            uniforms *= np.array([0.3, 0.6, 1.0], np.float32)
        latents = self.fresh(B * N_Q)
        q = gen.f32_to_bf16_bits(rng.standard_normal((B, N_Q, 96, 576)).astype(np.float32))
        for d, h in ((self.d_target, target), (self.d_draft, draft), (self.d_tokens, tokens), (self.d_uniforms, uniforms),
                     (self.d_latents, latents), (self.d_q.view(torch.int16), q.view(np.int16))):
            d.copy_(torch.from_numpy(np.ascontiguousarray(h)))
        run()
        assert dsa.get_device_error(self.ws) == 0

        assert S.pages_resize(self.table, self.ctx, self.refs, self.ctx + N_Q, [self.pool]) == 0
        for b in range(B):
            self.write(b, self.ctx[b] - N_Q + np.arange(N_Q), latents[b * N_Q:][:N_Q])
        inp = dataclasses.replace(self.inp, ctx=self.ctx.copy(), block_table=self.table.copy(), lat_pool=self.pool, q=q)
        out, lse = bf16_to_np(self.d_out), self.d_lse.cpu().numpy()
        for b in range(B):
            for t in range(N_Q):
                check_row(inp, self.d_prefix.cpu().numpy(), PREFIX, b, t, out[b * N_Q + t], lse[b * N_Q + t])
        acc, nxt, new, err = S.verify_draft(target, draft, tokens, None, uniforms, self.ctx)
        assert err == 0
        assert (self.d_acc.cpu().numpy() == acc).all() and (self.d_next.cpu().numpy() == nxt).all()
        assert S.pages_resize(self.table, self.ctx, self.refs, new, [self.pool]) == 0
        self.same()
        return acc

    def same(self):
        assert (self.d_ctx.cpu().numpy() == self.ctx).all() and (self.d_refs.cpu().numpy() == self.refs).all()
        assert (self.d_table.cpu().numpy() == self.table).all()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("lat_fmt", ["fp8", "nvfp4"])
def test_a_server_of_speculative_steps(lat_fmt, captured):
    import torch

    s = Server(lat_fmt)
    s.prompt()
    s.fork([0, 0, 0], [1, 2, 3])
    assert s.refs[s.table[0, 0]] == B + 1
    accepted = [s.step(s.launch)]  # copies the open page for three of the four
    run = s.launch
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.launch()
        run = graph.replay
    accepted += [s.step(run) for _ in range(3)] + [s.step(run, bold=True) for _ in range(3)]
    assert len(set(np.concatenate(accepted).tolist())) > 1  # drafts passed and did not

    # request 0 ends; the pools are packed, and attention over the moved pages gives the same bits
    s.resize([0] + [-1] * (B - 1))
    s.attend()
    before = s.d_out.clone(), s.d_lse.clone()
    assert dsa.get_device_error(s.ws) == dsa.DSA_DEVERR_CTX  # the empty slot's rows
    where = torch.full((s.inp.num_pages,), -7, dtype=torch.int32, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.pages_compact(s.p, s.pools, s.d_table, s.d_ctx, s.d_refs, where, live, s.ws)
    ref_where, ref_live, err = S.pages_compact(s.table, s.ctx, s.refs, [s.pool])
    assert err == 0 and (where.cpu().numpy() == ref_where).all() and live.item() == ref_live
    s.same()
    s.d_prefix.copy_(where[s.d_prefix.long()])
    s.attend()
    assert dsa.get_device_error(s.ws) == dsa.DSA_DEVERR_CTX
    assert torch.equal(before[0].view(torch.int16), s.d_out.view(torch.int16)) and torch.equal(before[1], s.d_lse)

    # its slot goes on as a fork of another
    s.fork([2], [0])
    for bold in (False, True):
        s.step(run, bold)
    s.resize([0] * B)
    s.same()
    assert (s.refs > 0).sum() == PREFIX // 64


def test_operators_between_decode_steps_on_one_workspace():
    """The fused step, the front end's counters and the serving operators take turns on one workspace whose room they
    share: every step gives the bits of the first."""
    import torch

    from dsa_testlib import Dev

    inp = gen.make_inputs(12, 1, [3000, 700, 64, 65, 900, 2300, 128, 1, 400, 2049, 77, 1500], seed=50, bt_mode="permuted")
    d = Dev(inp)
    own = dsa.make_params(batch=12, n_q=1, max_pages_per_req=inp.max_pages, num_pages=1, key_page_stride=8448,
                          lat_page_stride=36864)
    assert d.ws.numel() == dsa.workspace_size(own)  # no room beyond the decode step's
    first = [x.clone() for x in d.decode()]
    z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")
    table, ctx, refs = z(12, inp.max_pages), z(12), z(inp.num_pages)
    lens = torch.arange(12, dtype=torch.int32, device="cuda") * 70
    pools = dsa.make_pools([])
    out, lse = z(12, 96, 512, dtype=torch.bfloat16), z(12, 96, dtype=torch.float32)
    target, acc, tok = torch.full((12, 1, 50), 0.02, device="cuda"), z(12), z(12, 1)
    got = []
    for _ in range(3):
        dsa.prefix_mla_decode(d.p, d.q, d.lat_pool, None, 0, d.block_table, d.ctx, out, lse, d.ws)
        got.append(out.clone())
        got += [x.clone() for x in d.decode()]
        dsa.pages_resize(d.p, lens, pools, table, ctx, refs, d.ws)
        dsa.pages_compact(d.p, pools, table, ctx, refs, None, None, d.ws)
        got += [out.clone()] + [x.clone() for x in d.decode()]
        dsa.verify_draft(d.p, target, None, None, None, z(12, 1, dtype=torch.float32), None, acc, tok, None, d.ws[:256])
    assert dsa.get_device_error(d.ws) == 0
    for i, x in enumerate(got):
        assert torch.equal(x, got[0] if i % 4 == 0 else first[i % 4 - 1]), i
    assert (ctx == lens).all() and (refs > 0).sum() == sum(-(-70 * i // 64) for i in range(12))
