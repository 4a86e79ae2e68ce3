"""Cases of the serving operators around the decode step: attention of a batch
that shares a prefix, the cache's page operations, and the verification of
drafted tokens. Each case can be run in a plain form (elementary torch
operations, 32 bits, or 64 where 32 lose what matters) or through the library.

Kinds of case and their fields:
  attn     batch, n_q, prefix (tokens, whole pages), tail (the longest private
           part), fmt ("fp8" or "nvfp4" latents)
  verify   batch, n_q (drafts + 1), vocab, dtype, ragged (draft counts differ),
           drafts ("sampled" with draft probabilities, "given" without)
  resize   batch, prefix, tail, layers, grow (the most tokens a request gains);
           a third of the requests shrink, some to nothing
  fork     batch, ctx: one request is forked into all the other slots
  compact  batch, prefix, tail, layers, spread (pool pages per page in use)
"""
import math
import random

import numpy as np
import torch

own = False

HEADS, D_NOPE, D_ROPE, PAGE = 96, 512, 64, 64
D_QK = D_NOPE + D_ROPE
ROW_BYTES = {"fp8": 576, "nvfp4": 352}
SCALE = 1.0 / 192 ** 0.5
LATENT_SCALE = 0.75
KEY_PAGE, LAT_PAGE = PAGE * 132, PAGE * 576
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one request on a short cached system prompt: the latency of a call
        {"name": "attn_b1_4k", "kind": "attn", "batch": 1, "n_q": 1, "prefix": 4096, "tail": 50, "fmt": "fp8"},
        # eight requests on one document, five drafted tokens each, 4-bit latents
        {"name": "attn_b8x6_16k_nvfp4", "kind": "attn", "batch": 8, "n_q": 6, "prefix": 16384, "tail": 700, "fmt": "nvfp4"},
        # many samples of one prompt
        {"name": "attn_b64_32k", "kind": "attn", "batch": 64, "n_q": 1, "prefix": 32768, "tail": 1900, "fmt": "fp8"},
        # a few agents on one very long context
        {"name": "attn_b13x2_256k", "kind": "attn", "batch": 13, "n_q": 2, "prefix": 262144, "tail": 333, "fmt": "fp8"},
        # nothing shared: dense attention of every request over its own context
        {"name": "attn_b24_own_8k", "kind": "attn", "batch": 24, "n_q": 1, "prefix": 0, "tail": 8111, "fmt": "fp8"},
        # one request's drafts
        {"name": "verify_b1x6_32k", "kind": "verify", "batch": 1, "n_q": 6, "vocab": 32000, "dtype": "f32", "ragged": False, "drafts": "sampled"},
        # a serving batch over a large vocabulary
        {"name": "verify_b64x6_128k", "kind": "verify", "batch": 64, "n_q": 6, "vocab": 131072, "dtype": "f32", "ragged": False, "drafts": "sampled"},
        # a full batch, an odd vocabulary, drafts of different lengths
        {"name": "verify_b256x8_100k_bf16", "kind": "verify", "batch": 256, "n_q": 8, "vocab": 100003, "dtype": "bf16", "ragged": True, "drafts": "sampled"},
        # one decode step's bookkeeping for a small batch, one layer's pools
        {"name": "resize_b8", "kind": "resize", "batch": 8, "prefix": 2048, "tail": 900, "layers": 1, "grow": 6},
        # the first step after a prompt was forked 192 times: the open page of every request is copied, eight layers
        {"name": "resize_b192_x8", "kind": "resize", "batch": 192, "prefix": 16416, "tail": 0, "layers": 8, "grow": 70},
        # a prompt of 128 K tokens forked into every slot
        {"name": "fork_b96_128k", "kind": "fork", "batch": 96, "ctx": 131041},
        # a fragmented pool packed to its front, eight layers
        {"name": "compact_b64_x8", "kind": "compact", "batch": 64, "prefix": 8192, "tail": 1500, "layers": 8, "spread": 2.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "verify", "resize", "fork", "compact"])
    if kind == "attn":
        while True:
            c = {"kind": kind, "batch": _log(rng, 1, 64), "n_q": rng.choice([1, 1, 2, 3, 4, 6, 8]),
                 "prefix": PAGE * rng.choice([0, _log(rng, 1, 4096), _log(rng, 1, 4096), _log(rng, 1, 4096)]),
                 "tail": _log(rng, 8, 8191), "fmt": rng.choice(["fp8", "fp8", "nvfp4"])}
            if work(c)["flops"] <= 7e11:
                return c
    if kind == "verify":
        while True:
            c = {"kind": kind, "batch": _log(rng, 1, 256), "n_q": rng.randint(1, 8), "vocab": _log(rng, 500, 131072),
                 "dtype": rng.choice(["f32", "f32", "bf16", "f16"]), "ragged": rng.random() < 0.5,
                 "drafts": rng.choice(["sampled", "sampled", "given"])}
            if c["batch"] * c["vocab"] <= 256 * 100003:
                return c
    if kind == "fork":
        return {"kind": kind, "batch": _log(rng, 2, 96), "ctx": _log(rng, 1, 131041)}
    c = {"kind": kind, "batch": _log(rng, 1, 192), "prefix": _log(rng, 1, 16384), "tail": _log(rng, 1, 1500)}
    c["layers"] = rng.choice([1, 2, 4, 8])
    if kind == "resize":
        c["grow"] = _log(rng, 1, 128)
    else:
        c["batch"] = min(c["batch"], 64)
        c["spread"] = round(rng.uniform(1.05, 2.0), 2)
    return c


# ---------------------------------------------------------------- sizes that follow from a case


def _tails(c):
    """Private tokens of each request (its new tokens among them): the longest
    first, the others spread down to n_q."""
    r = random.Random(c["batch"] * 1009 + c["tail"])
    hi = max(c["tail"], c["n_q"])
    return [hi] + [r.randint(c["n_q"], hi) for _ in range(c["batch"] - 1)]


def _old_lens(c):
    """Context lengths of a page case before the call."""
    r = random.Random(c["batch"] * 1013 + c["tail"])
    return [c["prefix"] + (r.randint(0, c["tail"]) if c["tail"] else 0) for _ in range(c["batch"])]


def _new_lens(c):
    r = random.Random(c["batch"] * 1019 + c["grow"])
    out = []
    for b, n in enumerate(_old_lens(c)):
        if c["tail"] and b % 3 == 1:  # rejected drafts, an ended request, a rollback
            out.append(r.choice([max(0, n - r.randint(0, 8)), 0, r.randint(0, n)]))
        else:
            out.append(n + r.randint(1, c["grow"]))
    return out


def _pages(n):
    return -(-n // PAGE)


def work(c):
    if c["kind"] == "attn":
        rows = c["batch"] * c["n_q"]
        tails = _tails(c)
        pairs = rows * c["prefix"] + sum(c["n_q"] * t - c["n_q"] * (c["n_q"] - 1) // 2 for t in tails)
        return {"bytes": (c["prefix"] + sum(tails)) * ROW_BYTES[c["fmt"]] + rows * HEADS * (2 * D_QK + 2 * D_NOPE + 4),
                "flops": 2 * (D_QK + D_NOPE) * HEADS * pairs}
    if c["kind"] == "verify":
        size = 4 if c["dtype"] == "f32" else 2
        rows = 2 if c["n_q"] > 1 and c["drafts"] == "sampled" else 1
        return {"bytes": c["batch"] * (rows * c["vocab"] * size + c["n_q"] * 20), "flops": c["batch"] * rows * c["vocab"]}
    page = c.get("layers", 0) * (KEY_PAGE + LAT_PAGE)
    if c["kind"] == "fork":
        return {"bytes": 4 * _pages(c["ctx"]) * (c["batch"] - 1) + 8 * _pages(c["ctx"]), "flops": 0}
    old = _old_lens(c)
    shared = c["prefix"] // PAGE
    if c["kind"] == "resize":
        new = _new_lens(c)
        moved = sum(c["batch"] > 1 and m > n and n % PAGE != 0 and n == c["prefix"] for n, m in zip(old, new))
        changed = sum(abs(_pages(n) - _pages(m)) for n, m in zip(old, new))
        return {"bytes": 2 * moved * page + 8 * changed + 4 * _num_pages(c) + 12 * c["batch"], "flops": 0}
    live = shared + sum(_pages(n) - shared for n in old)
    moved = live * (1 - 1 / c["spread"])
    return {"bytes": 2 * moved * page + 8 * _num_pages(c) + 4 * sum(_pages(n) for n in old), "flops": 0}


def _num_pages(c):
    shared = c["prefix"] // PAGE
    live = shared + sum(_pages(n) - shared for n in _old_lens(c))
    if c["kind"] == "compact":
        return int(live * c["spread"]) + 1
    return live + c["batch"] * (2 + c["grow"] // PAGE) + 16


# ---------------------------------------------------------------- inputs


def _normal_e4m3(g, n):
    return torch.randn(n, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)


def _latent_pool(g, num_pages, fmt):
    rows = num_pages * PAGE
    if fmt == "fp8":
        return _normal_e4m3(g, (rows, 576)).view(num_pages, PAGE * 576)
    pool = torch.empty(rows, 352, dtype=torch.uint8, device="cuda")
    pool[:, :256] = torch.randint(0, 256, (rows, 256), generator=g, device="cuda", dtype=torch.uint8)
    pool[:, 256:288] = (torch.rand(rows, 32, generator=g, device="cuda") * 0.5 + 0.1).to(torch.float8_e4m3fn).view(torch.uint8)
    pool[:, 288:] = _normal_e4m3(g, (rows, 64))
    return pool.view(num_pages, PAGE * 352)


def _prepare_attn(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    tails = _tails(c)
    shared = c["prefix"] // PAGE
    counts = [_pages(c["prefix"] + t) - shared for t in tails]
    num_pages = shared + sum(counts) + 3
    perm = rng.permutation(num_pages).astype(np.int32)
    table = np.full((c["batch"], shared + max(counts)), -1, np.int32)
    table[:, :shared] = perm[:shared]
    at = shared
    for b, n in enumerate(counts):
        table[b, shared:shared + n] = perm[at:at + n]
        at += n
    rows = c["batch"] * c["n_q"]
    s = {"case": c, "lat": _latent_pool(g, num_pages, c["fmt"]),
         "q": torch.randn(rows, HEADS, D_QK, generator=g, device="cuda").to(torch.bfloat16),
         "table": torch.from_numpy(table).cuda(), "prefix_pages": torch.from_numpy(perm[:shared].copy()).cuda(),
         "ctx": torch.tensor([c["prefix"] + t for t in tails], dtype=torch.int32, device="cuda"),
         "out": torch.empty(rows, HEADS, D_NOPE, dtype=torch.bfloat16, device="cuda"),
         "lse": torch.empty(rows, HEADS, dtype=torch.float32, device="cuda")}
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        s["params"] = dsa.make_params(
            batch=c["batch"], n_q=c["n_q"], max_pages_per_req=table.shape[1], num_pages=num_pages, key_page_stride=KEY_PAGE,
            lat_page_stride=PAGE * ROW_BYTES[c["fmt"]], lat_fmt=dsa.DSA_LAT_FP8_576 if c["fmt"] == "fp8" else dsa.DSA_LAT_NVFP4_352,
            softmax_scale=SCALE, latent_scale=LATENT_SCALE)
        s["ws"] = torch.zeros(dsa.workspace_size(s["params"]), dtype=torch.uint8, device="cuda")
    return s


def _prepare_verify(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, n, V = c["batch"], c["n_q"], c["vocab"]
    dt = DTYPES[c["dtype"]]
    logits = torch.randn(B, n, V, generator=g, device="cuda") * 2.5
    s = {"case": c, "target": torch.softmax(logits, -1).to(dt), "draft": None}
    if n > 1:
        q = torch.softmax(logits[:, :-1] + 0.7 * torch.randn(B, n - 1, V, generator=g, device="cuda"), -1)
        s["tokens"] = torch.multinomial(q.view(-1, V), 1, generator=g).view(B, n - 1).to(torch.int32)
        if c["drafts"] == "sampled":
            s["draft"] = q.to(dt)
        else:  # drafts that often agree with the target, as copied text does
            likely = s["target"][:, :-1].argmax(-1).to(torch.int32)
            s["tokens"] = torch.where(torch.rand(B, n - 1, generator=g, device="cuda") < 0.8, likely, s["tokens"])
    else:
        s["tokens"] = torch.zeros(B, 0, dtype=torch.int32, device="cuda")
    s["counts"] = torch.randint(0, n, (B,), generator=g, device="cuda", dtype=torch.int32) if c["ragged"] else None
    s["uniforms"] = torch.rand(B, n, generator=g, device="cuda")
    s["ctx"] = torch.randint(n, 100000, (B,), generator=g, device="cuda", dtype=torch.int32)
    s["accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
    s["out"] = torch.empty(B, n, dtype=torch.int32, device="cuda")
    s["new_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        s["params"] = dsa.make_params(batch=B, n_q=n, max_pages_per_req=1600, num_pages=1600, key_page_stride=KEY_PAGE,
                                      lat_page_stride=LAT_PAGE)
        s["ws"] = torch.zeros(dsa.workspace_size(s["params"]), dtype=torch.uint8, device="cuda")
    return s


def _prepare_pages(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    B = c["batch"]
    if c["kind"] == "fork":
        n = _pages(c["ctx"])
        num_pages, width = n + 64, n
        perm = rng.permutation(num_pages).astype(np.int32)
        table = np.full((B, width), -1, np.int32)
        lens, refs = np.zeros(B, np.int32), np.zeros(num_pages, np.int32)
        src = int(rng.integers(B))
        table[src, :n], lens[src], refs[perm[:n]] = perm[:n], c["ctx"], 1
    else:
        old = _old_lens(c)
        # every request holds the whole pages of the prefix; a request whose
        # context ends with the prefix shares its open page too
        shared = c["prefix"] // PAGE
        num_pages = _num_pages(c)
        width = max(_pages(max(n, m)) for n, m in zip(old, _new_lens(c) if c["kind"] == "resize" else old))
        perm = rng.permutation(num_pages).astype(np.int32)
        table = np.full((B, max(width, 1)), -1, np.int32)
        lens, refs = np.array(old, np.int32), np.zeros(num_pages, np.int32)
        at, open_page = shared, -1
        for b, n in enumerate(old):
            table[b, :shared] = perm[:shared]
            if n == c["prefix"] and n % PAGE:
                if open_page < 0:
                    open_page, at = at, at + 1
                table[b, shared] = perm[open_page]
            else:
                k = _pages(n) - shared
                table[b, shared:shared + k] = perm[at:at + k]
                at += k
            np.add.at(refs, table[b, :_pages(n)], 1)
    width = table.shape[1]
    start = torch.from_numpy(np.concatenate([table.ravel(), lens, refs])).cuda()
    cur = start.clone()
    s = {"case": c, "start": start, "cur": cur, "table": cur[:B * width].view(B, width), "ctx": cur[B * width:B * width + B],
         "refs": cur[B * width + B:], "pools": []}
    if c["kind"] == "fork":
        others = rng.permutation([b for b in range(B) if b != src]).astype(np.int32)
        s["src"] = torch.full((B - 1,), src, dtype=torch.int32, device="cuda")
        s["dst"] = torch.from_numpy(others).cuda()
    else:
        for size in (KEY_PAGE, LAT_PAGE):
            s["pools"].append(torch.randint(-2 ** 31, 2 ** 31, (num_pages, c["layers"] * size // 4), generator=g, device="cuda",
                                            dtype=torch.int32))
    if c["kind"] == "resize":
        s["new_lens"] = torch.tensor(_new_lens(c), dtype=torch.int32, device="cuda")
    if c["kind"] == "compact":
        s["map"] = torch.empty(num_pages, dtype=torch.int32, device="cuda")
        s["live"] = torch.empty(1, dtype=torch.int32, device="cuda")
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        s["params"] = dsa.make_params(batch=B, n_q=1, max_pages_per_req=width, num_pages=num_pages, key_page_stride=KEY_PAGE,
                                      lat_page_stride=LAT_PAGE)
        s["ws"] = torch.zeros(dsa.workspace_size(s["params"]), dtype=torch.uint8, device="cuda")
        s["plan"] = dsa.make_pools([(p, p.shape[1] * 4, p.shape[1] * 4) for p in s["pools"]])
    return s


def prepare(case, seed):
    if case["kind"] == "attn":
        return _prepare_attn(case, seed)
    if case["kind"] == "verify":
        return _prepare_verify(case, seed)
    return _prepare_pages(case, seed)


# ---------------------------------------------------------------- one pass


def run(s):
    kind = s["case"]["kind"]
    if kind == "attn":
        return _attn(s)
    if kind == "verify":
        return _verify(s)
    s["cur"].copy_(s["start"])  # the page operations change their state in place
    return {"resize": _resize, "fork": _fork, "compact": _compact}[kind](s)


def _decode(rows, fmt):
    """Latents [n, 576] in 32 bits of n rows of the pool."""
    if fmt == "fp8":
        return rows.view(torch.float8_e4m3fn).float()
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)
    nib = torch.stack([rows[:, :256] & 15, rows[:, :256] >> 4], -1).view(-1, 512)
    scale = rows[:, 256:288].contiguous().view(torch.float8_e4m3fn).float()
    nope = lut[nib.long()].view(-1, 32, 16) * scale[:, :, None]
    return torch.cat([nope.view(-1, 512), rows[:, 288:].contiguous().view(torch.float8_e4m3fn).float()], 1)


def _attn(s):
    c = s["case"]
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        dsa.prefix_mla_decode(s["params"], s["q"], s["lat"], s["prefix_pages"], c["prefix"], s["table"], s["ctx"], s["out"],
                              s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    B, n, P, fmt = c["batch"], c["n_q"], c["prefix"], c["fmt"]
    shared = P // PAGE
    pool = s["lat"].view(-1, PAGE * ROW_BYTES[fmt])
    q = s["q"].float() * SCALE
    # the shared part: one product for the whole batch
    pre = _decode(pool[s["prefix_pages"].long()].view(P, ROW_BYTES[fmt]), fmt) * LATENT_SCALE
    lp = (q.view(-1, D_QK) @ pre.T).view(B, n, HEADS, P)
    # the private part, padded to the longest
    own_pages = s["table"][:, shared:].long()
    M = own_pages.shape[1] * PAGE
    tail = _decode(pool[own_pages.clamp(min=0)].view(B * M, ROW_BYTES[fmt]), fmt).view(B, M, D_QK) * LATENT_SCALE
    pos = P + torch.arange(M, device="cuda")
    seen = s["ctx"].long()[:, None] - n + 1 + torch.arange(n, device="cuda")
    hide = pos[None, None, :] >= seen[:, :, None]
    tail = tail.masked_fill(hide[:, -1, :, None], 0.0)
    lt = (q.view(B, n * HEADS, D_QK) @ tail.transpose(1, 2)).view(B, n, HEADS, M).masked_fill(hide[:, :, None, :], -math.inf)
    m = lt.amax(-1, keepdim=True)
    if P:
        m = torch.maximum(m, lp.amax(-1, keepdim=True))
    lt = torch.exp(lt - m)
    total = lt.sum(-1, keepdim=True)
    out = (lt.view(B, n * HEADS, M) @ tail[:, :, :D_NOPE]).view(B, n, HEADS, D_NOPE)
    if P:
        lp = torch.exp(lp - m)
        total = total + lp.sum(-1, keepdim=True)
        out = out + (lp.view(-1, P) @ pre[:, :D_NOPE]).view(B, n, HEADS, D_NOPE)
    out = out / total
    lse = (m + torch.log(total)).view(B * n, HEADS)
    return {"out": out.view(B * n, HEADS, D_NOPE).to(torch.bfloat16), "lse": lse}


def _verify(s):
    c = s["case"]
    B, n, V = c["batch"], c["n_q"], c["vocab"]
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        dsa.verify_draft(s["params"], s["target"], s["draft"], s["tokens"], s["counts"], s["uniforms"], s["ctx"], s["accepted"],
                         s["out"], s["new_lens"], s["ws"])
        return {"accepted": s["accepted"], "tokens": s["out"], "new_lens": s["new_lens"]}
    idx = torch.arange(n, device="cuda")
    if n > 1:
        tok = s["tokens"].long()
        px = s["target"][:, :-1].gather(2, tok[:, :, None])[:, :, 0].double()
        u = s["uniforms"][:, :-1].double()
        if s["draft"] is None:
            yes = u < px
        else:
            yes = u * s["draft"].gather(2, tok[:, :, None])[:, :, 0].double() < px
        counts = torch.full((B,), n - 1, device="cuda") if s["counts"] is None else s["counts"].long()
        yes = yes & (idx[:-1] < counts[:, None])
        a = yes.long().cumprod(1).sum(1)
    else:
        counts = a = torch.zeros(B, dtype=torch.long, device="cuda")
    p = s["target"][torch.arange(B, device="cuda"), a].double()
    w = p
    if n > 1:
        at = a.clamp(max=n - 2)
        rejected = (a < counts)[:, None]
        here = torch.arange(B, device="cuda")
        if s["draft"] is None:
            q = torch.zeros_like(p).scatter_(1, s["tokens"].long()[here, at][:, None], math.inf)
        else:
            q = s["draft"][here, at].double()
        w = torch.where(rejected, (p - q).clamp(min=0.0), p)
        w = torch.where(w.sum(1, keepdim=True) > 0, w, p)
    cum = w.cumsum(1)
    drawn = torch.searchsorted(cum, s["uniforms"][:, -1:].double() * cum[:, -1:], right=True).clamp(max=V - 1)
    padded = torch.cat([s["tokens"].long(), drawn], 1)
    out = torch.where(idx < a[:, None], padded, torch.where(idx == a[:, None], drawn, -1))
    return {"accepted": a.to(torch.int32), "tokens": out.to(torch.int32), "new_lens": (s["ctx"] - n + 1 + a).to(torch.int32)}


def _resize(s):
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        dsa.pages_resize(s["params"], s["new_lens"], s["plan"], s["table"], s["ctx"], s["refs"], s["ws"])
        return {"table": s["table"], "ctx": s["ctx"], "refs": s["refs"], "pools": s["pools"]}
    table, ctx, refs = s["table"], s["ctx"], s["refs"]
    old, new = ctx.long(), s["new_lens"].long()
    have, want = (old + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    j = torch.arange(table.shape[1], device="cuda")
    last = (old // PAGE).clamp(max=table.shape[1] - 1)[:, None]
    open_page = table.long().gather(1, last)[:, 0]
    grows = new > old
    copy = grows & (old % PAGE != 0) & (refs[open_page.clamp(min=0)] > 1)
    need = torch.where(grows, want - have + copy, 0)
    upto = need.cumsum(0)
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)
    ok = (need == 0) | (upto <= (refs == 0).sum())
    first = upto - need + copy  # rank of the first page appended
    add = (grows & ok)[:, None] & (j >= have[:, None]) & (j < want[:, None])
    drop = (new < old)[:, None] & (j >= want[:, None]) & (j < have[:, None])
    rank = (first[:, None] + j - have[:, None]).clamp(0, free.numel() - 1)
    refs.index_add_(0, table.long()[drop], torch.full_like(table[drop], -1))
    table.copy_(torch.where(add, free[rank].to(torch.int32), torch.where(drop, -1, table)))
    refs[table.long()[add]] = 1
    who = (copy & ok).nonzero()[:, 0]
    src, dst = open_page[who], free[(upto - need)[who]]
    table[who, last[who, 0]] = dst.to(torch.int32)
    refs[dst] = 1
    refs.index_add_(0, src, torch.full_like(src, -1, dtype=torch.int32))
    for pool in s["pools"]:
        pool[dst] = pool[src]
    ctx.copy_(torch.where(ok, new, old).to(torch.int32))
    return {"table": table, "ctx": ctx, "refs": refs, "pools": s["pools"]}


def _fork(s):
    table, ctx, refs = s["table"], s["ctx"], s["refs"]
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        dsa.pages_fork(s["params"], s["src"], s["dst"], table, ctx, refs, s["ws"])
        return {"table": table, "ctx": ctx, "refs": refs}
    src, dst = s["src"].long(), s["dst"].long()
    used = torch.arange(table.shape[1], device="cuda") < ((ctx[src].long() + PAGE - 1) // PAGE)[:, None]
    rows = table[src]
    table[dst] = torch.where(used, rows, table[dst])
    ctx[dst] = ctx[src]
    refs.index_add_(0, rows[used].long(), torch.ones_like(rows[used]))
    return {"table": table, "ctx": ctx, "refs": refs}


def _compact(s):
    table, ctx, refs = s["table"], s["ctx"], s["refs"]
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        dsa.pages_compact(s["params"], s["plan"], table, ctx, refs, s["map"], s["live"], s["ws"])
        return {"table": table, "ctx": ctx, "refs": refs, "map": s["map"], "live": s["live"], "pools": s["pools"]}
    page = torch.arange(refs.numel(), device="cuda")
    used = refs > 0
    live = used.sum()
    src = page[used & (page >= live)]
    dst = page[~used & (page < live)]
    where = torch.where(used, page, -1)
    where[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    for pool in s["pools"]:
        pool[dst] = pool[src]
    mine = torch.arange(table.shape[1], device="cuda") < ((ctx.long() + PAGE - 1) // PAGE)[:, None]
    table.copy_(torch.where(mine, where[table.long().clamp(min=0)].to(torch.int32), table))
    return {"table": table, "ctx": ctx, "refs": refs, "map": where.to(torch.int32), "live": live.to(torch.int32)[None],
            "pools": s["pools"]}


# ---------------------------------------------------------------- the definition in 64 bits


def _values(rows, fmt):
    """Latents of raw rows in 64 bits, from the formats' bit fields."""
    def e4m3(x):
        x = x.long()
        e, f = (x >> 3) & 15, (x & 7).double()
        mag = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2((e - 10).double()))
        return torch.where(x >= 128, -mag, mag)

    if fmt == "fp8":
        return e4m3(rows)
    table = torch.tensor(E2M1, dtype=torch.float64, device=rows.device)
    codes = torch.empty(rows.shape[0], 512, dtype=torch.long, device=rows.device)
    codes[:, 0::2], codes[:, 1::2] = (rows[:, :256] & 15).long(), (rows[:, :256] >> 4).long()
    nope = table[codes & 7] * torch.where(codes >= 8, -1.0, 1.0).double()
    return torch.cat([nope * e4m3(rows[:, 256:288]).repeat_interleave(16, 1), e4m3(rows[:, 288:])], 1)


def exact(case, seed):
    if case["kind"] != "attn":
        return None  # whole numbers only
    s = _prepare_attn(case, seed)
    fmt, n = case["fmt"], case["n_q"]
    out, lse = [], []
    rows = s["lat"].view(-1, PAGE, ROW_BYTES[fmt])
    pre = _values(rows[s["prefix_pages"].long()].reshape(case["prefix"], ROW_BYTES[fmt]), fmt) * LATENT_SCALE
    for b, ctx in enumerate(s["ctx"].tolist()):
        mine = s["table"][b, case["prefix"] // PAGE:_pages(ctx)].long()
        tail = _values(rows[mine].reshape(len(mine) * PAGE, ROW_BYTES[fmt]), fmt) * LATENT_SCALE
        for t in range(n):
            c = torch.cat([pre, tail[:ctx - n + t + 1 - case["prefix"]]])
            z = (s["q"][b * n + t].double() @ c.T) * SCALE
            z_lse = torch.logsumexp(z, 1)
            lse.append(z_lse)
            out.append(torch.exp(z - z_lse[:, None]) @ c[:, :D_NOPE])
    return {"out": torch.stack(out), "lse": torch.stack(lse)}
