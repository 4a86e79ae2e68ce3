"""Cases of the operators of a bounded latent cache: the attention's front end (norms, rotation and
the write into the cache), attention with a sliding window and sinks, the accumulated attention
weight of every cached token, and eviction by it. Each case can be run in a plain form (elementary
torch operations, 32 bits, or 64 where 32 lose what matters) or through the library.

Kinds of case and their fields:
  latent   batch, n_q, fmt ("fp8" or "nvfp4" latents), norm_q (the query heads are normalised too),
           interleaved (rotation pairs (2i, 2i + 1), else (i, i + 32)), far (positions of their own, up
           to a million, else the cache slots)
  window   batch, n_q, sinks, window, longest (the longest context), fmt
  mass     batch, n_q, sinks, window, longest, fmt
  evict    batch, longest, budget (tokens a request may keep), sinks, recent, prefix (first tokens,
           whole pages, whose pages all requests share), layers; every fifth request is left alone
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
EPS = 1e-6
KEY_PAGE, LAT_PAGE = PAGE * 132, PAGE * 576
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of one request: the latency of a call
        {"name": "latent_b1", "kind": "latent", "batch": 1, "n_q": 1, "fmt": "fp8", "norm_q": False, "interleaved": True, "far": False},
        # a speculative step of a serving batch on a cache that tokens were evicted from, 4-bit latents
        {"name": "latent_b64x6_nvfp4", "kind": "latent", "batch": 64, "n_q": 6, "fmt": "nvfp4", "norm_q": True, "interleaved": False, "far": True},
        # a chunk of two long prompts
        {"name": "latent_b2x4097", "kind": "latent", "batch": 2, "n_q": 4097, "fmt": "fp8", "norm_q": True, "interleaved": True, "far": False},
        # one request that streams
        {"name": "window_b1_1k", "kind": "window", "batch": 1, "n_q": 1, "sinks": 4, "window": 1024, "longest": 50000, "fmt": "fp8"},
        # a serving batch of long conversations
        {"name": "window_b64_4k", "kind": "window", "batch": 64, "n_q": 1, "sinks": 64, "window": 4096, "longest": 131072, "fmt": "fp8"},
        # chunks of three prompts, an odd window, 4-bit latents
        {"name": "window_b3x333_2k_nvfp4", "kind": "window", "batch": 3, "n_q": 333, "sinks": 5, "window": 2049, "longest": 9000, "fmt": "nvfp4"},
        # one request's step
        {"name": "mass_b1_4k", "kind": "mass", "batch": 1, "n_q": 1, "sinks": 0, "window": 4100, "longest": 4100, "fmt": "fp8"},
        # a serving batch, all of its tokens
        {"name": "mass_b40_16k", "kind": "mass", "batch": 40, "n_q": 1, "sinks": 0, "window": 16384, "longest": 16384, "fmt": "fp8"},
        # the last rows of a few prompts judge the tokens before them, 4-bit latents
        {"name": "mass_b6x8_20k_nvfp4", "kind": "mass", "batch": 6, "n_q": 8, "sinks": 16, "window": 20001, "longest": 30000, "fmt": "nvfp4"},
        # a small batch over its budget, one layer's pools
        {"name": "evict_b4_4k", "kind": "evict", "batch": 4, "longest": 4096, "budget": 2048, "sinks": 4, "recent": 256, "prefix": 0, "layers": 1},
        # a serving batch with a shared prompt, four layers
        {"name": "evict_b48_12k_x4", "kind": "evict", "batch": 48, "longest": 12000, "budget": 8192, "sinks": 64, "recent": 1024, "prefix": 640, "layers": 4},
        # one very long context cut to a quarter
        {"name": "evict_b1_512k", "kind": "evict", "batch": 1, "longest": 524289, "budget": 131072, "sinks": 16, "recent": 4096, "prefix": 0, "layers": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["latent", "window", "window", "mass", "mass", "evict"])
    fmt = rng.choice(["fp8", "fp8", "nvfp4"])
    if kind == "latent":
        while True:
            c = {"kind": kind, "batch": _log(rng, 1, 256), "n_q": rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 4097)]), "fmt": fmt,
                 "norm_q": rng.random() < 0.5, "interleaved": rng.random() < 0.5, "far": rng.random() < 0.5}
            if c["batch"] * c["n_q"] <= 8194:
                return c
    if kind == "evict":
        while True:
            c = {"kind": kind, "batch": _log(rng, 1, 64), "longest": _log(rng, 65, 524289), "layers": rng.choice([1, 1, 2, 4])}
            c["budget"] = _log(rng, 1 + c["longest"] // 8, c["longest"])
            c["sinks"] = rng.choice([0, _log(rng, 1, 200)])
            c["recent"] = rng.choice([0, _log(rng, 1, 2000)])
            c["prefix"] = min(PAGE * rng.choice([0, 0, _log(rng, 1, 30)]), c["longest"] // 2 // PAGE * PAGE)
            if c["batch"] * c["longest"] * c["layers"] <= 48 * 12000 * 4:
                return c
    while True:
        c = {"kind": kind, "batch": _log(rng, 1, 64), "n_q": rng.choice([1, 1, 2, 3, 5, 8]), "sinks": rng.choice([0, _log(rng, 1, 300)]),
             "window": _log(rng, 16, 32768), "fmt": fmt}
        if kind == "window":
            c["n_q"] = rng.choice([c["n_q"], c["n_q"], _log(rng, 9, 400)])
        c["longest"] = max(c["n_q"], _log(rng, c["window"] // 2, 131072))
        if work(c)["flops"] <= 4e11 and c["batch"] * min(c["longest"], c["sinks"] + c["window"] + c["n_q"] + 2 * PAGE) <= 1000000:
            return c


# ---------------------------------------------------------------- sizes that follow from a case


def _lens(c):
    """Context length of each request, its new tokens among them: the longest
    first, the others down to half of it."""
    r = random.Random(c["batch"] * 1009 + c["longest"])
    lo = max(c.get("n_q", 1), c.get("prefix", 0) + 1, c["longest"] // 2)
    return [c["longest"]] + [r.randint(min(lo, c["longest"]), c["longest"]) for _ in range(c["batch"] - 1)]


def _budgets(c):
    return [-1 if b % 5 == 4 else c["budget"] for b in range(c["batch"])]


def _pages(n):
    return -(-n // PAGE)


def _used_pages(c, n):
    """Logical pages of a context of n tokens that some row sees."""
    sinks, first = min(c["sinks"], n), max(0, n - c["n_q"] + 1 - c["window"])
    if first <= sinks:
        return list(range(_pages(n)))
    return sorted(set(range(_pages(sinks))) | set(range(first // PAGE, _pages(n))))


def _pairs(c, n):
    """(row, token) pairs of a context of n tokens, and the tokens that some row sees."""
    seen = [n - c["n_q"] + t + 1 for t in range(c["n_q"])]
    pairs = sum(min(L, min(c["sinks"], max(0, L - c["window"])) + c["window"]) for L in seen)
    first = max(0, seen[0] - c["window"])
    return pairs, n - max(0, first - c["sinks"])


def work(c):
    if c["kind"] == "latent":
        rows = c["batch"] * c["n_q"]
        return {"bytes": rows * (2 * HEADS * D_QK * 2 + D_QK * 2 + ROW_BYTES[c["fmt"]]), "flops": rows * (HEADS + 1) * (4 * D_NOPE + 3 * D_ROPE)}
    if c["kind"] in ("window", "mass"):
        rows = c["batch"] * c["n_q"]
        got = [_pairs(c, n) for n in _lens(c)]
        pairs, tokens = sum(p for p, _ in got), sum(t for _, t in got)
        if c["kind"] == "window":
            return {"bytes": tokens * ROW_BYTES[c["fmt"]] + rows * HEADS * (2 * D_QK + 2 * D_NOPE + 4), "flops": 2 * (D_QK + D_NOPE) * HEADS * pairs}
        return {"bytes": tokens * (ROW_BYTES[c["fmt"]] + 8) + rows * HEADS * (2 * D_QK + 4), "flops": 2 * D_QK * HEADS * pairs}
    moved = read = table = 0
    for n, b in zip(_lens(c), _budgets(c)):
        if 0 <= b < n:
            moved += max(0, b - c["sinks"])  # (the tokens before the first that goes stay, about the sinks)
            read += 4 * (n + b)
            table += 4 * _pages(n)
    return {"bytes": 2 * moved * c["layers"] * (132 + 576) + 2 * read + table, "flops": 0}


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


def _tables(rng, used, width):
    """Block table of requests that hold the logical pages `used[b]`; the others are released (-1)."""
    num_pages = sum(len(u) for u in used) + 3
    perm = rng.permutation(num_pages).astype(np.int32)
    table = np.full((len(used), width), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, u] = perm[at:at + len(u)]
        at += len(u)
    return table, num_pages


def _prepare_latent(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    B, n = c["batch"], c["n_q"]
    rows = B * n
    r = random.Random(B * 1021 + n)
    lens = [n + r.randint(0, 500) for _ in range(B)]
    table, num_pages = _tables(rng, [list(range(_pages(x))) for x in lens], _pages(max(lens)))
    # the projections' outputs: the absorbed query head by head, the rotary part behind 128 other
    # values of its head, the latent and its rotary part side by side
    q_nope = torch.randn(HEADS, rows, D_NOPE, generator=g, device="cuda").to(torch.bfloat16)
    q_up = torch.randn(rows, HEADS, 192, generator=g, device="cuda").to(torch.bfloat16)
    kv = (torch.randn(rows, D_QK, generator=g, device="cuda") * 3).to(torch.bfloat16)
    s = {"case": c, "q_nope": q_nope.transpose(0, 1), "q_rope": q_up[:, :, 128:], "c_kv": kv[:, :D_NOPE], "k_rope": kv[:, D_NOPE:],
         "gamma_kv": (1 + 0.2 * torch.randn(D_NOPE, generator=g, device="cuda")).to(torch.bfloat16),
         "gamma_q": (1 + 0.2 * torch.randn(D_NOPE, generator=g, device="cuda")).to(torch.bfloat16) if c["norm_q"] else None,
         "inv_freq": (10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32)).float(),
         "positions": torch.randint(0, 1 << 20, (rows,), generator=g, device="cuda", dtype=torch.int32) if c["far"] else None,
         "lat": torch.zeros(num_pages, PAGE * ROW_BYTES[c["fmt"]], dtype=torch.uint8, device="cuda"),
         "table": torch.from_numpy(table).cuda(), "ctx": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "q": torch.empty(rows, HEADS, D_QK, dtype=torch.bfloat16, device="cuda")}
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        s["params"] = _params(dsa, c, table, num_pages)
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return s


def _params(dsa, c, table, num_pages):
    fmt = c.get("fmt", "fp8")
    return dsa.make_params(
        batch=c["batch"], n_q=c.get("n_q", 1), max_pages_per_req=table.shape[1], num_pages=num_pages, key_page_stride=KEY_PAGE,
        lat_page_stride=PAGE * ROW_BYTES[fmt], lat_fmt=dsa.DSA_LAT_FP8_576 if fmt == "fp8" else dsa.DSA_LAT_NVFP4_352,
        softmax_scale=SCALE, latent_scale=LATENT_SCALE)


def _prepare_window(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    lens = _lens(c)
    table, num_pages = _tables(rng, [_used_pages(c, n) for n in lens], _pages(max(lens)))
    rows = c["batch"] * c["n_q"]
    s = {"case": c, "lat": _latent_pool(g, num_pages, c["fmt"]),
         "q": torch.randn(rows, HEADS, D_QK, generator=g, device="cuda").to(torch.bfloat16),
         "table": torch.from_numpy(table).cuda(), "ctx": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    if c["kind"] == "window":
        s["out"] = torch.empty(rows, HEADS, D_NOPE, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(rows, HEADS, dtype=torch.float32, device="cuda")
    else:
        s["lse"] = torch.empty(rows, HEADS, dtype=torch.float32, device="cuda")
        for b in range(c["batch"]):  # the log-sum-exps that the step's attention left
            z, _ = _logits(s, slice(b, b + 1))
            s["lse"][b * c["n_q"]:(b + 1) * c["n_q"]] = torch.logsumexp(z, -1).view(-1, HEADS)
        s["start"] = torch.rand(c["batch"], table.shape[1] * PAGE, generator=g, device="cuda") * 4
        s["mass"] = s["start"].clone()
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        s["params"] = _params(dsa, c, table, num_pages)
        s["ws"] = torch.zeros(dsa.workspace_size(s["params"]), dtype=torch.uint8, device="cuda")
    return s


def _prepare_evict(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    B, lens, shared = c["batch"], _lens(c), c["prefix"] // PAGE
    counts = [_pages(n) - shared for n in lens]
    width = _pages(max(lens))
    live = shared + sum(counts)
    num_pages = live + (B * shared if B > 1 else 0) + 5
    perm = rng.permutation(num_pages).astype(np.int32)
    table, refs = np.full((B, width), -1, np.int32), np.zeros(num_pages, np.int32)
    at = shared
    for b, n in enumerate(counts):
        table[b, :shared] = perm[:shared]
        table[b, shared:shared + n] = perm[at:at + n]
        at += n
        refs[table[b, :shared + n]] += 1
    # accumulated weights spread over some octaves, many of them alike, the last ones still at 0
    mass = torch.exp(1.5 * torch.randn(B, width * PAGE, generator=g, device="cuda"))
    mass = torch.where(torch.rand(B, width * PAGE, generator=g, device="cuda") < 0.3, torch.round(mass * 8) / 8, mass)
    mass[:, -20:] = 0
    start = torch.from_numpy(np.concatenate([table.ravel(), np.array(lens, np.int32), refs])).cuda()
    cur = start.clone()
    s = {"case": c, "start": start, "cur": cur, "table": cur[:B * width].view(B, width), "ctx": cur[B * width:B * width + B],
         "refs": cur[B * width + B:], "mass0": mass, "mass": mass.clone(),
         "budgets": torch.tensor(_budgets(c), dtype=torch.int32, device="cuda"),
         "kept": torch.full((B, width * PAGE), -1, dtype=torch.int32, device="cuda"),
         "keys": torch.randint(-2 ** 31, 2 ** 31, (num_pages, c["layers"], KEY_PAGE // 4), generator=g, device="cuda", dtype=torch.int32),
         "lats": torch.randint(-2 ** 31, 2 ** 31, (num_pages, c["layers"], PAGE, 576 // 4), generator=g, device="cuda", dtype=torch.int32)}
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        s["params"] = _params(dsa, c, table, num_pages)
        s["ws"] = torch.zeros(dsa.workspace_size(s["params"]), dtype=torch.uint8, device="cuda")
        s["pools"] = dsa.make_token_pools([
            (s["keys"], dsa.DSA_TOKEN_KEY_FP8, c["layers"], KEY_PAGE, c["layers"] * KEY_PAGE),
            (s["lats"], dsa.DSA_TOKEN_LAT_FP8, c["layers"], LAT_PAGE, c["layers"] * LAT_PAGE)])
    return s


def prepare(case, seed):
    if case["kind"] == "latent":
        return _prepare_latent(case, seed)
    if case["kind"] == "evict":
        return _prepare_evict(case, seed)
    return _prepare_window(case, seed)


# ---------------------------------------------------------------- one pass


def run(s):
    return {"latent": _latent, "window": _window, "mass": _mass, "evict": _evict}[s["case"]["kind"]](s)


def _rotate(x, cos, sin, interleaved):
    """x [..., 64], cos and sin [..., 32]"""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    return torch.stack([lo, hi], -1).flatten(-2) if interleaved else torch.cat([lo, hi], -1)


def _to_e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _to_e2m1(x):
    """Magnitudes on the 4-bit grid (ties to the even code)."""
    a = x.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(a / step) * step


def _norm(x):
    """x / rms, the mean of the squares in 64 bits (the cache's codes are next to a border now and then)"""
    return x * torch.rsqrt(x.double().square().mean(-1, keepdim=True) + EPS).float()


def _latent(s):
    c = s["case"]
    B, n, fmt = c["batch"], c["n_q"], c["fmt"]
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        dsa.latent_frontend(s["params"], s["q_nope"], s["q_rope"], s["gamma_q"], s["c_kv"], s["k_rope"], s["gamma_kv"], s["inv_freq"],
                            s["positions"], s["lat"], s["table"], s["ctx"], s["q"], s["ws"], eps=EPS, interleaved=c["interleaved"])
    else:
        slot = s["ctx"].long()[:, None] - n + torch.arange(n, device="cuda")
        pos = (slot.view(-1) if s["positions"] is None else s["positions"]).double()
        angle = pos[:, None] * s["inv_freq"].double()
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        nope = s["q_nope"].float()
        if s["gamma_q"] is not None:
            nope = _norm(nope) * s["gamma_q"].float()
        s["q"].copy_(torch.cat([nope, _rotate(s["q_rope"].float(), cos[:, None], sin[:, None], c["interleaved"])], -1))
        lat = _norm(s["c_kv"].float()) * s["gamma_kv"].float() * (1 / LATENT_SCALE)
        rot = _to_e4m3(_rotate(s["k_rope"].float(), cos, sin, c["interleaved"]) * (1 / LATENT_SCALE)).view(torch.uint8)
        if fmt == "fp8":
            rows = torch.cat([_to_e4m3(lat).view(torch.uint8), rot], 1)
        else:
            block = lat.view(-1, 32, 16)
            scale = _to_e4m3(block.abs().amax(-1) / torch.full((1,), 6.0, device="cuda"))
            wide = scale.float()[:, :, None]
            code = torch.bucketize(_to_e2m1(block / wide), torch.tensor(E2M1, device="cuda")) + 8 * torch.signbit(block)
            code = torch.where(wide > 0, code, 0).view(-1, D_NOPE)
            rows = torch.cat([(code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8), scale.view(torch.uint8), rot], 1)
        page = s["table"].long().gather(1, slot // PAGE)
        s["lat"].view(-1, ROW_BYTES[fmt])[(page * PAGE + slot % PAGE).view(-1)] = rows
    if fmt == "fp8":
        return {"q": s["q"], "cache": s["lat"].view(torch.float8_e4m3fn)}
    # (pairs of 4-bit values have no type to be returned as without a pass of their own over them: they are
    # returned packed, and have to be equal)
    rows = s["lat"].view(-1, ROW_BYTES[fmt])
    return {"q": s["q"], "pairs": rows[:, :256], "scales_rope": rows[:, 256:].view(torch.float8_e4m3fn)}


def _decode(rows, fmt):
    """Latents [n, 576] in 32 bits of n rows of the pool."""
    if fmt == "fp8":
        return rows.view(torch.float8_e4m3fn).float()
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)
    nib = torch.stack([rows[:, :256] & 15, rows[:, :256] >> 4], -1).view(-1, 512)
    scale = rows[:, 256:288].contiguous().view(torch.float8_e4m3fn).float()
    nope = lut[nib.long()].view(-1, 32, 16) * scale[:, :, None]
    return torch.cat([nope.view(-1, 512), rows[:, 288:].contiguous().view(torch.float8_e4m3fn).float()], 1)


def _union(s, who):
    """For the requests `who`: the tokens that some row sees [B, M] (padded), whether row t sees them
    [B, n_q, M], and their latents [B, M, 576] in 32 bits (0 where no row does)."""
    c = s["case"]
    n, sinks, window = c["n_q"], c["sinks"], c["window"]
    ctx, table = s["ctx"][who].long(), s["table"][who].long()
    first = (ctx - n + 1 - window).clamp(min=0)
    head = ctx.new_full(ctx.shape, sinks).minimum(first)  # tokens before the window's first that stay
    M = min(c["longest"], sinks + window + n - 1)
    j = torch.arange(M, device="cuda")
    tok = torch.where(j < head[:, None], j, first[:, None] + j - head[:, None])
    L = ctx[:, None] - n + 1 + torch.arange(n, device="cuda")
    t = tok[:, None, :]
    sees = (t < L[:, :, None]) & ((t < sinks) | (t >= L[:, :, None] - window))
    any_row = sees.any(1)
    page = table.gather(1, (tok // PAGE).clamp(max=table.shape[1] - 1)).clamp(min=0)
    rows = s["lat"].view(-1, ROW_BYTES[c["fmt"]])[(page * PAGE + tok % PAGE).view(-1)]
    lat = _decode(rows, c["fmt"]).view(*tok.shape, D_QK) * LATENT_SCALE
    return tok, any_row, sees, lat.masked_fill(~any_row[:, :, None], 0.0)


def _logits(s, who):
    """Logits [B, n_q, HEADS, M] of the requests `who` (-inf where hidden), and what _union gives."""
    n = s["case"]["n_q"]
    tok, any_row, sees, lat = _union(s, who)
    B = tok.shape[0]
    q = s["q"].view(-1, n, HEADS, D_QK)[who].float() * SCALE
    z = (q.view(B, n * HEADS, D_QK) @ lat.transpose(1, 2)).view(B, n, HEADS, -1)
    return z.masked_fill_(~sees[:, :, None, :], -math.inf), (tok, any_row, sees, lat)


def _window(s):
    c = s["case"]
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        dsa.window_mla_decode(s["params"], s["q"], s["lat"], c["sinks"], c["window"], s["table"], s["ctx"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    z, (tok, _, _, lat) = _logits(s, slice(None))
    B, n = c["batch"], c["n_q"]
    m = z.amax(-1, keepdim=True)
    z = z.sub_(m).exp_()
    total = z.sum(-1, keepdim=True)
    out = (z.view(B, n * HEADS, -1) @ lat[:, :, :D_NOPE]).view(B, n, HEADS, D_NOPE) / total
    return {"out": out.view(B * n, HEADS, D_NOPE).to(torch.bfloat16), "lse": (m + torch.log(total)).view(B * n, HEADS)}


def _mass(s):
    c = s["case"]
    s["mass"].copy_(s["start"])  # the weights are added in place
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        dsa.attention_mass(s["params"], s["q"], s["lat"], c["sinks"], c["window"], s["table"], s["ctx"], s["lse"], 0, s["mass"], s["ws"])
        return {"mass": s["mass"]}
    z, (tok, any_row, _, _) = _logits(s, slice(None))
    z = z.sub_(s["lse"].view(c["batch"], c["n_q"], HEADS, 1)).exp_()
    at = tok.clamp(max=s["mass"].shape[1] - 1)
    s["mass"].scatter_add_(1, at, z.sum((1, 2)).masked_fill_(~any_row, 0.0))
    return {"mass": s["mass"]}


def _evict(s):
    c = s["case"]
    s["cur"].copy_(s["start"])  # the call changes its state in place
    s["mass"].copy_(s["mass0"])
    table, ctx, refs, mass = s["table"], s["ctx"], s["refs"], s["mass"]
    done = {"table": table, "ctx": ctx, "refs": refs, "mass": mass, "kept": s["kept"], "keys": s["keys"], "lats": s["lats"]}
    if own:
        import dsa_sparse_mla_paged_gb300 as dsa

        dsa.tokens_evict(s["params"], s["budgets"], c["sinks"], c["recent"], mass, s["pools"], table, ctx, refs, s["kept"], s["ws"])
        return done
    B, width = table.shape
    n, budget = ctx.long(), s["budgets"].long()
    tok = torch.arange(width * PAGE, device="cuda")
    goes = (budget >= 0) & (n > budget)
    head = budget.clamp(max=c["sinks"])
    tail = (budget - head).clamp(max=c["recent"])
    mid = goes[:, None] & (tok >= head[:, None]) & (tok < (n - tail)[:, None])
    # rank by weight, ties by token; then the kept tokens in order
    order = torch.argsort(torch.where(mid, mass, -math.inf), dim=1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, tok.expand(B, -1))
    keep = torch.where(mid, rank < (budget - head - tail)[:, None], tok < n[:, None])
    new = torch.where(goes, budget, n)
    kept = torch.argsort((~keep).to(torch.int8), dim=1, stable=True)
    live = tok < new[:, None]
    # pages that change, and a fresh page for each that others hold
    changed = ((kept != tok) & live).view(B, width, PAGE).any(-1)
    old_pages = table.long().clamp(min=0)
    shared = changed & (refs[old_pages] > 1)
    need = shared.sum(1)
    upto = need.cumsum(0)
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)
    at = ((upto - need)[:, None] + shared.cumsum(1) - 1).clamp(0, free.numel() - 1)
    to = torch.where(shared, free[at], old_pages)
    move = live & changed.repeat_interleave(PAGE, 1)
    who, i = move.nonzero(as_tuple=True)
    src, dst = kept[who, i], to[who, i // PAGE]
    page, slot = old_pages[who, src // PAGE], src % PAGE
    i = i % PAGE
    s["lats"][dst, :, i] = s["lats"][page, :, slot]
    split = PAGE * 32  # a key page: 64 rows of 32 words, then a scale each
    values, scales = s["keys"][:, :, :split].unflatten(2, (PAGE, 32)), s["keys"][:, :, split:]
    values[dst, :, i] = values[page, :, slot]
    scales[dst, :, i] = scales[page, :, slot]
    # tables, counts, lengths and weights
    have = torch.arange(width, device="cuda")
    drop = (have >= ((new + PAGE - 1) // PAGE)[:, None]) & (have < ((n + PAGE - 1) // PAGE)[:, None])
    gone = old_pages[drop | shared]
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    refs[to[shared]] = 1
    table.copy_(torch.where(drop, -1, torch.where(shared, to, table.long())))
    ctx.copy_(new)
    moved = mass.gather(1, kept)
    mass.copy_(torch.where(live, moved, torch.where(tok < n[:, None], 0.0, mass)))
    s["kept"].copy_(torch.where(live, kept, s["kept"].long()))
    return done


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


def _exact_latent(c, seed):
    s = _prepare_latent(c, seed)
    n, half = c["n_q"], torch.arange(32, device="cuda")
    i0, i1 = (2 * half, 2 * half + 1) if c["interleaved"] else (half, half + 32)
    q = torch.empty(c["batch"] * n, HEADS, D_QK, dtype=torch.float64, device="cuda")
    for b, ctx in enumerate(s["ctx"].tolist()):
        at = slice(b * n, (b + 1) * n)
        pos = torch.arange(ctx - n, ctx, device="cuda").double() if s["positions"] is None else s["positions"][at].double()
        angle = torch.outer(pos, s["inv_freq"].double())[:, None, :]
        x = s["q_nope"][at].double()
        if c["norm_q"]:
            x = x / torch.sqrt(x.pow(2).sum(2, keepdim=True) / D_NOPE + EPS) * s["gamma_q"].double()
        q[at, :, :D_NOPE] = x
        x = s["q_rope"][at].double()
        q[at, :, D_NOPE + i0] = x[:, :, i0] * angle.cos() - x[:, :, i1] * angle.sin()
        q[at, :, D_NOPE + i1] = x[:, :, i1] * angle.cos() + x[:, :, i0] * angle.sin()
    # (the cache's codes have no value in 64 bits: a rounding to 8 or 4 bits is what is asked for)
    return {"q": q, "cache": None} if c["fmt"] == "fp8" else {"q": q, "pairs": None, "scales_rope": None}


def exact(case, seed):
    if case["kind"] == "evict":
        return None  # whole numbers, and values that are moved as they are
    if case["kind"] == "latent":
        return _exact_latent(case, seed)
    s = _prepare_window(case, seed)
    fmt, n = case["fmt"], case["n_q"]
    pool = s["lat"].view(-1, PAGE, ROW_BYTES[fmt])
    out, lse = [], []
    mass = None if case["kind"] == "window" else s["start"].double()
    for b, ctx in enumerate(s["ctx"].tolist()):
        used = torch.tensor(_used_pages(case, ctx), device="cuda")
        lat = _values(pool[s["table"][b].long()[used]].reshape(-1, ROW_BYTES[fmt]), fmt) * LATENT_SCALE
        tok = (used[:, None] * PAGE + torch.arange(PAGE, device="cuda")).view(-1)
        for t0 in range(0, n, 32):
            t1 = min(n, t0 + 32)
            L = torch.arange(ctx - n + 1 + t0, ctx - n + 1 + t1, device="cuda")[:, None]
            hide = (tok >= L) | ((tok >= case["sinks"]) & (tok < L - case["window"]))
            z = (s["q"][b * n + t0:b * n + t1].double() @ lat.T) * SCALE
            z.masked_fill_(hide[:, None, :], -math.inf)
            if mass is None:
                z_lse = torch.logsumexp(z, 2)
                lse.append(z_lse)
                out.append(torch.exp(z - z_lse[:, :, None]) @ lat[:, :D_NOPE])
            else:
                keep = tok < ctx
                w = torch.exp(z - s["lse"][b * n + t0:b * n + t1, :, None].double()).sum((0, 1))
                mass[b].index_add_(0, tok[keep], w[keep])
    return {"out": torch.cat(out), "lse": torch.cat(lse)} if mass is None else {"mass": mass}
