"""Plain restatement, in numpy, of the operators of a bounded latent cache: the attention's front end, attention with a
sliding window and sinks, the accumulated weight of every token, and eviction by it. One row, one request and
one token at a time; shares no code with the library.
"""
from __future__ import annotations

import numpy as np

from oracle import dsa as O
from oracle.formats import bf16_decode
from oracle.serving import ERR_BLOCK_TABLE, ERR_CTX, ERR_NO_PAGES, ERR_PAGES, PAGE, pages_of

# ---------------------------------------------------------------- front end


def rotate(x, angles, interleaved: bool):
    """x [..., 64], angles [32], float64."""
    out = np.empty_like(x)
    for i in range(32):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        c, s = np.cos(angles[i]), np.sin(angles[i])
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def rms_norm(x, gamma, eps: float):
    """x [..., 512], float64."""
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma


def front_row(q_nope, q_rope, gamma_q, c_kv, k_rope, gamma_kv, inv_freq, position: int, eps: float, interleaved: bool):
    """One row in float64 (bf16 values given as such): (query [96, 576], latent values [576] before they are
    divided by the latent scale and quantised)."""
    angles = int(position) * inv_freq.astype(np.float64)
    nope = q_nope if gamma_q is None else rms_norm(q_nope, gamma_q, eps)
    q = np.concatenate([nope, rotate(q_rope, angles, interleaved)], -1)
    return q, np.concatenate([rms_norm(c_kv, gamma_kv, eps), rotate(k_rope, angles, interleaved)])


# ---------------------------------------------------------------- window


def visible(L: int, sinks: int, window: int) -> np.ndarray:
    """The tokens that a row with L tokens before its end attends to."""
    s = np.arange(L)
    return s[(s < sinks) | (s >= L - window)]


def good_tokens(inp, b: int, tokens: np.ndarray) -> np.ndarray:
    """Those of `tokens` whose page exists."""
    pg = inp.block_table[b, tokens // PAGE]
    return tokens[(pg >= 0) & (pg < inp.num_pages)]


def window_mla(inp, sinks: int, window: int, b: int, t: int, query_error):
    """Row (b, t): (out, lse, mass, bulk, extra, tail) as oracle.serving.prefix_mla gives them."""
    tok = good_tokens(inp, b, visible(O.visible_len(inp.ctx[b], inp.n_q, t), sinks, window))
    c = O.dequant_latents(inp, b, tok)
    q = bf16_decode(inp.q[b, t])
    out, lse = O.mla_attention(q, c, inp.softmax_scale)
    p = np.exp(inp.softmax_scale * (q @ c.T) - lse[:, None])
    size = np.abs(c).T
    return (out, lse, p @ size[:512].T, inp.softmax_scale * (np.abs(q) @ size).max(axis=1),
            inp.softmax_scale * (query_error(q) @ size).max(axis=1), p.max(axis=1)[:, None] * size[:512].sum(axis=1))


def attention_mass(inp, sinks: int, window: int, lse, b: int, query_error):
    """Request b: (tokens that some row sees, the weight added to each, a bound on what an fp32 evaluation is
    off by there). lse float32 [n_q, 96], finite or not. An evaluation's logits are off by d = 66 * 2^-23 bulk + extra
    (see tests/test_gpu_prefix.py), log2(e) * lse and the difference by 2^-22 of their size, the exponential by 2^-21."""
    total, bound = np.zeros(int(inp.ctx[b])), np.zeros(int(inp.ctx[b]))
    seen = np.zeros(int(inp.ctx[b]), bool)
    for t in range(inp.n_q):
        tok = good_tokens(inp, b, visible(O.visible_len(inp.ctx[b], inp.n_q, t), sinks, window))
        c, q = O.dequant_latents(inp, b, tok), bf16_decode(inp.q[b, t])
        ok = np.isfinite(lse[t])
        z = inp.softmax_scale * (q @ c.T)
        with np.errstate(all="ignore"):
            p = np.where(ok[:, None], np.exp(z - lse[t].astype(np.float64)[:, None]), 0.0)
        size = np.abs(c).T
        d = inp.softmax_scale * (66 * 2.0 ** -23 * (np.abs(q) @ size) + query_error(q) @ size)
        d = d + 2.0 ** -22 * (np.abs(z) + np.where(ok, np.abs(lse[t]), 0.0)[:, None]) + 2.0 ** -21
        total[tok] += p.sum(axis=0)
        bound[tok] += (p * np.expm1(np.minimum(d, 1.0))).sum(axis=0)
        seen[tok] = True
    return np.nonzero(seen)[0], total[seen], bound[seen] + (96 + inp.n_q) * 2.0 ** -24 * total[seen]


# ---------------------------------------------------------------- eviction

# formats of a token's row: bytes of a row, bytes of its scale behind the page's rows
ROWS = {"key_fp8": (128, 4), "key_mxfp4": (64, 4), "lat_fp8": (576, 0), "lat_nvfp4": (352, 0)}


def _order(m: float):
    """Larger is kept first; a NaN is below everything, -0 is 0."""
    return (0, 0.0) if np.isnan(m) else (1, float(m) + 0.0)


def chosen(mass, n: int, budget: int, sinks: int, recent: int):
    """The tokens of n that stay, in order."""
    head = min(sinks, budget)
    tail = min(recent, budget - head)
    middle = sorted(range(head, n - tail), key=lambda i: (_order(mass[i]), -i), reverse=True)[:budget - head - tail]
    return list(range(head)) + sorted(middle) + list(range(n - tail, n))


def tokens_evict(table, ctx, refs, mass, budgets, sinks, recent, pools, kept=None):
    """One request after another, in place. pools: (format, [uint8 [num_pages, page bytes] of each layer]). Returns the
    error bits."""
    err, cap, n_pages = 0, table.shape[1] * PAGE, len(refs)
    start_refs, state = refs.copy(), "ok"
    free = [p for p in range(n_pages) if refs[p] <= 0]
    old_pools = [[layer.copy() for layer in layers] for _, layers in pools]  # every request reads what the call found
    for b, budget in enumerate(budgets):
        n = int(ctx[b])
        ok = 0 <= n <= cap
        if budget >= 0 and not ok:
            err |= ERR_CTX
        if kept is not None and ok:
            kept[b, :n] = np.arange(n) if not 0 <= budget < n else kept[b, :n]
        if budget < 0 or not ok or n <= budget:
            continue
        stay = chosen(mass[b], n, int(budget), sinks, recent)
        old = table[b, :pages_of(n)].copy()
        inside = (old >= 0) & (old < n_pages)
        bad = (0 if inside.all() else ERR_BLOCK_TABLE) | (ERR_PAGES if (start_refs[old[inside]] < 1).any() else 0)
        new = old[:pages_of(budget)].copy()
        changes = [j for j in range(len(new)) if any(stay[i] != i for i in range(j * PAGE, min(budget, (j + 1) * PAGE)))]
        copies = [] if bad else [j for j in changes if start_refs[old[j]] > 1]
        if copies and (state == "full" or len(copies) > len(free)):
            state = "full"
            bad |= ERR_NO_PAGES
        if bad:
            err |= bad
            if kept is not None:
                kept[b, :n] = np.arange(n)
            continue
        for j in copies:
            new[j] = free.pop(0)
            refs[new[j]] = 1
            refs[old[j]] -= 1
        for j in range(len(new), len(old)):
            refs[old[j]] -= 1
        for (fmt, layers), before in zip(pools, old_pools):
            row, scale = ROWS[fmt]
            for layer, source in zip(layers, before):
                for j in changes:
                    for i in range(j * PAGE, min(budget, (j + 1) * PAGE)):
                        src, dst, a, z = source[old[stay[i] // PAGE]], layer[new[j]], stay[i] % PAGE, i % PAGE
                        dst[z * row:(z + 1) * row] = src[a * row:(a + 1) * row]
                        at = PAGE * row
                        dst[at + z * scale:at + (z + 1) * scale] = src[at + a * scale:at + (a + 1) * scale]
        table[b, :len(new)] = new
        table[b, len(new):len(old)] = -1
        mass[b, :budget] = mass[b, stay]
        mass[b, budget:n] = 0
        if kept is not None:
            kept[b, :budget] = stay
        ctx[b] = budget
    return err
