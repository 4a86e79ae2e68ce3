"""Plain restatement, in numpy and Python integers, of the calls around the
decode step: dense attention over a shared prefix and a private rest, the page
operations, and the verification of drafted tokens. One request, one page and
one token at a time; shares no code with the library.
"""
from __future__ import annotations

import numpy as np

from oracle import dsa as O
from oracle.formats import bf16_decode

PAGE = 64
ERR_BLOCK_TABLE, ERR_CTX, ERR_PAGES, ERR_NO_PAGES, ERR_DRAFT, ERR_PROB = 0x1, 0x2, 0x10, 0x20, 0x40, 0x80


def pages_of(n: int) -> int:
    return -(-n // PAGE)


# ---------------------------------------------------------------- attention


def prefix_mla(inp, prefix_pages, prefix_len: int, b: int, t: int, query_error=None):
    """Row (b, t) over the shared tokens and then its own: (out, lse, mass, bulk),
    where mass[h] = sum_s p_s |c_s| (512 dims) and bulk = max_s scale * sum_d |q_d c_sd|,
    the magnitudes that rounding errors are relative to. query_error(q): bounds on how
    far each query value is off; further results are then max_s scale * sum_d error_d |c_sd|
    and max_s p_s * sum_s |c_s|."""
    L = O.visible_len(inp.ctx[b], inp.n_q, t)
    saved = inp.block_table[b].copy()
    inp.block_table[b, :prefix_len // PAGE] = prefix_pages
    c = O.dequant_latents(inp, b, np.arange(L))
    inp.block_table[b] = saved
    q = bf16_decode(inp.q[b, t])
    out, lse = O.mla_attention(q, c, inp.softmax_scale)
    p = np.exp(inp.softmax_scale * (q @ c.T) - lse[:, None])
    size = np.abs(c).T
    res = out, lse, p @ size[:512].T, inp.softmax_scale * (np.abs(q) @ size).max(axis=1)
    if query_error is None:
        return res
    return *res, inp.softmax_scale * (query_error(q) @ size).max(axis=1), p.max(axis=1)[:, None] * size[:512].sum(axis=1)


# ---------------------------------------------------------------- pages


def pages_resize(table, ctx, refs, new_lens, pools):
    """One request after another, in place. Returns the error bits."""
    err, cap = 0, table.shape[1] * PAGE
    start, state = refs.copy(), "ok"
    free = [p for p in range(len(refs)) if refs[p] <= 0]
    for b, new in enumerate(new_lens):
        old = int(ctx[b])
        if new < 0:
            continue
        if old < 0 or old > cap or new > cap:
            err |= ERR_CTX
            continue
        if new <= old:
            for j in range(pages_of(new), pages_of(old)):
                pg = table[b, j]
                if not 0 <= pg < len(refs):
                    err |= ERR_BLOCK_TABLE
                elif start[pg] <= 0 or refs[pg] <= 0:
                    err |= ERR_PAGES
                else:
                    refs[pg] -= 1
                table[b, j] = -1
            ctx[b] = new
            continue
        copy = -1
        if old % PAGE:
            copy = int(table[b, old // PAGE])
            if not 0 <= copy < len(refs):
                err |= ERR_BLOCK_TABLE
                continue
            if start[copy] <= 0:
                err |= ERR_PAGES
                continue
            if start[copy] <= 1:
                copy = -1
        need = pages_of(new) - pages_of(old) + (copy >= 0)
        if need and (state == "full" or need > len(free)):
            state = "full"  # every later request that needs pages waits too
            err |= ERR_NO_PAGES
            continue
        if copy >= 0:
            pg = free.pop(0)
            for pool in pools:
                pool[pg] = pool[copy]
            refs[pg], table[b, old // PAGE] = 1, pg
            refs[copy] -= 1
        for j in range(pages_of(old), pages_of(new)):
            table[b, j] = free.pop(0)
            refs[table[b, j]] = 1
        ctx[b] = new
    return err


def pages_fork(table, ctx, refs, src, dst):
    err, before, taken = 0, ctx.copy(), set()
    for s, d in zip(src, dst):
        inside = 0 <= s < len(ctx) and 0 <= d < len(ctx)
        if not inside or d in taken or before[d] != 0 or s == d:
            err |= ERR_PAGES
            if 0 <= d < len(ctx):
                taken.add(d)
            continue
        taken.add(d)
        n = int(before[s])
        if n < 0 or n > table.shape[1] * PAGE:
            err |= ERR_CTX
            continue
        for j in range(pages_of(n)):
            table[d, j] = table[s, j]
            if 0 <= table[s, j] < len(refs):
                refs[table[s, j]] += 1
            else:
                err |= ERR_BLOCK_TABLE
        ctx[d] = n
    return err


def pages_compact(table, ctx, refs, pools):
    """In place; returns (page_map, live, error bits)."""
    err, n = 0, len(refs)
    live = sum(1 for r in refs if r > 0)
    where = [p if refs[p] > 0 else -1 for p in range(n)]
    holes = [p for p in range(live) if refs[p] <= 0]
    for p in range(live, n):
        if refs[p] > 0:
            d = holes.pop(0)
            where[p] = d
            for pool in pools:
                pool[d] = pool[p]
            refs[d], refs[p] = refs[p], 0
    for b in range(len(ctx)):
        if not 0 <= ctx[b] <= table.shape[1] * PAGE:
            err |= ERR_CTX
            continue
        for j in range(pages_of(int(ctx[b]))):
            if not 0 <= table[b, j] < n:
                err |= ERR_BLOCK_TABLE
            elif where[table[b, j]] < 0:
                err |= ERR_PAGES
            else:
                table[b, j] = where[table[b, j]]
    return np.array(where, dtype=np.int32), live, err


# ---------------------------------------------------------------- drafts


def _units(x: float) -> int:
    """A probability as a multiple of 2^-60, rounded down; -1 for what is none."""
    if not 0.0 <= x <= 1.0:
        return -1
    num, den = float(x).as_integer_ratio()
    return num * (1 << 60) // den


def verify_draft(target, draft, tokens, n_draft, uniforms, ctx):
    """target float [B, n_q, V], draft float [B, n_q - 1, V] or None, tokens int [B, n_q - 1],
    n_draft int [B] or None, uniforms float32 [B, n_q]. Returns (accepted, out, new_lens, error bits)."""
    tokens, uniforms = np.asarray(tokens), np.asarray(uniforms, dtype=np.float32)
    B, n_q, V = target.shape
    acc, out, new = np.zeros(B, np.int32), np.full((B, n_q), -1, np.int32), np.zeros(B, np.int32)
    err = 0
    for b in range(B):
        k = n_q - 1 if n_draft is None else int(n_draft[b])
        if not 0 <= k <= n_q - 1:
            err |= ERR_DRAFT
            k = min(max(k, 0), n_q - 1)
        # a token out of range, or an entry that is no probability, is reported even behind a rejected draft of the same 32
        a = k
        for i in range(k):
            x = int(tokens[b, i])
            if not 0 <= x < V:
                err |= ERR_DRAFT
                a = min(a, i)
                continue
            p, q = float(target[b, i, x]), 1.0 if draft is None else float(draft[b, i, x])
            if not (0 <= p <= 1 and 0 <= q <= 1):
                err |= ERR_PROB
                p, q = (v if 0 <= v <= 1 else 0.0 for v in (p, q))
            if not float(uniforms[b, i]) * q < p:
                a = min(a, i)
        p = [_units(float(v)) for v in target[b, a]]
        q = [0] * V
        if a < k:
            if draft is None:
                x = int(tokens[b, a])
                if 0 <= x < V:
                    q[x] = 1 << 61
            else:
                q = [_units(float(v)) for v in draft[b, a]]
                if min(q) < 0:
                    err |= ERR_PROB
        if min(p) < 0:
            err |= ERR_PROB
        p = [max(v, 0) for v in p]
        w = [max(x - max(y, 0), 0) for x, y in zip(p, q)]
        if sum(w) == 0:
            w = p
        total = sum(w)
        acc[b] = a
        out[b, :a] = tokens[b, :a]
        if total == 0 or total > 4 << 60:
            err |= ERR_PROB
        else:
            u = float(uniforms[b, n_q - 1])
            u = min(u, float(np.float32(1) - np.float32(2) ** -24)) if u >= 0 else 0.0
            num, den = u.as_integer_ratio()
            cum = 0
            for v in range(V):
                cum += w[v]
                if cum * den > num * total:
                    out[b, a] = v
                    break
        if ctx is not None:
            if ctx[b] < n_q:
                err |= ERR_CTX
                new[b] = -1
            else:
                new[b] = ctx[b] - n_q + 1 + a
    return acc, out, new, err
