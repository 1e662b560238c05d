"""fp64 reference of the prompt side: tables, append by slot, expanded latents
and attention of ragged chunks.  Plain loops over requests and tokens; shares
no code with the CUDA path.
"""

from __future__ import annotations

import numpy as np

from . import steps

PAGE = 64

ERR_PAGE, ERR_LONG, ERR_POOL, ERR_TOKENS, ERR_LENGTH = 1, 2, 16, 32, 64


def build_tables(cached, new, free_pages, free_count, block_table, max_tokens, num_pages):
    """One step's tables, request by request and page by page."""
    table = np.array(block_table, dtype=np.int64)
    mpps = table.shape[1]
    err = 0
    count = int(min(max(free_count, 0), num_pages))
    if count != free_count:
        err |= ERR_LENGTH
    stack = list(free_pages[:count])
    pos = [0] * max_tokens
    slots = [-1] * max_tokens
    q_start, kv_start, lens = [0], [0], []
    at, short = 0, False
    for b in range(len(cached)):
        c, n = int(cached[b]), int(new[b])
        ok = True
        if c < 0 or n < 0:
            err |= ERR_LENGTH
            c, n, ok = max(c, 0), max(n, 0), False
        elif c + n > min(mpps * PAGE, 2 ** 31 - 1):
            err |= ERR_LONG
            ok = False
        held, need = -(-c // PAGE), -(-(c + n) // PAGE)
        fits = at + n <= max_tokens or n == 0
        if not fits:
            err |= ERR_TOKENS
        if ok and need > held:
            # a request that lacks pages shuts the list for those after it
            if short or need - held > len(stack):
                err |= ERR_POOL
                short, ok = True, False
        got = []
        if ok and fits:
            got = [int(stack.pop()) for _ in range(need - held)]
            for i, page in enumerate(got):
                table[b, held + i] = page
                if not 0 <= page < num_pages:
                    err |= ERR_PAGE
        ok = ok and fits
        for i in range(n):
            t = at + i
            if t >= max_tokens:
                break
            p = c + i
            pos[t] = min(p, 2 ** 31 - 1)
            if ok:
                page = int(table[b, p // PAGE])
                if 0 <= page < num_pages:
                    slots[t] = page * PAGE + p % PAGE
                else:
                    err |= ERR_PAGE
        at += n
        lens.append(c + n if ok else c)
        q_start.append(min(at, max_tokens))
        kv_start.append(kv_start[-1] + lens[-1])
    return dict(block_table=table, seq_lens=np.array(lens), free_left=np.array([len(stack)]), q_start=np.array(q_start),
                kv_start=np.minimum(kv_start, 2 ** 31 - 1), pos=np.array(pos, dtype=np.int64), slots=np.array(slots, dtype=np.int64), err=err)


def append_rows(cache, rows, pos, slots, turned, base):
    """cache [pages][64][row] fp64 with rows written by slot; columns
    ``turned`` (list of (offset, width)) rotated at pos first (base 0: not)."""
    out = np.array(cache, dtype=np.float64)
    for t, s in enumerate(slots):
        if s < 0 or s >= out.shape[0] * PAGE:
            continue
        r = np.array(rows[t], dtype=np.float64)
        if base:
            for off, width in turned:
                r[off:off + width] = steps.rope(r[off:off + width], np.array(pos[t]), base)
        out[s // PAGE, s % PAGE] = r
    return out


def gather(cache, block_table, b, n, mpps):
    """The first n cached rows of sequence b."""
    idx = [(int(block_table[b, j // PAGE]) if block_table is not None else b * mpps + j // PAGE, j % PAGE) for j in range(n)]
    return np.array([cache[p, s] for p, s in idx], dtype=np.float64).reshape(n, cache.shape[-1])


def expand(rows, w_uk, w_uv, groups):
    """k [H][n][d_k], v [H][n][d_v], and the sums of absolute products that
    bound an fp32 accumulation's error, of n cached rows [c_0 | ... | k^R]."""
    H, d_k, d_c = w_uk.shape
    k, v, ka, va = [], [], [], []
    for h in range(H):
        g = h // (H // groups)
        c = rows[:, g * d_c:(g + 1) * d_c]
        k.append(c @ w_uk[h].T)
        v.append(c @ w_uv[h])
        ka.append(np.abs(c) @ np.abs(w_uk[h]).T)
        va.append(np.abs(c) @ np.abs(w_uv[h]))
    return np.array(k), np.array(v), np.array(ka), np.array(va)


def attention(q, k, v, scale, causal):
    """One head of one sequence: q [nq][d], k [nk][d], v [nk][dv].  Returns
    out, lse, sum_j p_j |v_j|, and each row's largest scale * sum_d |q_d k_d|
    over the keys it attends."""
    nq, nk = len(q), len(k)
    out, mass = np.zeros((nq, v.shape[1])), np.zeros((nq, v.shape[1]))
    lse, reach = np.full(nq, -np.inf), np.zeros(nq)
    for i in range(nq):
        n = min(nk, max(i + nk - nq + 1, 0)) if causal else nk
        if n == 0:
            continue
        s = scale * (k[:n] @ q[i])
        reach[i] = abs(scale) * (np.abs(k[:n]) @ np.abs(q[i])).max()
        m = s.max()
        e = np.exp(s - m)
        lse[i] = m + np.log(e.sum())
        p = e / e.sum()
        out[i] = p @ v[:n]
        mass[i] = p @ np.abs(v[:n])
    return out, lse, mass, reach
