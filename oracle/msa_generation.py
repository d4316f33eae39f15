"""Float64 CPU oracle of the generation step's operators: per-head RMS norms
with RoPE (and their gradient), the append to a paged cache, and attention
for trees of drafted tokens over [memory ; cache ; tree].

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product
library.

Sources: "EverMind-AI/MSA: routing top-k compressed documents inside
attention ..." (hysenlabs.com), §"Routing happens inside attention ..." (the
selected documents' K/V joined with the query's growing local K/V) and
§"Document-wise RoPE ..."; the per-head norms are those of the Qwen3 backbone
the pages name.  Everything is computed in float64, row by row where a loop
is plainer than an index expression.
"""

from __future__ import annotations

import numpy as np

from .msa_oracle import _f64, rope_rotate


def head_norm(x, weight, eps: float):
    """x / sqrt(mean(x^2) + eps) * weight over the last axis; x itself
    without a weight."""
    x = _f64(x)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * _f64(weight)


def norm_rope(x, weight, positions, eps: float = 1e-6, rope_base: float = 10000.0):
    """x [N][heads][D], positions [N] (None: not rotated)."""
    z = head_norm(x, weight, eps)
    if positions is None:
        return z
    return rope_rotate(z, positions, rope_base)


def norm_rope_backward(x, weight, positions, dy, eps: float = 1e-6,
                       rope_base: float = 10000.0):
    """(dx, dweight) of norm_rope; dweight is None without a weight."""
    x, dz = _f64(x), _f64(dy)
    if positions is not None:
        dz = rope_rotate(dz, -_f64(positions), rope_base)
    if weight is None:
        return dz, None
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    g = dz * _f64(weight)
    dx = r * g - x * r ** 3 * (g * x).mean(axis=-1, keepdims=True)
    return dx, (dz * x * r).sum(axis=(0, 1))


def paged_rows(b, rows, block_table, page_size: int):
    """(page, row in the page) of each of sequence b's cache rows."""
    return [(int(block_table[b][r // page_size]), r % page_size) for r in rows]


def paged_append(pages, x, tok_offsets, cache_len, block_table):
    """A copy of pages [n_pages][H][page][D] with x [N][H][D]'s rows written
    behind each sequence's cache_len rows."""
    out = np.array(pages, dtype=np.float64)
    for b in range(len(cache_len)):
        for i, t in enumerate(range(int(tok_offsets[b]), int(tok_offsets[b + 1]))):
            [(pg, row)] = paged_rows(b, [int(cache_len[b]) + i], block_table, out.shape[2])
            out[pg, :, row] = x[t]
    return out


def ancestors(parents) -> np.ndarray:
    """[n][n] bool: what each token of one tree sees of it (itself and its
    ancestors); nothing for a pruned token (parent < -1) or one below it."""
    n = len(parents)
    see = np.zeros((n, n), dtype=bool)
    for i in range(n):
        path, a = [], i
        while a >= 0:
            path.append(a)
            a = int(parents[a])
        if a == -1:
            see[i, path] = True
    return see


def tree_attn(q, tok_offsets, parents, k_mem, v_mem, mem_len, k_pages, v_pages, block_table,
              cache_len, scale: float = 0.0):
    """(out [N][Hq][D], bound [N][Hq][D], top [N][Hq]): the attention of every
    token, sum_j p_j |v_j| (what a relative error of the weights p moves the
    output by) and the largest scale sum_d |q_d k_d| of the keys it sees.
    Rows that belong to no sequence, and rows that see nothing, are zero."""
    q = _f64(q)
    N, Hq, D = q.shape
    n_pages, H, page, _ = k_pages.shape
    G = Hq // H
    scale = scale if scale > 0 else 1.0 / np.sqrt(D)
    out, bound, top = np.zeros_like(q), np.zeros_like(q), np.zeros((N, Hq))
    for b in range(len(cache_len)):
        t0, t1 = int(tok_offsets[b]), int(tok_offsets[b + 1])
        n, L = t1 - t0, int(cache_len[b])
        par = list(range(-1, n - 1)) if parents is None else [int(p) for p in parents[t0:t1]]
        tree = ancestors(par)
        at = paged_rows(b, range(L + n), block_table, page)
        M = 0 if k_mem is None else int(mem_len[b])
        for g in range(H):
            ks = [k_mem[b, j, g] for j in range(M)] + [k_pages[pg, g, r] for pg, r in at]
            vs = [v_mem[b, j, g] for j in range(M)] + [v_pages[pg, g, r] for pg, r in at]
            ks, vs = np.array(ks).reshape(-1, D), np.array(vs).reshape(-1, D)
            for i in range(n):
                if not tree[i, i]:
                    continue
                see = np.concatenate([np.ones(M + L, dtype=bool), tree[i]])
                kk, vv = ks[see], vs[see]
                qq = q[t0 + i, g * G:(g + 1) * G]
                s = qq @ kk.T * scale
                p = np.exp(s - s.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
                out[t0 + i, g * G:(g + 1) * G] = p @ vv
                bound[t0 + i, g * G:(g + 1) * G] = p @ np.abs(vv)
                top[t0 + i, g * G:(g + 1) * G] = (np.abs(qq) @ np.abs(kk).T).max(axis=1) * scale
    return out, bound, top
