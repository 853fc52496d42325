"""fp64 oracle of a long-context step: rotated appends, page bounds, page
selection, attention over listed pages, forks and compaction. TEST
INFRASTRUCTURE ONLY (see the package docstring).
"""

from __future__ import annotations

import numpy as np

from .chunks import _chunk_tokens


def rotate(x, pos, inv_freq, interleaved=False, weight=None, eps=0.0):
    """One head row x [.., D] at position ``pos``, normalised where ``weight`` is given, in float64.

    Pinned by: norms of pairs kept, rotations of two positions composing to their sum, products of
    rotated rows depending on the distance alone, and multiplication by e^(i a) of complex pairs.
    """
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64) / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    half = len(inv_freq)
    a = float(pos) * np.asarray(inv_freq, dtype=np.float64)
    i = np.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, v = y[..., one].copy(), y[..., two].copy()
    y[..., one] = u * np.cos(a) - v * np.sin(a)
    y[..., two] = v * np.cos(a) + u * np.sin(a)
    return y


def kv_append_chunk_rope(q, k_new, v_new, k_pool, v_pool, block_table, seq_lens, q_indptr, inv_freq, q_weight=None,
                         k_weight=None, eps=1e-6, interleaved=False, q_out=None):
    """(queries, K pool, V pool) in float64; rows of no token as in ``q_out``. Slots past the table's
    row and pages out of range take no K or V."""
    made = np.zeros(q.shape) if q_out is None else np.array(q_out, dtype=np.float64)
    kp, vp = np.array(k_pool, dtype=np.float64), np.array(v_pool, dtype=np.float64)
    P, ps = kp.shape[:2]
    rows, tables, positions = _chunk_tokens(block_table, seq_lens, q_indptr)
    for r, table, pos in zip(rows, tables, positions):
        made[r] = rotate(q[r], pos, inv_freq, interleaved, q_weight, eps)
        if pos // ps < len(table) and 0 <= table[pos // ps] < P:
            kp[table[pos // ps], pos % ps] = rotate(k_new[r], pos, inv_freq, interleaved, k_weight, eps)
            vp[table[pos // ps], pos % ps] = v_new[r]
    return made, kp, vp


_STEP = np.float32(1.0) / np.float32(127.0)


def page_bounds(keys):
    """Codes [H, 2, D] and scales [H] of a page's keys [t, H, D], in float32 as the definition has it."""
    k = np.asarray(keys, dtype=np.float32)
    top, low = k.max(0), k.min(0)
    scale = np.maximum(np.abs(k).max((0, 2)), np.float32(1e-10)) * _STEP
    with np.errstate(invalid="ignore"):
        codes = np.stack([np.clip(np.ceil(top / scale[:, None]), -127, 127),
                          np.clip(np.floor(low / scale[:, None]), -127, 127)], 1)
    bad = ~np.isfinite(k).all((0, 2))
    codes[bad], scale[bad] = 0, np.inf
    return codes.astype(np.int8), scale.astype(np.float32)


def update_page_bounds(k_pool, bounds, scale, block_table, seq_lens, q_indptr):
    """Bounds of the pages that hold a new token; others as they are.

    Pinned by: every key of a page lying between its bounds, and one code less breaking that.
    """
    bounds, scale = bounds.copy(), scale.copy()
    P, ps = k_pool.shape[:2]
    for b in range(len(seq_lens)):
        n, L = int(q_indptr[b + 1]) - int(q_indptr[b]), int(seq_lens[b])
        for slot in range(max(0, L - n) // ps, (L + ps - 1) // ps if n > 0 else 0):
            if slot < block_table.shape[1] and 0 <= block_table[b, slot] < P:
                page = block_table[b, slot]
                bounds[page], scale[page] = page_bounds(k_pool[page, :L - slot * ps])
    return bounds, scale


def page_scores(q, bounds, scale):
    """Scores [n] of pages with codes [n, 2, D] and scales [n] for the query heads q [g, D] of one kv
    head, in float32 as the definition has it."""
    q = np.asarray(q, dtype=np.float32)
    qs = np.maximum(np.abs(q).max(-1), np.float32(1e-10)) * _STEP
    with np.errstate(invalid="ignore", over="ignore"):
        c = np.where(np.isfinite(qs)[:, None], np.clip(np.rint(q / qs[:, None]), -127, 127), 0).astype(np.int64)
        lim = bounds.astype(np.int64)
        dot = np.maximum(c[:, None] * lim[None, :, 0], c[:, None] * lim[None, :, 1]).sum(-1)
        score = dot.astype(np.float32) * qs[:, None] * scale[None].astype(np.float32)
    return np.where(np.isnan(score).any(0), np.inf, score.max(0)), np.isnan(score).any(0)


def select_pages(q, bounds, scale, block_table, seq_lens, page_size, pages, first=1, last=1):
    """Chosen slots int32 [B, q_len, H_kv, pages] for q [B, q_len, H_q, D], by sorting.

    Pinned by: exact scores never below any key's quantized product, and the choice not depending
    on the order in which pages are scored.
    """
    B, q_len, H_q, _ = q.shape
    P, H_kv = scale.shape
    g = H_q // H_kv
    out = np.full((B, q_len, H_kv, pages), -1, dtype=np.int32)
    for b in range(B):
        for j in range(q_len):
            pos = int(seq_lens[b]) - q_len + j
            have = min(pos // page_size + 1 if pos >= 0 else 0, block_table.shape[1])
            for h in range(H_kv):
                if have <= pages:
                    out[b, j, h, :have] = np.arange(have)
                    continue
                middle = np.arange(first, have - last)
                page = block_table[b, middle]
                ok = (page >= 0) & (page < P)
                page = np.where(ok, page, 0)
                score, nan = page_scores(q[b, j, h * g:(h + 1) * g], bounds[page, h], scale[page, h])
                rank = sorted(range(len(middle)), key=lambda i: (-(2 * nan[i] + 1) if ok[i] else 0,
                                                                  -score[i] if ok[i] else 0, i))
                chosen = np.concatenate([np.arange(first), middle[rank[:pages - first - last]],
                                         np.arange(have - last, have)])
                out[b, j, h] = np.sort(chosen)
    return out


def sparse_decode_attention(q, k_pool, v_pool, block_table, seq_lens, page_idx, scale):
    """(O, LSE) of q [B, q_len, H_q, D] over the listed slots, in float64.

    Pinned by: all slots listed equal to :func:`multi_query_decode_attention`, and equality with
    :func:`decode_attention` on a cache that holds the listed pages alone.
    """
    B, q_len, H_q, D = q.shape
    P, ps, H_kv, _ = k_pool.shape
    g = H_q // H_kv
    out, lse = np.zeros(q.shape), np.full(q.shape[:-1], -np.inf)
    for b in range(B):
        for j in range(q_len):
            pos = int(seq_lens[b]) - q_len + j
            for h in range(H_kv):
                k, v = [], []
                for slot in map(int, page_idx[b, j, h][:max(0, pos // ps + 1)]):
                    if slot < 0 or slot * ps > pos or slot >= block_table.shape[1]:
                        continue
                    page = block_table[b, slot]
                    if 0 <= page < P:
                        n = min(ps, pos - slot * ps + 1)
                        k.append(k_pool[page, :n, h])
                        v.append(v_pool[page, :n, h])
                if not k:
                    continue
                k, v = np.concatenate(k).astype(np.float64), np.concatenate(v).astype(np.float64)
                s = scale * q[b, j, h * g:(h + 1) * g].astype(np.float64) @ k.T
                m = s.max(-1, keepdims=True)
                e = np.exp(s - m)
                out[b, j, h * g:(h + 1) * g] = e / e.sum(-1, keepdims=True) @ v
                lse[b, j, h * g:(h + 1) * g] = (m + np.log(e.sum(-1, keepdims=True)))[:, 0]
    return out, lse


def kv_fork(buffers, block_table, seq_lens, parents, children, fresh, page_size):
    """New (buffers, table, lengths) after the forks, entry by entry.

    Pinned by: every sequence reading the same rows through the new table as its parent did.
    """
    buffers, table, lens = [b.copy() for b in buffers], block_table.copy(), seq_lens.copy()
    P = buffers[0].shape[0]
    for parent, child, page in zip(parents, children, fresh):
        if not (0 <= parent < len(lens) and 0 <= child < len(lens)) or parent == child:
            continue
        L = int(lens[parent])
        slots = -(-L // page_size)
        if L < 0 or slots > table.shape[1]:
            continue
        row = table[parent, :slots].copy()
        if L % page_size:
            if not (0 <= row[-1] < P and 0 <= page < P):
                continue
            for b in buffers:
                b[page] = b[row[-1]]
            row[-1] = page
        table[child, :slots] = row
        lens[child] = L
    return buffers, table, lens


def kv_compact(buffers, block_table, seq_lens, page_size):
    """New (buffers, table, page map, pages in use).

    Pinned by: every sequence reading the same rows through the new table, and the pages in use
    being exactly the first ones.
    """
    P = buffers[0].shape[0]
    live = np.arange(block_table.shape[1])[None] * page_size < np.asarray(seq_lens)[:, None]
    live &= (block_table >= 0) & (block_table < P)
    held = sorted({int(p) for p in block_table[live]})
    U = len(held)
    page_map = np.full(P, -1, dtype=np.int32)
    free = iter([p for p in range(U) if p not in set(held)])
    buffers = [b.copy() for b in buffers]
    for p in held:
        page_map[p] = p if p < U else next(free)
    for p in held:
        if page_map[p] != p:
            for b in buffers:
                b[page_map[p]] = b[p]
    table = block_table.copy()
    table[live] = page_map[block_table[live]]
    return buffers, table, page_map, U
