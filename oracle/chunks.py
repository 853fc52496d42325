"""fp64 oracle of prompts served in chunks: the attention of a ragged batch of
chunks over a paged cache, decode attention with first tokens that stay
visible beside a sliding window, the chunk appends and the read-back of a
quantized cache. TEST INFRASTRUCTURE ONLY (see the package docstring).

A chunk batch is one array of rows: rows ``q_indptr[b] .. q_indptr[b + 1] - 1``
are sequence ``b``'s newest tokens, which ``seq_lens[b]`` counts already, so
row ``q_indptr[b] + j`` of ``n`` sits at position ``seq_lens[b] - n + j``.
"""

from __future__ import annotations

import numpy as np

from .attention import gather_sequence, kv_append
from .fp8 import dequantize, kv_append_fp8


def visible(pos: int, window: int, sinks: int) -> np.ndarray:
    """Positions that the token at ``pos`` attends: all up to itself or, with a
    window, its last ``window`` tokens and the sequence's first ``sinks``."""
    t = np.arange(max(0, pos + 1))
    return t if window == 0 else t[(t > pos - window) | (t < sinks)]


def _attend_visible(q, k_pool, v_pool, block_table, pos, b, scale, window, sinks):
    """One query row [H_q, D] at position ``pos`` of sequence ``b``."""
    H_q = q.shape[0]
    if pos < 0:
        return np.zeros((H_q, v_pool.shape[3])), np.full(H_q, -np.inf)
    t, ps = visible(pos, window, sinks), k_pool.shape[1]
    pages = np.asarray(block_table[b])[t // ps]
    K, V = k_pool[pages, t % ps].astype(np.float64), v_pool[pages, t % ps].astype(np.float64)
    g = H_q // K.shape[1]
    s = scale * np.einsum("hgd,thd->hgt", q.reshape(-1, g, q.shape[1]).astype(np.float64), K)
    m = s.max(axis=-1, keepdims=True)
    e = np.exp(s - m)
    total = e.sum(axis=-1, keepdims=True)
    o = np.einsum("hgt,thd->hgd", e / total, V).reshape(H_q, -1)
    return o, (m + np.log(total)).reshape(H_q)


def decode_attention_sinks(q, k_pool, v_pool, block_table, seq_lens, scale, window, sinks):
    """Decode attention where the query of a sequence of ``L`` tokens attends
    its last ``window`` tokens and its first ``sinks``, in float64.

    Pinned by: no first tokens equal to :func:`decode_attention_window`, window
    + sinks >= L equal to :func:`decode_attention`, equality with
    :func:`decode_attention` on a cache re-paged to hold only the visible
    tokens, NaN in every other row, and a planted off-by-one caught.
    """
    rows = [_attend_visible(q[b], k_pool, v_pool, block_table, int(seq_lens[b]) - 1, b, scale, window, sinks)
            for b in range(len(seq_lens))]
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


def prefill_attention(q, k_pool, v_pool, block_table, seq_lens, q_indptr, scale, window=0, sinks=0):
    """Attention of a ragged batch of chunks, q [T, H_q, D], in float64.

    SwiftLLM page, section 5.1 (query, block tables, context lengths), causal,
    with the window and first tokens of :func:`decode_attention_sinks` where
    ``window`` > 0. Rows of no sequence give O = 0 and LSE = -inf here.

    Pinned by: torch's fp64 scaled_dot_product_attention with an explicit mask
    on contiguous K/V, equality with :func:`multi_query_decode_attention` for
    chunks of one length, and a planted off-by-one mask caught.
    """
    T, H_q, _ = q.shape
    out, lse = np.zeros((T, H_q, v_pool.shape[3])), np.full((T, H_q), -np.inf)
    for b in range(len(seq_lens)):
        r0, r1 = int(q_indptr[b]), int(q_indptr[b + 1])
        for r in range(r0, r1):
            out[r], lse[r] = _attend_visible(q[r], k_pool, v_pool, block_table, int(seq_lens[b]) - (r1 - r), b, scale,
                                             window, sinks)
    return out, lse


def _chunk_tokens(block_table, seq_lens, q_indptr):
    """(batch row, block-table row, position) of every new token with a position."""
    rows, tables, positions = [], [], []
    for b in range(len(seq_lens)):
        r0, r1 = int(q_indptr[b]), int(q_indptr[b + 1])
        for r in range(r0, r1):
            pos = int(seq_lens[b]) - (r1 - r)
            if pos >= 0:
                rows.append(r)
                tables.append(np.asarray(block_table[b]))
                positions.append(pos)
    return np.asarray(rows, dtype=np.int64), tables, positions


def kv_append_chunk(k_pool, v_pool, k_new, v_new, block_table, seq_lens, q_indptr):
    """Write the K/V rows of a chunk batch: :func:`kv_append` of each token.

    Pinned by: equality with single-token appends in order of position.
    """
    rows, tables, pos = _chunk_tokens(block_table, seq_lens, q_indptr)
    return kv_append(k_pool, v_pool, k_new[rows], v_new[rows], tables, pos, k_pool.shape[1])


def kv_append_chunk_fp8(k_pool, v_pool, k_scale, v_scale, k_new, v_new, block_table, seq_lens, q_indptr):
    """Quantize the K/V rows of a chunk batch: :func:`kv_append_fp8` of each token."""
    rows, tables, pos = _chunk_tokens(block_table, seq_lens, q_indptr)
    return kv_append_fp8(k_pool, v_pool, k_scale, v_scale, k_new[rows], v_new[rows], tables, pos, k_pool.shape[1])


def kv_read_fp8(pool, scale, block_table, seq_lens, kv_indptr, out):
    """Rows of a quantized cache in float32 (code times scale); other rows of
    ``out`` as they are. One pool at a time.

    Pinned by: torch's float8_e4m3fn conversion of the gathered codes.
    """
    made = np.array(out, dtype=np.float32, copy=True)
    ps = pool.shape[1]
    for b in range(len(seq_lens)):
        r0 = int(kv_indptr[b])
        n = min(int(seq_lens[b]), int(kv_indptr[b + 1]) - r0)
        made[r0:r0 + n] = dequantize(gather_sequence(pool, block_table[b], n, ps),
                                     gather_sequence(scale, block_table[b], n, ps))
    return made

