"""Pins of the chunk oracle: library attention with an explicit mask, the older
oracle functions where the operations coincide, and planted mistakes."""

import numpy as np
import pytest
import torch

import oracle


def _cache(rng, lens, H_kv, D, ps, spare=3):
    """Shuffled pages with NaN in every row that no token owns."""
    need = [(L + ps - 1) // ps for L in lens]
    P = sum(need) + spare
    order = rng.permutation(P)
    bt = np.full((len(lens), max(1, max(need))), order[-1], dtype=np.int32)
    k, v = np.full((P, ps, H_kv, D), np.nan), np.full((P, ps, H_kv, D), np.nan)
    at = 0
    for b, L in enumerate(lens):
        bt[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for t in range(L):
            k[bt[b, t // ps], t % ps] = rng.standard_normal((H_kv, D))
            v[bt[b, t // ps], t % ps] = rng.standard_normal((H_kv, D))
    return k, v, bt


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (5, 3), (1, 0), (1, 20), (100, 7)])
def test_prefill_is_masked_sdpa(window, sinks):
    rng = np.random.default_rng(window * 31 + sinks)
    lens, n, H_q, H_kv, D, ps = [13, 40, 7, 21], [13, 9, 0, 1], 4, 2, 16, 8
    k, v, bt = _cache(rng, lens, H_kv, D, ps)
    indptr = np.concatenate([[0], np.cumsum(n)])
    q = rng.standard_normal((indptr[-1], H_q, D))
    out, lse = oracle.prefill_attention(q, k, v, bt, lens, indptr, 0.3, window, sinks)
    for b, L in enumerate(lens):
        if n[b] == 0:
            continue
        K = torch.from_numpy(oracle.gather_sequence(k, bt[b], L, ps)).permute(1, 0, 2).repeat_interleave(2, 0)
        V = torch.from_numpy(oracle.gather_sequence(v, bt[b], L, ps)).permute(1, 0, 2).repeat_interleave(2, 0)
        Q = torch.from_numpy(q[indptr[b]:indptr[b + 1]]).permute(1, 0, 2)
        mask = torch.zeros(n[b], L, dtype=torch.bool)
        for j in range(n[b]):
            for t in range(L - n[b] + j + 1):
                mask[j, t] = window == 0 or L - n[b] + j - t < window or t < sinks
        ref = torch.nn.functional.scaled_dot_product_attention(Q, K, V, attn_mask=mask, scale=0.3).permute(1, 0, 2)
        assert np.abs(ref.numpy() - out[indptr[b]:indptr[b + 1]]).max() < 1e-12
        s = (Q @ K.transpose(1, 2) * 0.3).masked_fill(~mask, float("-inf"))
        assert np.abs(torch.logsumexp(s, 2).T.numpy() - lse[indptr[b]:indptr[b + 1]]).max() < 1e-12


def test_prefill_of_equal_chunks_is_multi_query_decode():
    rng = np.random.default_rng(1)
    lens, n = [9, 30], 4
    k, v, bt = _cache(rng, lens, 2, 16, 8)
    q = rng.standard_normal((2, n, 4, 16))
    out, lse = oracle.prefill_attention(q.reshape(2 * n, 4, 16), k, v, bt, lens, [0, n, 2 * n], 0.25)
    ref, ref_lse = oracle.multi_query_decode_attention(q, k, v, bt, lens, 0.25)
    assert np.abs(out.reshape(ref.shape) - ref).max() < 1e-12
    assert np.abs(lse.reshape(ref_lse.shape) - ref_lse).max() < 1e-12


def test_rows_without_a_position_see_nothing():
    rng = np.random.default_rng(2)
    k, v, bt = _cache(rng, [2], 1, 16, 8)
    out, lse = oracle.prefill_attention(rng.standard_normal((5, 1, 16)), k, v, bt, [2], [0, 5], 0.25)
    assert np.all(out[:3] == 0) and np.all(np.isneginf(lse[:3])) and np.all(np.isfinite(lse[3:]))


@pytest.mark.parametrize("window,sinks", [(6, 3), (1, 1), (8, 8), (4, 0), (3, 17)])
def test_sinks_decode_equals_decode_of_the_visible_tokens(window, sinks):
    rng = np.random.default_rng(window + 100 * sinks)
    lens, ps = [30, 3, 1, 0, 17], 8
    k, v, bt = _cache(rng, lens, 2, 16, ps)
    q = rng.standard_normal((len(lens), 4, 16))
    out, lse = oracle.decode_attention_sinks(q, k, v, bt, lens, 0.25, window, sinks)
    kept = [[t for t in range(L) if t >= L - window or t < sinks] for L in lens]
    k2, v2, bt2 = _cache(rng, [len(x) for x in kept], 2, 16, ps)
    for b, ts_ in enumerate(kept):
        for i, t in enumerate(ts_):
            k2[bt2[b, i // ps], i % ps] = k[bt[b, t // ps], t % ps]
            v2[bt2[b, i // ps], i % ps] = v[bt[b, t // ps], t % ps]
    ref, ref_lse = oracle.decode_attention(q, k2, v2, bt2, [len(x) for x in kept], 0.25)
    assert np.abs(out - ref).max() < 1e-12
    fin = np.isfinite(ref_lse)
    assert np.array_equal(fin, np.isfinite(lse)) and np.abs(lse[fin] - ref_lse[fin]).max() < 1e-12
    if sinks == 0:
        win, _ = oracle.decode_attention_window(q, k, v, bt, lens, 0.25, window)
        assert np.abs(out - win).max() < 1e-12
    off, _ = oracle.decode_attention_sinks(q, k, v, bt, lens, 0.25, window, sinks + 1)
    if sinks + window < 30:
        assert np.abs(off - out).max() > 1e-3


def test_chunk_append_is_single_appends_in_order():
    rng = np.random.default_rng(3)
    lens, n, ps = [11, 5, 8], [11, 0, 3], 4
    k, v, bt = _cache(rng, lens, 1, 16, ps)
    indptr = np.concatenate([[0], np.cumsum(n)])
    kn, vn = rng.standard_normal((14, 1, 16)), rng.standard_normal((14, 1, 16))
    got = oracle.kv_append_chunk(k, v, kn, vn, bt, lens, indptr)
    for b in (0, 2):
        for j in range(n[b]):
            k, v = oracle.kv_append(k, v, kn[indptr[b] + j][None], vn[indptr[b] + j][None], bt[b][None],
                                    [lens[b] - n[b] + j], ps)
    assert np.array_equal(got[0], k, equal_nan=True) and np.array_equal(got[1], v, equal_nan=True)


def test_read_back_is_torchs_conversion():
    rng = np.random.default_rng(4)
    lens, ps = [5, 0, 9], 4
    _, _, bt = _cache(rng, lens, 2, 16, ps)
    P = int(bt.max()) + 1
    pool = rng.integers(0, 126, size=(P, ps, 2, 16)).astype(np.uint8)
    scale = rng.random((P, ps, 2)).astype(np.float32)
    out = rng.standard_normal((24, 2, 16)).astype(np.float32)
    indptr = [1, 9, 9, 20]
    got = oracle.kv_read_fp8(pool, scale, bt, lens, indptr, out)
    val = torch.from_numpy(pool).view(torch.float8_e4m3fn).float().numpy() * scale[..., None]
    ref = out.copy()
    for b, L in enumerate(lens):
        for t in range(L):
            ref[indptr[b] + t] = val[bt[b, t // ps], t % ps]
    assert np.array_equal(got, ref)
