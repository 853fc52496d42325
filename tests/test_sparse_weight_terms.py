"""The weights of ts_paged_decode_sparse_attn's bf16 products count with two bf16 terms.

Half of the tokens have the score 0 and the value -c, half the score -x and the value 1,
with c = e^-x rounded to bf16: the result is (e^-x - c) / (1 + e^-x), what the rounding of
the weight leaves. With weights rounded once it would be 0.

Bound, with A = sum_t softmax_t |V_t| and L tokens: the score is one exact product times a
rounded factor (two roundings of a base-2 score of 2 at most: 2 * 2 * 2^-24 ln 2 of the weight),
2^s is off by 2^-22 of itself at most, and a weight's second term, 2^-8 of it at most, by 2^-8 of
itself: 2^-16 + 7 * 2^-24. The sums of L weights and of L values: 2 (2 L + 2) 2^-24, each
addition off by two half units at most, a join's two products and its division by the sum
6 * 2^-24. The result's own rounding is 2^-8 of it."""

import numpy as np
import pytest
import torch

import oracle

X = [0.62890625, 1.1171875, 0.53125, 0.62109375]  # of one kv head each: c is a third of a step or more from e^-x


def _bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16).double().numpy()


def _inputs(pages, ps, H_kv, g, D, B=2):
    P = B * pages + 1
    order = np.random.default_rng(pages).permutation(P)
    table = order[:-1].reshape(B, pages).astype(np.int32)
    lens = np.array([pages * ps, pages * ps - 6][:B])
    q, k, v = np.zeros((B, 1, H_kv * g, D)), np.zeros((P, ps, H_kv, D)), np.zeros((P, ps, H_kv, D))
    q[..., 0] = 1.0
    x = np.array([X[h % len(X)] for h in range(H_kv)])
    k[:, 1::2, :, 0] = -x
    sign = np.where(np.arange(D) % 3 == 0, -1.0, 1.0) * 2.0 ** (np.arange(D) % 5)
    v[:, 1::2] = sign
    v[:, ::2] = -_bf16(np.exp(-x))[:, None] * sign
    k[order[-1]] = v[order[-1]] = np.nan
    idx = np.broadcast_to(np.arange(pages, dtype=np.int32), (B, 1, H_kv, pages)).copy()
    return q, k, v, table, lens, idx


def _bound(q, k, v, table, lens, idx):
    o, _ = oracle.sparse_decode_attention(q, k, v, table, lens, idx, 1.0)
    a, _ = oracle.sparse_decode_attention(q, k, np.abs(v), table, lens, idx, 1.0)
    L = lens.max()
    return o, 1.01 * (2.0 ** -8 * np.abs(o) + (2.0 ** -16 + (7 + 4 * L + 4 + 6) * 2.0 ** -24) * a)


def test_weights_rounded_once_miss_the_bound():
    q, k, v, table, lens, idx = _inputs(6, 16, 4, 1, 64)
    o, bound = _bound(q, k, v, table, lens, idx)
    assert np.all(_bf16(k[table[0, 0]]) == k[table[0, 0]]) and np.all(_bf16(v[table[0, 0]]) == v[table[0, 0]])
    for b in range(2):
        for h in range(4):
            t = np.arange(lens[b])
            keys, values = (x[table[b, t // 16], t % 16, h] for x in (k, v))
            w = np.exp(keys[:, 0])
            once = _bf16(w)
            rest = _bf16(w - once)
            wrong = np.abs(once @ values / w.sum() - o[b, 0, h])
            assert np.all(wrong > 4 * bound[b, 0, h])
            assert np.all(np.abs((once + rest) @ values / w.sum() - o[b, 0, h]) < 0.2 * bound[b, 0, h])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 4, 8])
@pytest.mark.parametrize("ps", [8, 16, 32])
@pytest.mark.parametrize("ctas", [None, "1"])  # whole in a CTA, cut and joined
def test_weights_count_with_two_terms(D, g, ps, ctas, monkeypatch):
    import paged_kv_cache_46_gb300 as ts
    from long_context_cases import DEV, i32
    if ctas is not None:
        monkeypatch.setenv("TS_PAGED_DECODE_CTAS", ctas)
    q, k, v, table, lens, idx = _inputs(6, ps, 4, g, D)
    o, bound = _bound(q, k, v, table, lens, idx)
    out = ts.ts_paged_decode_sparse_attn(*(torch.from_numpy(x).to(torch.bfloat16).to(DEV) for x in (q, k, v)),
                                         i32(table), i32(lens), i32(idx), 1.0)
    err = np.abs(out.double().cpu().numpy() - o)
    assert np.all(err <= bound), f"off by {np.max(err / bound):.2f} of its bound"
