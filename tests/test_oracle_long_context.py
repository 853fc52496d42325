"""Pins of the long-context oracle to something other than itself (CPU)."""

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    rng = np.random.default_rng(1)
    x, f = rng.normal(size=(3, 64)), 10000.0 ** (-np.arange(16) / 16)
    y = oracle.rotate(x, 777, f, interleaved)
    assert np.array_equal(y[:, 32:], x[:, 32:])  # columns behind the rotated ones
    one, two = (np.arange(0, 32, 2), np.arange(1, 32, 2)) if interleaved else (np.arange(16), np.arange(16, 32))
    z = (x[:, one] + 1j * x[:, two]) * np.exp(1j * 777 * f)
    assert np.allclose(y[:, one] + 1j * y[:, two], z, rtol=0, atol=1e-12)
    twice = oracle.rotate(oracle.rotate(x, 500, f, interleaved), 277, f, interleaved)
    assert np.allclose(twice, y, rtol=0, atol=1e-12)
    a, b = rng.normal(size=64), rng.normal(size=64)
    near = oracle.rotate(a, 40, f, interleaved) @ oracle.rotate(b, 31, f, interleaved)
    far = oracle.rotate(a, 9040, f, interleaved) @ oracle.rotate(b, 9031, f, interleaved)
    assert abs(near - far) < 1e-10
    w = rng.normal(size=64)
    n = oracle.rotate(x, 0, f, interleaved, w, 0.0)
    assert np.allclose(((n / w) ** 2).mean(-1), 1.0)


def test_bounds_hold_their_keys_and_no_code_less_does():
    rng = np.random.default_rng(2)
    k = (rng.normal(size=(16, 4, 64)) * np.exp(rng.normal(size=(1, 4, 64)))).astype(np.float32)
    codes, scale = oracle.page_bounds(k)
    s = scale.astype(np.float64)[:, None]
    # the scale is rounded down by at most 2 units, so the largest key may pass 127 steps by that
    slack = 127 * s * 2.0 ** -22
    top, low = k.max(0).astype(np.float64), k.min(0).astype(np.float64)
    assert np.all(codes[:, 0] * s >= top - slack) and np.all((codes[:, 0] - 1.0) * s < top + slack)
    assert np.all(codes[:, 1] * s <= low + slack) and np.all((codes[:, 1] + 1.0) * s > low - slack)
    k[3, 2, 5] = np.inf
    codes, scale = oracle.page_bounds(k)
    assert np.isinf(scale[2]) and not codes[2].any() and np.isfinite(scale[[0, 1, 3]]).all()


def test_scores_bound_the_quantized_products():
    rng = np.random.default_rng(3)
    k, q = rng.normal(size=(50, 16, 1, 64)).astype(np.float32), rng.normal(size=(4, 64)).astype(np.float32)
    pages = [oracle.page_bounds(x) for x in k]
    codes, scale = np.stack([c[0] for c, _ in pages]), np.stack([s[0] for _, s in pages])
    score, nan = oracle.page_scores(q, codes, scale)
    qs = np.abs(q).max(-1, keepdims=True) / 127
    product = (np.rint(q / qs) * qs) @ k[:, :, 0].transpose(0, 2, 1)  # [50, 4, 16]
    assert not nan.any() and np.all(score >= product.max((1, 2)) - 1e-4)


def _case(seed, lens, q_len=1, H_q=4, H_kv=2, D=64, ps=8):
    rng = np.random.default_rng(seed)
    need = [-(-n // ps) for n in lens]
    P = sum(need) + 3
    order = rng.permutation(P)
    table, at = np.full((len(lens), max(need) + 1), order[-1], dtype=np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    k, v = rng.normal(size=(P, ps, H_kv, D)), rng.normal(size=(P, ps, H_kv, D))
    return rng.normal(size=(len(lens), q_len, H_q, D)), k, v, table, np.asarray(lens, dtype=np.int32), rng


def test_selection_is_the_best_pages_in_any_order_of_scoring():
    q, k, _, table, lens, rng = _case(4, [300, 40, 7], q_len=2)
    bounds, scale = (np.stack(x) for x in zip(*(oracle.page_bounds(page) for page in k)))
    idx = oracle.select_pages(q, bounds, scale, table, lens, 8, 9, first=2, last=3)
    assert idx.shape == (3, 2, 2, 9)
    assert np.array_equal(idx[1, 1, 0], [0, 1, 2, 3, 4, -1, -1, -1, -1]) and (idx[2, :, :, 0] == 0).all()
    for h in range(2):
        got = idx[0, 1, h]
        assert list(got) == sorted(got) and list(got[:2]) == [0, 1] and list(got[-3:]) == [35, 36, 37]
        score, _ = oracle.page_scores(q[0, 1, 2 * h:2 * h + 2], bounds[table[0, :38], h], scale[table[0, :38], h])
        rest = np.setdiff1d(np.arange(2, 35), got)
        assert score[got[2:-3]].min() >= score[rest].max()
    same = np.zeros_like(bounds)
    idx = oracle.select_pages(q, same, np.ones_like(scale), table, lens, 8, 9, first=2, last=3)
    assert list(idx[0, 0, 0]) == [0, 1, 2, 3, 4, 5, 35, 36, 37]  # equal scores: the lowest pages


def test_sparse_attention_over_all_pages_and_over_a_cache_of_the_listed_ones():
    q, k, v, table, lens, rng = _case(5, [61, 24, 2], q_len=2)
    every = np.broadcast_to(np.arange(9), (3, 2, 2, 9))
    o, lse = oracle.sparse_decode_attention(q, k, v, table, lens, every, 0.125)
    o_ref, l_ref = oracle.multi_query_decode_attention(q, k, v, table, lens, 0.125)
    assert np.allclose(o, o_ref, atol=1e-12) and np.allclose(lse, l_ref, atol=1e-12)
    idx = np.full((3, 1, 2, 4), -1)
    idx[0, 0] = [[7, 2, -1, 0], [1, 7, 5, 6]]
    o, lse = oracle.sparse_decode_attention(q[:, :1], k, v, table, lens, idx, 0.125)
    for h in range(2):
        slots = [s for s in idx[0, 0, h] if 0 <= s < 7] + [7]
        mine = table[:1, slots]
        o_ref, l_ref = oracle.decode_attention(q[:1, 0], k, v, mine, np.array([8 * (len(slots) - 1) + 5]),
                                               0.125)
        assert np.allclose(o[0, 0, 2 * h:2 * h + 2], o_ref[0, 2 * h:2 * h + 2], atol=1e-12)
        assert np.allclose(lse[0, 0, 2 * h:2 * h + 2], l_ref[0, 2 * h:2 * h + 2], atol=1e-12)
    assert not o[1].any() and np.isneginf(lse[1]).all()


def _rows(pool, table, lens, ps):
    return [oracle.gather_sequence(pool, table[b], int(lens[b]), ps) for b in range(len(lens))]


def test_forks_read_what_their_parents_read():
    _, k, v, table, lens, rng = _case(6, [61, 24, 2, 0, 0, 0])
    table[3:] = -7
    free = [p for p in range(len(k)) if p not in table[:3]]
    want = _rows(k, table, lens, 8)
    (k2, v2), t2, l2 = oracle.kv_fork([k, v], table, lens, [0, 0, 1], [5, 3, 4], [*free[:2], -1], 8)
    for child, parent in ((5, 0), (3, 0), (4, 1)):
        assert l2[child] == lens[parent]
        assert np.array_equal(_rows(k2, t2, l2, 8)[child], want[parent])
    assert np.array_equal(_rows(k2, t2, l2, 8)[0], want[0])
    assert t2[5, 7] == free[0] and t2[3, 7] == free[1] and np.array_equal(t2[5, :7], table[0, :7])
    assert np.array_equal(t2[4, :3], table[1, :3]) and (t2[4, 3:] == -7).all()


def test_compaction_keeps_what_sequences_read():
    _, k, v, table, lens, rng = _case(7, [61, 24, 2, 100, 9])
    keep = [1, 3, 4]
    table, lens = table[keep], lens[keep]
    table[2, :1] = table[1, :1]  # a shared page
    want = _rows(k, table, lens, 8)
    (k2, _), t2, page_map, used = oracle.kv_compact([k, v], table, lens, 8)
    assert all(np.array_equal(a, b) for a, b in zip(want, _rows(k2, t2, lens, 8)))
    assert used == 3 + 13 + 1 and sorted(page_map[page_map >= 0]) == list(range(used))
    assert all(page_map[p] in (p, -1) for p in range(used))
