"""Long-context calls at sizes, orders and neighbours that single-call tests do not
reach: tens of thousands of rows, empty batches, two streams at once, a whole step in
one captured graph, and calls that follow one another without a wait."""

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_46_gb300 as ts
from chunk_cases import check_attention
from long_context_cases import DEV, Cache, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _small_batch(seed, lens, g, H_kv, D, ps, dtype="bf16"):
    c = Cache(seed, lens, H_kv, D, ps, dtype)
    q = c.normal(len(lens), g * H_kv, D)
    codes, scale = c.bounds()
    return c, q, torch.from_numpy(codes).to(DEV), torch.from_numpy(scale).to(DEV)


def test_tens_of_thousands_of_rows_equal_the_rows_alone():
    """50 sequences, and the same 50 again and again: 70,000 rows."""
    lens = np.random.default_rng(91).integers(0, 120, 50)
    c, q, codes, scale = _small_batch(91, lens, 2, 2, 64, 8)
    d = c.device()
    times = 1400
    few = dict(block_table=d["block_table"], seq_lens=d["seq_lens"])
    many = dict(block_table=d["block_table"].repeat(times, 1), seq_lens=d["seq_lens"].repeat(times))
    q = q.to(DEV)
    idx = ts.ts_select_pages(q, codes, scale, page_size=8, pages=6, **few)
    want = oracle.select_pages(q[:, None].double().cpu().numpy(), codes.cpu().numpy(), scale.cpu().numpy(), c.table,
                               c.lens, 8, 6)
    assert np.array_equal(idx.cpu().numpy(), want[:, 0])
    all_idx = ts.ts_select_pages(q.repeat(times, 1, 1), codes, scale, page_size=8, pages=6, **many)
    assert torch.equal(all_idx.view(times, *idx.shape), idx.expand(times, *idx.shape))
    pools = dict(k_pool=d["k_pool"], v_pool=d["v_pool"], scale=0.125, return_lse=True)
    out, lse = ts.ts_paged_decode_sparse_attn(q.repeat(times, 1, 1), page_idx=all_idx, **pools, **many)
    a = oracle.sparse_decode_attention(q[:, None].double().cpu().numpy(), *(x.double().numpy() for x in
                                       (c.k_pool, c.v_pool)), c.table, c.lens, want, 0.125)
    b, _ = oracle.sparse_decode_attention(q[:, None].double().cpu().numpy(), c.k_pool.double().numpy(),
                                          c.v_pool.double().abs().numpy(), c.table, c.lens, want, 0.125)
    reach = 0.125 * np.nanmax(c.k_pool.double().abs().sum(-1).numpy()) * float(q.abs().max())
    for part in (0, 700, times - 1):
        rows = slice(part * 50, part * 50 + 50)
        check_attention(out[rows], lse[rows], (a[0][:, 0], a[1][:, 0], b[:, 0], reach), 64, 48, "bf16")


def test_empty_batches():
    c, q, codes, scale = _small_batch(92, [30, 7], 2, 2, 64, 8)
    d = c.device()
    none = dict(block_table=d["block_table"][:0], seq_lens=d["seq_lens"][:0])
    q = q.to(DEV)
    idx = ts.ts_select_pages(q[:0], codes, scale, page_size=8, pages=3, **none)
    assert idx.shape == (0, 2, 3)
    out = ts.ts_paged_decode_sparse_attn(q[:0], d["k_pool"], d["v_pool"], page_idx=idx, scale=1.0, **none)
    assert out.shape == (0, 4, 64)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    rows = ts.ts_kv_append_chunk_rope(q[:0], q[:0, :2], q[:0, :2], d["k_pool"], d["v_pool"], q_indptr=one,
                                      inv_freq=torch.ones(32, device=DEV), **none)
    assert rows.shape == (0, 4, 64)
    ts.ts_kv_page_bounds(d["k_pool"], codes, scale, q_indptr=one, rows=0, **none)


def test_sequences_without_tokens_beside_others():
    for lens in ([0, 0, 0], [0, 900, 0], [1, 0, 900]):
        c, q, codes, scale = _small_batch(93, lens, 4, 2, 128, 16)
        d = c.device()
        q = q.to(DEV)
        idx = ts.ts_select_pages(q, codes, scale, d["block_table"], d["seq_lens"], 16, 9)
        out, lse = ts.ts_paged_decode_sparse_attn(q, **d, page_idx=idx, scale=0.1, return_lse=True)
        none = torch.from_numpy(c.lens == 0).to(DEV)
        assert (idx[none] == -1).all() and not out[none].any() and torch.isneginf(lse[none]).all()
        assert torch.isfinite(out).all() and torch.isfinite(lse[~none]).all()


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own."""
    runs = []
    for seed in (94, 95):
        c, q, codes, scale = _small_batch(seed, [3000, 1500, 40, 800], 4, 4, 128, 16)
        d, q = c.device(), q.to(DEV)
        ws = [ts.new_workspace(n) for n in (ts.ts_select_pages_workspace_size(4, 1, 4, c.table.shape[1]),
                                            ts.ts_paged_decode_sparse_workspace_size(4, 1, 16, 4, 128, 16, 30))]
        idx = ts.ts_select_pages(q, codes, scale, d["block_table"], d["seq_lens"], 16, 30, workspace=ws[0])
        out, lse = ts.ts_paged_decode_sparse_attn(q, **d, page_idx=idx, scale=0.1, return_lse=True, workspace=ws[1])
        runs.append((q, codes, scale, d, ws, idx, out, lse, torch.cuda.Stream()))
    torch.cuda.synchronize()
    results = []
    for _ in range(20):
        for q, codes, scale, d, ws, *_, stream in runs:
            i = ts.ts_select_pages(q, codes, scale, d["block_table"], d["seq_lens"], 16, 30, workspace=ws[0],
                                   stream=stream)
            o, l = ts.ts_paged_decode_sparse_attn(q, **d, page_idx=i, scale=0.1, return_lse=True, workspace=ws[1],
                                                  stream=stream)
            results.append((i, o, l))
    torch.cuda.synchronize()
    for n, (i, o, l) in enumerate(results):
        *_, idx, out, lse, _ = runs[n % 2]
        assert torch.equal(i, idx) and torch.equal(o, out) and torch.equal(l, lse)


def test_a_captured_step_follows_its_lengths():
    """Append, bounds, selection and attention of a decode step in one graph, replayed token by token."""
    H_q, H_kv, D, ps, B = 8, 2, 128, 16, 3
    c = Cache(96, [700, 33, 160], H_kv, D, ps, spare=12, slots=4)
    free = list(c.free)
    for b in range(B):  # pages for the tokens to come
        for slot in range(-(-int(c.lens[b]) // ps), -(-int(c.lens[b] + 20) // ps)):
            c.table[b, slot] = free.pop()
    d = c.device()
    codes, scale = c.bounds()
    a = dict(codes=torch.from_numpy(codes).to(DEV), scale=torch.from_numpy(scale).to(DEV))
    x = c.normal(20, B, H_q + 2 * H_kv, D).to(DEV)
    row, ptr = torch.zeros_like(x[0]), i32(np.arange(B + 1))
    freq = torch.from_numpy(10000.0 ** (-np.arange(D // 2) / (D // 2))).float().to(DEV)
    ws = [ts.new_workspace(n) for n in (ts.ts_select_pages_workspace_size(B, 1, H_kv, c.table.shape[1]),
                                        ts.ts_paged_decode_sparse_workspace_size(B, 1, H_q, H_kv, D, ps, 8))]
    lens = d["seq_lens"]

    def step():
        q, k, v = row.split([H_q, H_kv, H_kv], 1)
        q = ts.ts_kv_append_chunk_rope(q, k, v, d["k_pool"], d["v_pool"], d["block_table"], lens, ptr, freq)
        ts.ts_kv_page_bounds(d["k_pool"], a["codes"], a["scale"], d["block_table"], lens, ptr, B)
        idx = ts.ts_select_pages(q, a["codes"], a["scale"], d["block_table"], lens, ps, 8, workspace=ws[0])
        return q, idx, *ts.ts_paged_decode_sparse_attn(q, **d, page_idx=idx, scale=D ** -0.5, return_lse=True,
                                                       workspace=ws[1])

    row.copy_(x[0])
    lens += 1
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, idx, out, lse = step()
    for t in range(1, 20):
        row.copy_(x[t])
        lens += 1
        graph.replay()
        torch.cuda.synchronize()
        if t % 6:
            continue
        L = lens.cpu().numpy()
        k, v, qd = (y.double().cpu().numpy() for y in (d["k_pool"], d["v_pool"], q[:, None]))
        want = oracle.select_pages(qd, a["codes"].cpu().numpy(), a["scale"].cpu().numpy(), c.table, L, ps, 8)
        assert np.array_equal(idx.cpu().numpy(), want[:, 0])
        o, l = oracle.sparse_decode_attention(qd, k, v, c.table, L, want, D ** -0.5)
        b, _ = oracle.sparse_decode_attention(qd, k, np.abs(v), c.table, L, want, D ** -0.5)
        reach = D ** -0.5 * np.nanmax(np.abs(k).sum(-1)) * np.abs(qd).max()
        check_attention(out, lse, (o[:, 0], l[:, 0], b[:, 0], reach), D, 8 * ps, "bf16")


def test_attention_right_behind_a_fork():
    """Attention reads tables and lengths before it waits for the kernel in front of it: a fork must be over by then."""
    lens = [300, 77, 48]
    c = Cache(97, lens + [0] * 3, 4, 128, 16, spare=8, slots=1)
    d = c.device()
    plan = ts.kv_buffers([d["k_pool"], d["v_pool"]])
    q = c.normal(6, 16, 128).to(DEV)
    fresh = i32(c.free[:3])
    table, zero = d["block_table"].clone(), d["seq_lens"].clone()
    want = ts.ts_paged_decode_attn(q, **d, scale=0.1)[:3]
    order = [torch.tensor(p, dtype=torch.int32, device=DEV) for p in ([3, 4, 5], [5, 4, 3], [4, 3, 5])]
    asked = []
    for o in order:
        asked.append(q.clone())
        asked[-1][o.long()] = q[:3]
    parents = i32([0, 1, 2])
    for n in range(60):
        children = order[n % 3]
        d["block_table"].copy_(table)
        d["seq_lens"].copy_(zero)
        ts.ts_kv_fork(plan, d["block_table"], d["seq_lens"], parents, children, fresh, 16)
        out = ts.ts_paged_decode_attn(asked[n % 3], **d, scale=0.1)  # row children[i] asks what row i asks
        assert torch.equal(out[:3], want) and torch.equal(out[children.long()], want), n


def test_attention_right_behind_a_compaction():
    for seed in range(98, 108):
        c = Cache(seed, [300, 77, 48, 1000, 20], 4, 128, 16, spare=60)
        keep = [0, 2, 3]
        k, v = c.k_pool.to(DEV), c.v_pool.to(DEV)
        table, lens = i32(c.table[keep]), i32(c.lens[keep])
        q = c.normal(3, 16, 128).to(DEV)
        want = ts.ts_paged_decode_attn(q, k, v, table, lens, 0.1)
        ts.ts_kv_compact([k, v], table, lens, 16, table_out=table)
        out = ts.ts_paged_decode_attn(q, k, v, table, lens, 0.1)
        assert torch.equal(out, want)


def test_results_are_left_alone_where_no_row_belongs():
    """Guards around results and workspaces stay as they were."""
    c, q, codes, scale = _small_batch(109, [900, 30, 2000], 4, 2, 128, 16)
    d, q = c.device(), q.to(DEV)
    B, K = 3, 11

    def guarded(shape, dtype, fill):
        n = int(np.prod(shape))
        room = torch.full((n + 256,), fill, dtype=dtype, device=DEV)
        return room, room[128:128 + n].view(shape)

    room_i, idx = guarded((B, 2, K), torch.int32, 77)
    room_o, out = guarded(tuple(q.shape), q.dtype, 5.0)
    room_l, lse = guarded((B, 8), torch.float32, 5.0)
    sizes = (ts.ts_select_pages_workspace_size(B, 1, 2, c.table.shape[1]),
             ts.ts_paged_decode_sparse_workspace_size(B, 1, 8, 2, 128, 16, K))
    rooms = [torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device=DEV) for n in sizes]
    ws = [r[:n] for r, n in zip(rooms, sizes)]
    ts.ts_select_pages(q, codes, scale, d["block_table"], d["seq_lens"], 16, K, page_idx=idx, workspace=ws[0])
    ts.ts_paged_decode_sparse_attn(q, **d, page_idx=idx, scale=0.1, out=out, lse=lse, workspace=ws[1])
    torch.cuda.synchronize()
    for room, view, fill in ((room_i, idx, 77), (room_o, out, 5.0), (room_l, lse, 5.0)):
        assert (room[:128] == fill).all() and (room[128 + view.numel():] == fill).all()
        assert not (view == fill).any()
    assert all((r[n:] == 0xAB).all() for r, n in zip(rooms, sizes))
    # a workspace with anything in it gives what a zeroed one gives
    i2 = ts.ts_select_pages(q, codes, scale, d["block_table"], d["seq_lens"], 16, K)
    o2, l2 = ts.ts_paged_decode_sparse_attn(q, **d, page_idx=i2, scale=0.1, return_lse=True)
    assert torch.equal(i2, idx) and torch.equal(o2, out) and torch.equal(l2, lse)
