"""GPU parity of chunked-prompt attention (ts_paged_prefill_attn) against the
fp64 oracle, at the sizes and masks where it can go wrong."""

import os

import numpy as np
import pytest
import torch

import paged_kv_cache_46_gb300 as ts
from chunk_cases import DEV, ChunkCase, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _run(case, ctas=None, **over):
    if ctas is not None:
        os.environ["TS_PAGED_DECODE_CTAS"] = str(ctas)
    try:
        a = case.device()
        a.update(over)
        ws = ts.new_workspace(ts.ts_paged_prefill_workspace_size(case.T, len(case.n), case.H_q, case.H_kv, case.D))
        out, lse = ts.ts_paged_prefill_attn(**a, workspace=ws, return_lse=True)
        torch.cuda.synchronize()
        assert ts.ts_read_device_error(ws) == 0
    finally:
        os.environ.pop("TS_PAGED_DECODE_CTAS", None)
    return out, lse


def _check(case, out, lse, what=""):
    check_attention(out, lse, case.oracle(), case.D, int(case.L.max()), case.dtype, what)


@pytest.mark.parametrize("n,ctx", [([1], [0]), ([1], [300]), ([33], [99]), ([128], [0]), ([129], [127]),
                                   ([2, 0, 65], [0, 40, 1000]), ([300, 1, 64, 31], [0, 128, 129, 5])])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths(n, ctx, D, dtype):
    case = ChunkCase(sum(n) + D, n, ctx, 8, 2, D, dtype=dtype)
    _check(case, *_run(case), f"n {n} ctx {ctx}")


@pytest.mark.parametrize("H_q,H_kv", [(1, 1), (4, 4), (6, 2), (8, 1), (14, 2), (64, 1), (32, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_groups(H_q, H_kv, dtype):
    """Group sizes that divide the tile's rows and that do not."""
    case = ChunkCase(H_q * 10 + H_kv, [45, 7], [20, 200], H_q, H_kv, 64, dtype=dtype)
    _check(case, *_run(case), f"{H_q}/{H_kv}")


@pytest.mark.parametrize("ps", [8, 16, 32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (37, 0), (100, 5), (128, 128), (200, 150),
                                          (64, 16), (10000, 3)])
def test_windows_and_first_tokens(ps, D, window, sinks):
    """NaN fills every row between the first tokens and the first query's window."""
    case = ChunkCase(window + sinks + ps, [150, 3, 70], [700, 260, 0], 8, 2, D, ps=ps, window=window, sinks=sinks)
    _check(case, *_run(case), f"W {window} S {sinks} ps {ps}")


@pytest.mark.parametrize("window,sinks", [(1, 0), (70, 9), (100, 64), (64, 200)])
def test_windows_f32(window, sinks):
    case = ChunkCase(window, [150, 3], [400, 260], 8, 2, 64, ps=8, dtype="f32", window=window, sinks=sinks)
    _check(case, *_run(case), f"W {window} S {sinks}")


@pytest.mark.parametrize("ctas", [1, 2, 7, 64, 152, 1000])
@pytest.mark.parametrize("window", [0, 300])
def test_cuts(ctas, window):
    """Items cut between CTAs in every way, down to one key tile each."""
    case = ChunkCase(ctas, [70, 200, 1, 64], [1500, 10, 900, 0], 8, 2, 128, window=window, sinks=20 if window else 0)
    _check(case, *_run(case, ctas), f"{ctas} CTAs")


def test_many_sequences():
    """More sequences than a CTA has threads, some without new tokens."""
    rng = np.random.default_rng(5)
    n = rng.integers(0, 4, size=500)
    case = ChunkCase(5, n, rng.integers(0, 60, size=500), 4, 2, 64)
    _check(case, *_run(case), "500 sequences")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_sequences_than_the_prologue_keeps(dtype):
    """Above 8192 sequences the units of a sequence are counted twice instead of kept."""
    rng = np.random.default_rng(6)
    n = (rng.random(8300) < 0.2).astype(int) * rng.integers(1, 4, size=8300)
    case = ChunkCase(6, n, rng.integers(0, 20, size=8300), 2, 1, 64, ps=8, dtype=dtype)
    _check(case, *_run(case), "8300 sequences")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_a_fused_projection_and_padding(dtype):
    """Strided query rows; rows behind the last sequence stay as they were."""
    case = ChunkCase(8, [40, 0, 90], [17, 3, 0], 8, 2, 64, dtype=dtype, fused=True, pad_rows=21)
    out = torch.full((case.T, 8, 64), 7.0, dtype=case.q.dtype, device=DEV)
    lse = torch.full((case.T, 8), 7.0, device=DEV)
    _run(case, out=out, lse=lse)
    real = int(case.indptr[-1])
    assert torch.all(out[real:] == 7.0) and torch.all(lse[real:] == 7.0)
    ref = case.oracle()
    check_attention(out[:real], lse[:real], (ref[0][:real], ref[1][:real], ref[2][:real], ref[3]), 64,
                    int(case.L.max()), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_in_front_of_the_cache_see_nothing(dtype):
    """seq_lens below the number of new tokens: O = 0, LSE = -inf for the first ones."""
    case = ChunkCase(9, [150, 20, 5], [0, 0, 10], 8, 2, 64, dtype=dtype)
    case.L = np.array([30, 0, 15])  # 120 tokens, all 20, and none without a position
    _check(case, *_run(case))


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales(scale):
    """No weighting at all, the reverse order, and a nearly one-hot softmax (many rescales)."""
    case = ChunkCase(10, [100], [400], 8, 2, 64)
    case.scale = scale
    _check(case, *_run(case), f"scale {scale}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rising_scores(dtype):
    """Scores that grow from key to key move the running maximum in every tile."""
    case = ChunkCase(11, [140], [500], 4, 1, 64, dtype=dtype)
    for t in range(640):
        case.k_pool[case.bt[0, t // 16], t % 16, :, 0] = t / 8.0
    case.q[:, :, 0] = 4.0
    _check(case, *_run(case))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_pages_count_as_absent(dtype):
    """Page ids out of range are not read: their tokens are absent, and the error word says so."""
    case = ChunkCase(12, [70], [230], 8, 2, 64, dtype=dtype)
    a = case.device()
    bt = case.bt.copy()
    bt[0, 3], bt[0, 9], bt[0, 10] = -1, 1 << 30, case.k_pool.shape[0]
    a["block_table"] = torch.from_numpy(bt).to(DEV)
    ws = ts.new_workspace(ts.ts_paged_prefill_workspace_size(case.T, 1, 8, 2, 64))
    out, lse = ts.ts_paged_prefill_attn(**a, workspace=ws, return_lse=True)
    torch.cuda.synchronize()
    assert ts.ts_read_device_error(ws) == ts.TS_DEVERR_PAGE_RANGE
    # the oracle: absent tokens score -inf, written with keys far below all others and no value
    o = np.zeros((70, 8, 64))
    l = np.zeros((70, 8))
    a_ref = np.zeros_like(o)
    q, k, v = (x.double().numpy() for x in (case.q, case.k_pool, case.v_pool))
    for j in range(70):
        t = np.arange(230 + j + 1)
        t = t[~np.isin(t // 16, [3, 9, 10])]
        K, V = k[case.bt[0, t // 16], t % 16], v[case.bt[0, t // 16], t % 16]
        for h in range(8):
            s = K[:, h // 4] @ q[j, h] * case.scale
            e = np.exp(s - s.max())
            l[j, h] = s.max() + np.log(e.sum())
            o[j, h] = e @ V[:, h // 4] / e.sum()
            a_ref[j, h] = e @ np.abs(V[:, h // 4]) / e.sum()
    check_attention(out, lse, (o, l, a_ref, case.oracle()[3]), 64, 300, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_past_the_block_table(dtype):
    """Tokens that seq_lens counts past the table's row are absent and flagged."""
    case = ChunkCase(13, [10], [54], 4, 2, 64, dtype=dtype)
    a = case.device()
    a["seq_lens"] = torch.tensor([64 + 40], dtype=torch.int32, device=DEV)
    ws = ts.new_workspace(ts.ts_paged_prefill_workspace_size(10, 1, 4, 2, 64))
    out, lse = ts.ts_paged_prefill_attn(**a, workspace=ws, return_lse=True)
    torch.cuda.synchronize()
    assert ts.ts_read_device_error(ws) == ts.TS_DEVERR_PAGE_RANGE
    case.n, case.L = np.array([10]), np.array([64])
    q, k, v = (x.double().numpy() for x in (case.q, case.k_pool, case.v_pool))
    t = np.arange(64)
    K, V = k[case.bt[0, t // 16], t % 16], v[case.bt[0, t // 16], t % 16]
    s = np.einsum("jhd,thd->jht", q, np.repeat(K, 2, 1)) * case.scale
    e = np.exp(s - s.max(-1, keepdims=True))
    o = np.einsum("jht,thd->jhd", e, np.repeat(V, 2, 1)) / e.sum(-1)[..., None]
    a_ref = np.einsum("jht,thd->jhd", e, np.abs(np.repeat(V, 2, 1))) / e.sum(-1)[..., None]
    check_attention(out, lse, (o, s.max(-1) + np.log(e.sum(-1)), a_ref, case.oracle()[3]), 64, 64, dtype)


@pytest.mark.parametrize("indptr", [[0, 50, 20, 60], [-3, 10, 20, 30], [0, 20, 40, 4000], [60, 40, 20, 0]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_offsets_out_of_order_stay_in_bounds(indptr, dtype):
    """Which rows are taken is not defined, but nothing outside the batch is touched."""
    case = ChunkCase(14, [20, 20, 20], [5, 5, 5], 4, 2, 64, dtype=dtype)
    a = case.device()
    a["q_indptr"] = torch.tensor(indptr, dtype=torch.int32, device=DEV)
    room = torch.full((60 + 128, 4, 64), 7.0, dtype=case.q.dtype, device=DEV)
    ts.ts_paged_prefill_attn(**a, out=room[64:124])
    torch.cuda.synchronize()
    assert torch.all(room[:64] == 7.0) and torch.all(room[124:] == 7.0)


def test_equal_calls_give_equal_bits():
    case = ChunkCase(15, [200, 31], [900, 40], 8, 2, 128)
    first, first_lse = _run(case)
    for _ in range(3):
        out, lse = _run(case)
        assert torch.equal(out, first) and torch.equal(lse, first_lse)


def test_captured_and_replayed_with_other_lengths():
    """One capture, replayed with new lengths and row offsets written in place,
    two graphs over workspaces of their own on two streams."""
    cases = [ChunkCase(16, [40, 90], [100, 0], 8, 2, 64), ChunkCase(17, [90, 40], [10, 300], 8, 2, 64)]
    graphs = []
    for case in cases:
        a = case.device()
        ws = ts.new_workspace(ts.ts_paged_prefill_workspace_size(case.T, 2, 8, 2, 64))
        out = torch.zeros(case.T, 8, 64, dtype=torch.bfloat16, device=DEV)
        lse = torch.zeros(case.T, 8, device=DEV)
        ts.ts_paged_prefill_attn(**a, workspace=ws, out=out, lse=lse)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ts.ts_paged_prefill_attn(**a, workspace=ws, out=out, lse=lse)
        graphs.append((g, a, ws, out, lse))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for n in ([40, 90], [1, 20], [100, 0]):
        for case, (g, a, ws, out, lse), s in zip(cases, graphs, streams):
            ctx = case.L - case.n
            case.n = np.minimum(np.array(n), case.L)
            case.indptr = np.concatenate([[0], np.cumsum(case.n)]).astype(np.int32)
            a["q_indptr"].copy_(torch.from_numpy(case.indptr))
            out.zero_(), lse.fill_(float("-inf"))
        torch.cuda.synchronize()
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for case, (g, a, ws, out, lse) in zip(cases, graphs):
            assert ts.ts_read_device_error(ws) == 0
            check_attention(out, lse, case.oracle(), 64, int(case.L.max()), "bf16", f"replay {n}")


def test_on_a_stream_of_its_own():
    case = ChunkCase(18, [64], [64], 8, 2, 64)
    s = torch.cuda.Stream()
    a = case.device()
    torch.cuda.synchronize()
    out, lse = ts.ts_paged_prefill_attn(**a, stream=s, workspace=ts.new_workspace(
        ts.ts_paged_prefill_workspace_size(case.T, 1, 8, 2, 64)), return_lse=True)
    s.synchronize()
    _check(case, out, lse)


def test_chunk_by_chunk_equals_whole_prompt():
    """A prompt in one chunk and in three, over the same cache."""
    whole = ChunkCase(19, [300], [0], 8, 2, 128)
    ref, ref_lse = _run(whole)
    a = whole.device()
    at = 0
    for n in (130, 1, 169):
        a2 = dict(a, q=a["q"][at:at + n], seq_lens=torch.tensor([at + n], dtype=torch.int32, device=DEV),
                  q_indptr=torch.tensor([0, n], dtype=torch.int32, device=DEV))
        out, lse = ts.ts_paged_prefill_attn(**a2, return_lse=True)
        o = tuple(x[at:at + n] for x in whole.oracle()[:3]) + (whole.oracle()[3],)
        check_attention(out, lse, o, 128, 300, "bf16", f"chunk at {at}")
        at += n
    _check(whole, ref, ref_lse)


@pytest.mark.parametrize("D,window,sinks", [(64, 0, 0), (64, 1024, 64), (128, 0, 0), (128, 1024, 64)])
def test_many_key_tiles_in_flight(D, window, sinks):
    """Long runs of products, whose scores, weights and sums take turns in the same columns: an
    order that is not enforced shows as rare wrong rows that differ from call to call."""
    case = ChunkCase(D + window, [1100, 900, 700], [2500, 1200, 0], 16, 4, D, window=window, sinks=sinks)
    ref = case.oracle()
    first, first_lse = _run(case)
    check_attention(first, first_lse, ref, D, int(case.L.max()), "bf16")
    for _ in range(20):
        out, lse = _run(case)
        assert torch.equal(out, first) and torch.equal(lse, first_lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_that_share_pages(dtype):
    """Two rows of the block table with the same pages: one prompt, two different chunks of it."""
    case = ChunkCase(21, [70], [130], 8, 2, 64, dtype=dtype)
    case.bt = np.repeat(case.bt, 2, axis=0)
    case.n, case.L = np.array([20, 50]), np.array([200, 100])
    case.indptr = np.array([0, 20, 70], dtype=np.int32)
    _check(case, *_run(case))


def test_what_a_call_allocates_belongs_to_its_stream(monkeypatch):
    """Memory freed while a call runs on a stream of its own is handed on in that stream's order."""
    case = ChunkCase(22, [64], [64], 8, 2, 64)
    s = torch.cuda.Stream()
    a = case.device()
    torch.cuda.synchronize()
    made = []
    new = ts.new_workspace
    monkeypatch.setattr(ts, "new_workspace", lambda *x: made.append(torch.cuda.current_stream()) or new(*x))
    for stream in (s, s.cuda_stream):
        out, lse = ts.ts_paged_prefill_attn(**a, stream=stream, return_lse=True)
        s.synchronize()
        _check(case, out, lse)
    q = a["q"][:1].contiguous()
    ts.ts_paged_decode_sink_attn(q, a["k_pool"], a["v_pool"], a["block_table"], a["seq_lens"], case.scale, 32, 4,
                                 stream=s)
    s.synchronize()
    assert [x.cuda_stream for x in made] == [s.cuda_stream] * 3


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H_q,n,ctx,window,sinks", [(64, [78, 75, 73], [13577, 16660, 18228], 2193, 35),
                                                    (32, [17, 33, 1, 5], [1000, 2000, 3000, 500], 0, 0)])
def test_tiles_with_the_buffers_for_themselves(H_q, n, ctx, window, sinks, D):
    """The last, short items of sequences: their only tile's scores run ahead of V tiles that are
    late. Calls behind one another, of two batches in turn, give equal bits, and the right ones."""
    cases = [ChunkCase(23 + i, n, ctx, H_q, 8, D, window=window, sinks=sinks) for i in range(2)]
    args = [c.device() for c in cases]
    ws = [ts.new_workspace(ts.ts_paged_prefill_workspace_size(c.T, len(n), H_q, 8, D)) for c in cases]
    first = [ts.ts_paged_prefill_attn(**a, workspace=w, return_lse=True) for a, w in zip(args, ws)]
    _check(cases[0], *first[0])
    off = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(200):
        for a, w, (out, lse) in zip(args, ws, first):
            got = ts.ts_paged_prefill_attn(**a, workspace=w, return_lse=True)
            off += (got[0] != out).sum() + (got[1] != lse).sum()
    assert off.item() == 0
    assert all(ts.ts_read_device_error(w) == 0 for w in ws)


@pytest.mark.parametrize("indptr", [[0, 50, 20, 60], [-3, 10, 20, 30], [0, 20, 40, 4000], [60, 40, 20, 0],
                                    [0, 60, 0, 60], [2 ** 31 - 1, -2 ** 31, 0, 60]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_offsets_out_of_order_reach_nothing_else_and_end(indptr, dtype):
    """Guards behind the workspace's stated size and around O and LSE stay; no role waits its limit out."""
    case = ChunkCase(14, [20, 20, 20], [400, 5, 1000], 4, 2, 64, dtype=dtype, window=0)
    a = case.device()
    a["q_indptr"] = torch.tensor(indptr, dtype=torch.int32, device=DEV)
    size = ts.ts_paged_prefill_workspace_size(60, 3, 4, 2, 64)
    room = ts.new_workspace(size + 4096)
    room[size:] = 0x5a
    out = torch.full((60 + 128, 4, 64), 7.0, dtype=case.q.dtype, device=DEV)
    lse = torch.full((60 + 128, 4), 7.0, device=DEV)
    ts.ts_paged_prefill_attn(**a, out=out[64:124], lse=lse[64:124], workspace=room[:size])
    torch.cuda.synchronize()
    assert ts.ts_read_device_error(room) & ts.TS_DEVERR_TIMEOUT == 0
    assert torch.all(room[size:] == 0x5a)
    for t in (out, lse):
        assert torch.all(t[:64] == 7.0) and torch.all(t[124:] == 7.0)
