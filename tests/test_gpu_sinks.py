"""GPU parity of decode with a sliding window and first tokens that stay
visible (ts_paged_decode_sink_attn). Every row that no query may read is NaN,
and the slots without a visible token point at an all-NaN page."""

import os

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_46_gb300 as ts
from chunk_cases import DEV, ChunkCase, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _case(seed, lens, H_q, H_kv, D, window, sinks, ps=16, dtype="bf16"):
    """One new token per sequence; a length of zero is a sequence without any."""
    lens = np.asarray(lens)
    return ChunkCase(seed, (lens > 0).astype(int), np.maximum(lens - 1, 0), H_q, H_kv, D, ps=ps, dtype=dtype,
                     window=window, sinks=sinks)


def _run(case, ctas=None):
    if ctas is not None:
        os.environ["TS_PAGED_DECODE_CTAS"] = str(ctas)
    try:
        a = case.device()
        q = torch.zeros(len(case.L), case.H_q, case.D, dtype=case.q.dtype, device=DEV)
        q[torch.from_numpy(case.L > 0).to(DEV)] = a["q"]
        ws = ts.new_workspace(ts.ts_paged_decode_workspace_size(len(case.L), case.H_q, case.D))
        out, lse = ts.ts_paged_decode_sink_attn(q, a["k_pool"], a["v_pool"], a["block_table"], a["seq_lens"],
                                                case.scale, case.window, case.sinks, workspace=ws, return_lse=True)
        torch.cuda.synchronize()
        assert ts.ts_read_device_error(ws) == 0
    finally:
        os.environ.pop("TS_PAGED_DECODE_CTAS", None)
    return out, lse, q


def _check(case, out, lse, q, what=""):
    """The bounds of chunk_cases; this path keeps the weights in float32 for bf16 too, and its
    logarithms and quotients are the fast ones, 2^-21 of the value: within the same bounds."""
    qd, k, v = (x.double().cpu().numpy() for x in (q, case.k_pool, case.v_pool))
    args = (case.bt, case.L, case.scale, case.window, case.sinks)
    o, l = oracle.decode_attention_sinks(qd, k, v, *args)
    a, _ = oracle.decode_attention_sinks(qd, k, np.abs(v), *args)
    qk = case.scale * np.nanmax(np.abs(k).sum(-1)) * np.abs(qd).max()
    check_attention(out, lse, (o, l, a, qk), case.D, int(case.L.max()), case.dtype, what)


@pytest.mark.parametrize("window,sinks,ps", [(100, 4, 16), (100, 16, 16), (37, 20, 8), (1, 1, 16), (1, 33, 32),
                                             (64, 64, 32), (500, 3, 8), (16, 16, 16), (90, 200, 16)])
@pytest.mark.parametrize("H_q,H_kv,D,dtype", [(32, 8, 128, "bf16"), (8, 8, 64, "bf16"), (16, 2, 64, "f32"),
                                              (4, 1, 128, "f32"), (4, 2, 64, "bf16")])
def test_sinks_match_oracle(window, sinks, ps, H_q, H_kv, D, dtype):
    """Lengths around the point where the window leaves the first tokens, page borders, 0 and 1."""
    both = window + sinks
    lens = [both, both + 1, max(1, both - 1), 1, 0, window, both + ps, both + ps - 1, both + 2 * ps + 3, 700]
    case = _case(both + ps, lens, H_q, H_kv, D, window, sinks, ps, dtype)
    _check(case, *_run(case), f"W {window} S {sinks} ps {ps}")


@pytest.mark.parametrize("ctas", [1, 2, 7, 152, 1000])
def test_windows_cut_across_ctas(ctas):
    case = _case(ctas, [4000, 801, 1234, 3999, 799, 33], 8, 2, 64, 800, 50)
    _check(case, *_run(case, ctas), f"{ctas} CTAs")


def test_more_sequences_than_threads():
    rng = np.random.default_rng(3)
    case = _case(3, rng.integers(0, 200, size=700), 4, 2, 64, 40, 5)
    _check(case, *_run(case), "700 sequences")


def test_no_first_tokens_is_the_window_and_a_covering_window_is_plain_decode():
    case = _case(4, [5, 100, 17, 300, 1, 64, 2048, 999], 32, 8, 128, 0, 0)
    a = case.device()
    args = (a["q"], a["k_pool"], a["v_pool"], a["block_table"], a["seq_lens"], case.scale)
    for got, want in ((ts.ts_paged_decode_sink_attn(*args, 128, 0, return_lse=True),
                       ts.ts_paged_decode_window_attn(*args, 128, return_lse=True)),
                      (ts.ts_paged_decode_sink_attn(*args, 2000, 48, return_lse=True),
                       ts.ts_paged_decode_attn(*args, return_lse=True))):
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bad_pages_are_flagged():
    case = _case(5, [400], 8, 2, 64, 100, 20)
    a = case.device()
    for slot in (1, 20):  # a page of the first tokens, one of the window's
        bt = case.bt.copy()
        bt[0, slot] = case.k_pool.shape[0]
        ws = ts.new_workspace(ts.ts_paged_decode_workspace_size(1, 8, 64))
        out = ts.ts_paged_decode_sink_attn(a["q"], a["k_pool"], a["v_pool"], torch.from_numpy(bt).to(DEV),
                                           a["seq_lens"], case.scale, 100, 20, workspace=ws)
        torch.cuda.synchronize()
        assert ts.ts_read_device_error(ws) == ts.TS_DEVERR_PAGE_RANGE and torch.all(torch.isfinite(out))
    bt = case.bt.copy()
    bt[0, 5] = -1  # between the two: never looked at
    ws = ts.new_workspace(ts.ts_paged_decode_workspace_size(1, 8, 64))
    ts.ts_paged_decode_sink_attn(a["q"], a["k_pool"], a["v_pool"], torch.from_numpy(bt).to(DEV), a["seq_lens"],
                                 case.scale, 100, 20, workspace=ws)
    torch.cuda.synchronize()
    assert ts.ts_read_device_error(ws) == 0


def test_captured_and_replayed_with_longer_contexts():
    case = _case(6, [300, 150], 8, 2, 64, 64, 10)
    a = case.device()
    full = ChunkCase(6, [1, 1], [299, 149], 8, 2, 64)  # a cache without NaN in front of the window
    kp, vp, bt = full.k_pool.to(DEV), full.v_pool.to(DEV), torch.from_numpy(full.bt).to(DEV)
    lens = torch.tensor([40, 30], dtype=torch.int32, device=DEV)
    ws = ts.new_workspace(ts.ts_paged_decode_workspace_size(2, 8, 64))
    out, lse = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 8, device=DEV)
    run = lambda: ts.ts_paged_decode_sink_attn(a["q"], kp, vp, bt, lens, case.scale, 64, 10, out=out, lse=lse,  # noqa: E731
                                               workspace=ws)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for new in ([40, 30], [74, 75], [300, 150], [0, 1]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        full.L, full.window, full.sinks = np.array(new), 64, 10
        _check(full, out, lse, a["q"], f"{new}")
