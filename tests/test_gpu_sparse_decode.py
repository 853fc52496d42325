"""GPU parity of ts_paged_decode_sparse_attn, held to the bounds of chunk_cases. Rows
that no query may read are NaN."""

import os

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


def _lists(c, q_len, pages, order="ascending"):
    """Distinct slots of each row, the last one among them; -1 where there are none."""
    out = np.full((len(c.lens), q_len, c.H_kv, pages), -1, dtype=np.int32)
    for b, L in enumerate(c.lens):
        for j in range(q_len):
            have = max(0, (int(L) - q_len + j) // c.ps + 1)
            for h in range(c.H_kv):
                n = min(pages, have)
                pick = c.rng.permutation(have)[:n]
                if n and have - 1 not in pick:
                    pick[0] = have - 1
                out[b, j, h, :n] = np.sort(pick)
                if order == "any":
                    out[b, j, h, :n] = c.rng.permutation(out[b, j, h, :n])
    return out


def _run(c, q, idx, ctas=None, scale=None, single=False):
    scale = c.D ** -0.5 if scale is None else scale
    if ctas is not None:
        os.environ["TS_PAGED_DECODE_CTAS"] = str(ctas)
    try:
        B, q_len, H_q, D = q.shape
        ws = ts.new_workspace(ts.ts_paged_decode_sparse_workspace_size(B, q_len, H_q, c.H_kv, D, c.ps, idx.shape[-1]))
        d = c.device()
        x, i = (q[:, 0], idx[:, 0]) if single else (q, idx)
        out, lse = ts.ts_paged_decode_sparse_attn(x.to(DEV), d["k_pool"], d["v_pool"], d["block_table"], d["seq_lens"],
                                                  i32(i), scale, workspace=ws, return_lse=True)
        assert out.shape == x.shape and lse.shape == x.shape[:-1]
        return out.view(q.shape), lse.view(q.shape[:-1]), ts.ts_read_device_error(ws)
    finally:
        os.environ.pop("TS_PAGED_DECODE_CTAS", None)


def _check(c, q, idx, out, lse, scale=None, what=""):
    scale = c.D ** -0.5 if scale is None else scale
    qd, k, v = (x.double().numpy() for x in (q, c.k_pool, c.v_pool))
    o, l = oracle.sparse_decode_attention(qd, k, v, c.table, c.lens, idx, scale)
    a, _ = oracle.sparse_decode_attention(qd, k, np.abs(v), c.table, c.lens, idx, scale)
    reach = np.nanmax(np.abs(k).sum(-1)) if np.isfinite(k).any() else 0.0
    qk = abs(scale) * reach * np.abs(qd).max()
    check_attention(out, lse, (o, l, a, qk), c.D, idx.shape[-1] * c.ps, "bf16" if c.dtype == torch.bfloat16 else "f32",
                    what)


def _case(seed, lens, q_len, g, H_kv, D, pages, ps=16, dtype="bf16", order="ascending", **kw):
    c = Cache(seed, lens, H_kv, D, ps, dtype, **kw)
    return c, c.normal(len(lens), q_len, g * H_kv, D), _lists(c, q_len, pages, order)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g,H_kv", [(4, 8), (1, 1), (2, 4), (8, 2), (8, 1), (1, 8)])
@pytest.mark.parametrize("ps", [8, 16, 32])
@pytest.mark.parametrize("ctas", [None, 1])  # items whole, and cut into even ranges
def test_shapes(dtype, D, g, H_kv, ps, ctas):
    c, q, idx = _case(51, [700, 1, 0, 16, 333, 64], 1, g, H_kv, D, 9, ps, dtype)
    out, lse, err = _run(c, q, idx, ctas)
    assert err == 0
    _check(c, q, idx, out, lse)


@pytest.mark.parametrize("pages", [1, 2, 3, 5, 17, 64, 200])
@pytest.mark.parametrize("ctas", [1, 3, 40, 1000])
def test_lists_of_any_length_cut_anywhere(pages, ctas):
    c, q, idx = _case(52, [1700, 31, 500], 1, 4, 2, 128, pages, order="any")
    out, lse, err = _run(c, q, idx, ctas)
    assert err == 0
    _check(c, q, idx, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [2, 5, 17])
@pytest.mark.parametrize("ctas", [None, 3])
def test_several_tokens(dtype, q_len, ctas):
    c, q, idx = _case(53, [300, 18, 3, 16 * 9 + 2], q_len, 4, 2, 64, 7, dtype=dtype, order="any")
    out, lse, err = _run(c, q, idx, ctas)
    assert err == 0
    _check(c, q, idx, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_all_pages_listed_is_the_whole_attention(dtype):
    c, q, _ = _case(54, [900, 100, 16], 1, 4, 2, 128, 1, dtype=dtype)
    idx = np.broadcast_to(np.arange(57, dtype=np.int32), (3, 1, 2, 57)).copy()
    out, lse, _ = _run(c, q, idx)
    d = c.device()
    o, l = ts.ts_paged_decode_attn(q[:, 0].contiguous().to(DEV), d["k_pool"], d["v_pool"], d["block_table"],
                                   d["seq_lens"], c.D ** -0.5, return_lse=True)
    tol = 2.0 ** -6 if dtype == "bf16" else 1e-5
    # bf16: two outputs rounded once each (2^-8 of a value below 4 at these inputs: 2^-6 / 2 each) and weights
    # rounded to bf16 in one of them at most; float32: sums of 900 weights and values in different orders
    assert (out[:, 0].float() - o.float()).abs().max() <= tol
    assert (lse[:, 0] - l).abs().max() <= 1e-4


@pytest.mark.parametrize("ctas", [None, 1])
def test_entries_that_are_not_pages(ctas):
    c, q, idx = _case(55, [200, 90, 40], 2, 2, 2, 64, 6, slots=3)
    idx[0, 0, 0] = [-1, -5, 12, -(2 ** 31), -1, 3]
    idx[0, 1, 1] = -1                                   # sees nothing
    idx[1, 0, 0] = [2 ** 31 - 1, 1000000, 6, 7, 5, -1]  # behind the position: skipped, not absent pages
    idx[2, 1, 0] = [2, 2, 1, 1, 0, -1]                  # a slot twice; three pages: three entries are taken
    out, lse, err = _run(c, q, idx, ctas)
    assert err == 0
    _check(c, q, idx, out, lse)
    assert not out[0, 1, 2:].any() and torch.isneginf(lse[0, 1, 2:]).all()


@pytest.mark.parametrize("ctas", [None, 1])
def test_bad_pages_are_absent_and_flagged(ctas):
    c, q, idx = _case(56, [400, 300, 200], 1, 4, 2, 128, 12)
    c.table[0, 3:20] = c.P
    c.table[1, 0:9] = -1
    out, lse, err = _run(c, q, idx, ctas)
    assert err == ts.TS_DEVERR_PAGE_RANGE
    _check(c, q, idx, out, lse)
    c, q, idx = _case(57, [400, 300, 200], 1, 4, 2, 128, 12)
    c.table = np.ascontiguousarray(c.table[:, :11])  # lists name slots past the table's row
    out, lse, err = _run(c, q, idx, ctas)
    assert err == ts.TS_DEVERR_PAGE_RANGE
    _check(c, q, idx, out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(scale):
    c, q, idx = _case(58, [500, 77], 1, 4, 2, 64, 10)
    for ctas in (None, 1):
        out, lse, _ = _run(c, q, idx, ctas, scale=scale)
        _check(c, q, idx, out, lse, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_are_not_finite(dtype):
    c, q, idx = _case(59, [640, 640, 640], 1, 2, 2, 64, 40, dtype=dtype)
    want, l_want, _ = _run(c, q, idx)
    c.k_pool[c.table[0, 5], 3, 1] = float("nan")
    c.k_pool[c.table[1, 0], 0, 0, 7] = float("inf")  # scores of + and - infinity
    c.v_pool[c.table[2, 9], 2, 0, 11] = float("nan")
    for ctas in (1, 50, None):
        out, lse, _ = _run(c, q, idx, ctas)
        assert torch.isnan(out[0, 0, 2:]).all() and torch.isnan(lse[0, 0, 2:]).all()
        up = (q[1, 0, :2, 7] > 0).to(DEV)
        assert torch.isnan(out[1, 0, :2][up]).all() and torch.isnan(lse[1, 0, :2][up]).all()
        assert torch.isfinite(out[1, 0, :2][~up]).all() and torch.isfinite(lse[1, 0, :2][~up]).all()
        assert torch.isnan(out[2, 0, :2, 11]).all() and torch.isfinite(lse[2]).all()
        assert torch.isfinite(out[0, 0, :2]).all() and torch.isfinite(out[1, 0, 2:]).all()
    minus = torch.full_like(c.k_pool, 0.0)
    minus[..., 0] = float("inf")
    c.k_pool = minus
    q[:, :, :, 0] = -1.0
    c.v_pool = torch.nan_to_num(c.v_pool)
    for ctas in (1, None):
        out, lse, _ = _run(c, q, idx, ctas)  # every score is -infinity: nothing is seen
        assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_values_make_their_columns_infinite(dtype):
    c, q, idx = _case(64, [640, 640], 1, 4, 2, 64, 40, dtype=dtype)
    want = _run(c, q, idx)[0]
    c.v_pool[c.table[0, 7], 3, 1, 9] = float("inf")
    c.v_pool[c.table[1, 30], 15, 0, 0] = -float("inf")
    for ctas in (1, 50, None):
        out, lse, _ = _run(c, q, idx, ctas)
        assert (out[0, 0, 4:, 9] == float("inf")).all() and (out[1, 0, :4, 0] == -float("inf")).all()
        out[0, 0, 4:, 9], out[1, 0, :4, 0] = want[0, 0, 4:, 9], want[1, 0, :4, 0]
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_rising_scores():
    """Each page's scores far above those before: every step moves the reference."""
    c, q, _ = _case(60, [1600], 1, 4, 1, 64, 1, dtype="f32")
    q[:] = 0
    q[..., 0] = 1.0
    for s in range(100):
        c.k_pool[c.table[0, s], :, :, 0] += 3.0 * s
    idx = np.arange(100, dtype=np.int32).reshape(1, 1, 1, 100)
    for ctas in (1, 1000):
        out, lse, _ = _run(c, q, idx, ctas, scale=1.0)
        _check(c, q, idx, out, lse, 1.0)
        out, lse, _ = _run(c, q, idx[..., ::-1].copy(), ctas, scale=1.0)
        _check(c, q, idx, out, lse, 1.0)


def test_equal_calls_give_equal_bits_and_workspaces_may_be_shared_in_order():
    c, q, idx = _case(61, [1700, 31, 500], 1, 4, 2, 128, 60)
    for ctas in (None, 2):
        first, l_first, _ = _run(c, q, idx, ctas, single=True)
        for _ in range(5):
            out, lse, _ = _run(c, q, idx, ctas, single=True)
            assert torch.equal(out, first) and torch.equal(lse, l_first)


@pytest.mark.parametrize("ctas", ["152", "1"])
def test_captured_step_with_other_lists_and_lengths(ctas, monkeypatch):
    monkeypatch.setenv("TS_PAGED_DECODE_CTAS", ctas)
    c, q, idx = _case(62, [1000, 64, 300], 1, 4, 2, 64, 20)
    d = c.device()
    ws = ts.new_workspace(ts.ts_paged_decode_sparse_workspace_size(3, 1, 8, 2, 64, 16, 20))
    a = dict(q=q[:, 0].to(DEV), **d, page_idx=i32(idx[:, 0]), scale=0.125, workspace=ws)
    a["out"], a["lse"] = torch.zeros_like(a["q"]), torch.zeros(3, 8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ts.ts_paged_decode_sparse_attn(**a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ts.ts_paged_decode_sparse_attn(**a)
    for lens in ([999, 17, 300], [40, 0, 1]):
        c.lens = np.array(lens)
        idx = _lists(c, 1, 20, "any")
        a["seq_lens"].copy_(i32(lens))
        a["page_idx"].copy_(i32(idx[:, 0]))
        graph.replay()
        torch.cuda.synchronize()
        _check(c, q, idx, a["out"].view(q.shape), a["lse"].view(3, 1, 8))


@pytest.mark.parametrize("ctas", ["152", "1"])
def test_pages_past_two_to_the_31_elements(ctas, monkeypatch):
    """A pool of 4.3 G elements: the listed pages lie at its end."""
    P, ps, H_kv, D = (1 << 18) + 100, 16, 8, 128
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("not enough free memory")
    monkeypatch.setenv("TS_PAGED_DECODE_CTAS", ctas)
    k, v = (torch.empty(P, ps, H_kv, D, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    c, q, idx = _case(63, [500, 100], 1, 4, 8, 128, 10)
    at = P - c.P
    k[at:], v[at:] = c.k_pool.to(DEV), c.v_pool.to(DEV)
    assert at * ps * H_kv * D > 1 << 32
    out, lse = ts.ts_paged_decode_sparse_attn(q[:, 0].contiguous().to(DEV), k, v, i32(c.table + at), i32(c.lens),
                                              i32(idx[:, 0]), D ** -0.5, return_lse=True)
    _check(c, q, idx, out.view(q.shape), lse.view(q.shape[:-1]))
