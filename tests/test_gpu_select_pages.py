"""GPU parity of ts_kv_page_bounds and ts_select_pages. Both are exact: codes, scales
and choices equal the definition's bit for bit, so nothing has a tolerance."""

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_46_gb300 as ts
from long_context_cases import DEV, DTYPES, Cache, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _bounds_args(c, n, seed=0):
    d = c.device()
    g = torch.Generator().manual_seed(seed)
    bounds = torch.randint(-127, 128, (c.P, c.H_kv, 2, c.D), generator=g, dtype=torch.int8).to(DEV)
    scale = torch.rand(c.P, c.H_kv, generator=g).to(DEV)
    return dict(k_pool=d["k_pool"], bounds=bounds, bound_scale=scale, block_table=d["block_table"],
                seq_lens=d["seq_lens"], q_indptr=i32(np.concatenate([[0], np.cumsum(n)])), rows=int(np.sum(n)))


def _check_bounds(c, a, n):
    before = a["bounds"].cpu().numpy().copy(), a["bound_scale"].cpu().numpy().copy()
    ts.ts_kv_page_bounds(**a)
    want = oracle.update_page_bounds(a["k_pool"].float().cpu().numpy(), *before, c.table, c.lens,
                                     np.concatenate([[0], np.cumsum(n)]))
    assert np.array_equal(a["bounds"].cpu().numpy(), want[0])
    assert np.array_equal(a["bound_scale"].cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H_kv,ps", [(8, 16), (1, 8), (2, 32), (4, 1), (3, 7), (11, 50)])
def test_bounds(dtype, D, H_kv, ps):
    n = [1, 0, 17, 64, 5, 1]
    c = Cache(21, np.array([0, 9, 31, 0, 400, 16]) + n, H_kv, D, ps, dtype)
    _check_bounds(c, _bounds_args(c, n), n)


def test_bounds_of_many_rows():
    rng = np.random.default_rng(22)
    n = rng.integers(0, 300, 30)  # more rows than a warp each
    n[3], n[4] = 0, 1
    c = Cache(22, n + rng.integers(0, 60, 30), 2, 64)
    assert n.sum() > 2048
    _check_bounds(c, _bounds_args(c, n), n)


def test_bounds_of_one_new_token_each_and_of_a_whole_cache():
    lens = np.arange(1, 70)
    c = Cache(23, lens, 2, 128)
    _check_bounds(c, _bounds_args(c, np.ones(69, dtype=int)), np.ones(69, dtype=int))
    _check_bounds(c, _bounds_args(c, lens), lens)


def test_bounds_skip_what_is_out_of_range():
    n = [20, 20, 6]
    c = Cache(24, [40, 50, 4], 2, 64, slots=1)
    c.table[0, 1] = c.P
    c.table[1, 2] = -5
    c.lens[2] = 4  # two of its six rows lie in front of the first token
    c.table = np.ascontiguousarray(c.table[:, :3])  # sequence 1 is longer than its row
    _check_bounds(c, _bounds_args(c, n), n)


def test_bounds_of_extreme_keys():
    n = [16 * 6]
    c = Cache(25, n, 2, 64, dtype="f32")
    page = lambda i: c.k_pool[c.table[0, i]]  # noqa: E731
    page(0)[5, 0, 3] = float("nan")
    page(1)[0, 1, 63] = float("inf")
    page(2)[15, 0, 0] = -float("inf")
    page(3)[:] = 0.0
    page(4)[:] *= 1e-38
    page(5)[:] *= 3e37
    a = _bounds_args(c, n)
    _check_bounds(c, a, n)
    scale = a["bound_scale"].cpu()
    assert torch.isinf(scale[c.table[0, 0], 0]) and torch.isfinite(scale[c.table[0, 0], 1])


def _select_case(seed, lens, q_len, g, H_kv, D, ps, dtype="bf16", whole=True):
    """Bounds of random keys around a centre of their page, made without a pool of keys."""
    c = Cache(seed, lens, H_kv, 1, ps, dtype, fill=False)
    rng = c.rng
    middle, reach = rng.normal(size=(2, c.P, H_kv, D))
    made = [oracle.page_bounds(np.stack([m + abs(r), m - abs(r)])) for m, r in zip(middle, reach)]
    c.codes, c.scale = np.stack([x for x, _ in made]), np.stack([x for _, x in made])
    c.q = torch.randn(len(lens), q_len, g * H_kv, D, generator=c.gen).to(DTYPES[dtype])
    return c


def _select(c, pages, first=1, last=1, single=False, ws=None, **over):
    q = c.q.to(DEV)
    B, q_len = q.shape[:2]
    if ws is None:
        ws = ts.new_workspace(ts.ts_select_pages_workspace_size(B, q_len, c.H_kv, c.table.shape[1]))
    a = dict(q=q[:, 0] if single else q, bounds=torch.from_numpy(c.codes).to(DEV),
             bound_scale=torch.from_numpy(c.scale).to(DEV), block_table=i32(c.table), seq_lens=i32(c.lens),
             page_size=c.ps, pages=pages, first=first, last=last, workspace=ws, **over)
    out = ts.ts_select_pages(**a)
    want = oracle.select_pages(c.q.float().numpy(), c.codes, c.scale, c.table, c.lens, c.ps, pages, first, last)
    got = out.cpu().numpy().reshape(want.shape)
    assert np.array_equal(got, want), f"{(got != want).sum()} of {got.size} entries"
    slots = c.table.shape[1]
    # not many short tables go through one kernel; wide ones never do
    if slots <= 2048 and c.lens.max() <= slots * c.ps and not over:
        a.update(block_table=i32(np.pad(c.table, ((0, 0), (0, 2049 - slots)), constant_values=-1)),
                 workspace=ts.new_workspace(ts.ts_select_pages_workspace_size(B, q_len, c.H_kv, 2049)))
        assert torch.equal(ts.ts_select_pages(**a), out)
    return out, ts.ts_read_device_error(ws)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g,H_kv", [(4, 8), (1, 1), (2, 4), (8, 2), (8, 8), (1, 8)])
def test_selection(dtype, D, g, H_kv):
    c = _select_case(31, [3000, 1, 16 * 12, 16 * 12 + 1, 0, 777], 1, g, H_kv, D, 16, dtype)
    assert _select(c, 12)[1] == 0


@pytest.mark.parametrize("ps", [8, 16, 32, 5, 1])
@pytest.mark.parametrize("pages,first,last", [(1, 0, 1), (2, 1, 1), (9, 3, 2), (40, 0, 3), (33, 1, 32), (700, 1, 2)])
def test_selection_sizes(ps, pages, first, last):
    c = _select_case(32, [2500, 40, 1201, 2], 2, 2, 2, 64, ps)
    assert _select(c, pages, first, last)[1] == 0


@pytest.mark.parametrize("slots,B,H_kv", [(511, 1, 1), (512, 9, 8), (513, 9, 8), (1024, 10, 4), (2047, 10, 8),
                                          (2048, 38, 2), (2048, 39, 2), (2049, 10, 8), (1023, 20, 8), (1024, 38, 8),
                                          (1025, 20, 8), (1024, 77, 4)])
def test_selection_of_table_widths(slots, B, H_kv):
    """On both sides of each rule that chooses between the kernels."""
    rng = np.random.default_rng(slots * B)
    lens = rng.integers(0, slots * 4 + 1, B)
    lens[-1] = slots * 4
    c = _select_case(42, lens, 1, 2, H_kv, 64, 4)
    assert c.table.shape[1] == slots
    assert _select(c, 19, 2, 3)[1] == 0


def test_selection_of_several_tokens_across_page_ends():
    c = _select_case(33, [18, 1000, 3, 16 * 20 + 2], 5, 4, 2, 128, 16)  # 3 < 5: rows in front of the first token
    assert _select(c, 6, 1, 2)[1] == 0


@pytest.mark.parametrize("n", [8193, 8194, 8200, 20000])
def test_selection_from_long_contexts(n):
    """More pages than the choosing CTA keeps on chip."""
    c = _select_case(34, [n * 8, 900], 1, 2, 1, 64, 8)
    assert _select(c, 50, 1, 1)[1] == 0
    assert _select(c, 4097, 2, 3)[1] == 0


def test_equal_scores_go_to_the_lowest_pages():
    c = _select_case(35, [4000, 500], 2, 2, 2, 64, 16)
    c.codes[:] = c.codes[:1]
    c.scale[:] = c.scale[:1]
    _select(c, 20, 1, 1)
    c.codes[::3] = 0  # three kinds of scores, zeros of either sign among them
    c.scale[::2] = -0.0
    _select(c, 20, 1, 1)
    c.q[:] = 0
    _select(c, 20, 2, 2)


def test_scores_that_are_not_finite():
    for value in (float("nan"), float("inf"), -float("inf")):
        c = _select_case(36, [2000, 1500], 1, 4, 2, 64, 16)
        c.q[0, 0, 1, 7] = value
        bad = c.table[1, [3, 30, 77]]
        c.codes[bad, 1], c.scale[bad, 1] = 0, np.inf
        out, err = _select(c, 10, 1, 2)
        assert err == 0 and {3, 30, 77} <= set(out[1, 0, 1].tolist()) and not {30, 77} <= set(out[1, 0, 0].tolist())
    c = _select_case(37, [3000], 1, 1, 1, 64, 16)
    c.scale[:] *= 1e30
    c.q *= 3e30  # bf16: products pass float32's range
    _select(c, 10)


def test_pages_out_of_range_and_past_the_table():
    c = _select_case(38, [3000, 640, 30], 1, 2, 2, 64, 16)
    c.table[0, 50:150:2] = -3
    c.table[1, 7] = c.P
    assert _select(c, 100, 1, 1)[1] == ts.TS_DEVERR_PAGE_RANGE
    assert _select(c, 180, 1, 1)[1] == ts.TS_DEVERR_PAGE_RANGE  # fewer good pages than places
    c = _select_case(39, [3000, 640, 30], 1, 2, 2, 64, 16)
    c.table = np.ascontiguousarray(c.table[:, :35])
    out, err = _select(c, 10)
    assert err == ts.TS_DEVERR_PAGE_RANGE and out[0, 0, 0, -1] == 34
    out, err = _select(c, 64)
    assert err == ts.TS_DEVERR_PAGE_RANGE and out[0, 0, 0, 34] == 34 and out[0, 0, 0, 35] == -1


def test_single_tokens_and_allocated_results():
    c = _select_case(40, [900, 33], 1, 4, 2, 128, 16)
    out, _ = _select(c, 7, single=True)
    assert out.shape == (2, 2, 7)
    a = dict(q=c.q[:, 0].to(DEV), bounds=torch.from_numpy(c.codes).to(DEV),
             bound_scale=torch.from_numpy(c.scale).to(DEV), block_table=i32(c.table), seq_lens=i32(c.lens),
             page_size=16, pages=7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x = ts.ts_select_pages(**a, stream=side)
    side.synchronize()
    assert torch.equal(x, out)


def test_captured_selection_with_other_lengths():
    c = _select_case(41, [3000, 100, 2000], 1, 4, 2, 128, 16)
    a = dict(q=c.q.to(DEV), bounds=torch.from_numpy(c.codes).to(DEV), bound_scale=torch.from_numpy(c.scale).to(DEV),
             block_table=i32(c.table), seq_lens=i32(c.lens), page_size=16, pages=9, first=1, last=2,
             page_idx=torch.zeros(3, 1, 2, 9, dtype=torch.int32, device=DEV),
             workspace=ts.new_workspace(ts.ts_select_pages_workspace_size(3, 1, 2, c.table.shape[1])))
    ts.ts_select_pages(**a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ts.ts_select_pages(**a)
    for lens in ([2999, 90, 17], [1, 0, 145], [1500, 100, 2000]):
        a["seq_lens"].copy_(i32(lens))
        graph.replay()
        want = oracle.select_pages(c.q.float().numpy(), c.codes, c.scale, c.table, np.array(lens), 16, 9, 1, 2)
        assert np.array_equal(a["page_idx"].cpu().numpy(), want)
