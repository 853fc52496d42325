"""ts_kv_compact on both sides of the sizes up to which one CTA plans the moves (32,768
entries of the table and 262,144 pages), byte for byte. Tables are mostly past their
lengths where they are wide, as those for the longest context that is allowed."""

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_46_gb300 as ts
from long_context_cases import DEV, i32
from test_gpu_kv_pages import _buffers, _equal
from traced import kernels_of

pytestmark = pytest.mark.gpu

ONE = ["page_plan_kernel", "page_move_kernel"]
THREE = ["page_clear_kernel", "page_mark_kernel", "page_scan_kernel", "page_move_kernel"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _expected(host, table, lens, ps):
    """As oracle.kv_compact (see test_expectation), at once for tens of thousands of pages."""
    P = host[0].shape[0]
    live = (np.arange(table.shape[1]) * ps < np.asarray(lens)[:, None]) & (table >= 0) & (table < P)
    held = np.zeros(P, dtype=bool)
    held[table[live]] = True
    U, page = int(held.sum()), np.arange(P)
    source, target = page[held & (page >= U)], page[~held & (page < U)]
    page_map = np.where(held, page, -1).astype(np.int32)
    page_map[source] = target
    out = [x.copy() for x in host]
    for x in out:
        x[target] = x[source]
    new = table.copy()
    new[live] = page_map[table[live]]
    return out, new, page_map, U


def _case(seed, B, slots, P, pages):
    """Sequences that hold about `pages` pages together, some of them shared; ps = 4."""
    rng = np.random.default_rng(seed)
    table = rng.integers(-5, P + 5, (B, slots)).astype(np.int32)  # slots that nobody holds name anything
    held = rng.permutation(P)[:pages]
    lens = np.zeros(B, dtype=np.int64)
    share = rng.multinomial(pages, np.full(B, 1 / B))
    at = 0
    for b, n in enumerate(np.minimum(share, slots)):
        table[b, :n] = held[at:at + n]
        lens[b] = max(0, 4 * n - rng.integers(0, 4))
        at += int(n)
    if B > 1 and lens[0] >= 8 and lens[-1] >= 8:
        table[-1, :2] = table[0, :2]
    if B > 2 and lens[1] >= 8:
        table[1, 1] = P      # held by name, out of range
        lens[2] = -3
    return table, lens


def _run(table, lens, P, sizes, in_place, names):
    host, dev = _buffers(P, sizes)
    plan, bt = ts.kv_buffers(dev), i32(table)
    ws = ts.new_workspace(ts.ts_kv_compact_workspace_size(P))
    want = _expected(host, table, lens, 4)

    def check(got):
        assert _equal(dev, want[0])
        assert np.array_equal(got[0].cpu().numpy(), want[1])
        assert np.array_equal(got[1].cpu().numpy(), want[2]) and int(got[2]) == want[3]

    def call():
        return ts.ts_kv_compact(plan, bt, i32(lens), 4, table_out=bt if in_place else None, workspace=ws)

    got, launched = kernels_of(call)
    assert launched == names
    check(got)
    for _ in range(3):  # without the events of a trace between the launches, on a workspace that was used
        for x, y in zip(dev, host):
            x.copy_(torch.from_numpy(y))
        bt.copy_(i32(table))
        check(call())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,slots,P,names", [
    (8, 4096, 5000, ONE), (3, 10923, 5000, THREE),          # 32,768 and 32,769 entries
    (7, 400, 262_144, ONE), (7, 400, 262_145, THREE),
    (64, 2048, 3000, THREE), (1, 40_000, 262_177, THREE), (40_000, 1, 35_000, THREE)])
def test_both_sides_of_each_limit(B, slots, P, names, in_place):
    table, lens = _case(B + slots, B, slots, P, min(2500, P // 2))
    _run(table, lens, P, [16, 5], in_place, names)


@pytest.mark.parametrize("share", [0.0, 0.1, 0.5, 0.95, 1.0])
def test_a_serving_table(share):
    """64 rows of 2,048 slots, up to all of 90,001 pages held."""
    P = 90_001
    table, lens = _case(7, 64, 2048, P, int(share * P))
    _run(table, lens, P, [32, 1], share == 0.5, THREE)


@pytest.mark.parametrize("B,P,names", [(0, 262_144, ONE), (2, 262_145, THREE),
                                       (0, 262_145, ["page_clear_kernel", "page_scan_kernel", "page_move_kernel"])])
def test_nothing_held(B, P, names):
    host, dev = _buffers(P, [4])
    table = torch.zeros(B, 4, dtype=torch.int32, device=DEV)
    (_, page_map, used), launched = kernels_of(
        lambda: ts.ts_kv_compact(dev, table, torch.zeros(B, dtype=torch.int32, device=DEV), 16))
    assert launched == names
    assert (page_map == -1).all() and int(used) == 0 and _equal(dev, host)


def test_captured_with_other_lengths():
    P, ps = 20_000, 4
    table, lens = _case(9, 40, 1000, P, 9000)
    host, dev = _buffers(P, [64, 6])
    plan, bt, on = ts.kv_buffers(dev), i32(table), i32(lens)
    out = dict(table_out=torch.zeros_like(bt), page_map=torch.zeros(P, dtype=torch.int32, device=DEV),
               used=torch.zeros(1, dtype=torch.int32, device=DEV),
               workspace=ts.new_workspace(ts.ts_kv_compact_workspace_size(P)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _, launched = kernels_of(lambda: ts.ts_kv_compact(plan, bt, on, ps, stream=side, **out))
    assert launched == THREE
    side.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ts.ts_kv_compact(plan, bt, on, ps, **out)
    for new in (lens, lens // 2, np.where(np.arange(40) % 3 == 0, lens, 0), lens * 0):
        for x, y in zip(dev, host):
            x.copy_(torch.from_numpy(y))
        on.copy_(i32(new))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, new_table, page_map, used = _expected(host, table, new, ps)
        assert _equal(dev, want) and np.array_equal(out["table_out"].cpu().numpy(), new_table)
        assert np.array_equal(out["page_map"].cpu().numpy(), page_map) and int(out["used"]) == used


def test_expectation():
    table, lens = _case(11, 6, 50, 300, 100)
    host = [np.random.default_rng(0).integers(0, 256, (300, 8), dtype=np.uint8)]
    a, b = _expected(host, table, lens, 4), oracle.kv_compact(host, table, lens, 4)
    assert all(np.array_equal(x, y) for x, y in zip(a[0], b[0]))
    assert np.array_equal(a[1], b[1]) and np.array_equal(a[2], b[2]) and a[3] == b[3]
