"""GPU parity of ts_kv_fork and ts_kv_compact: whole pages and whole numbers, so every
byte equals the oracle's."""

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_46_gb300 as ts
from long_context_cases import DEV, Cache, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _buffers(P, sizes, seed=0):
    """Random bytes [P, size]; a size that is a tuple (size, offset) starts `offset` bytes off an aligned address."""
    g = torch.Generator().manual_seed(seed)
    host, dev = [], []
    for size in sizes:
        size, off = size if isinstance(size, tuple) else (size, 0)
        x = torch.randint(0, 256, (P, size), generator=g, dtype=torch.uint8)
        room = torch.zeros(P * size + 16, dtype=torch.uint8, device=DEV)
        y = room[off:off + P * size].view(P, size)
        y.copy_(x)
        host.append(x.numpy())
        dev.append(y)
    return host, dev


def _equal(dev, want):
    return all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(dev, want))


SIZES = [[4096, 4096, 2048, 32], [16], [1], [4], [6, 30, 20], [16384, 16400, 65536 + 16], [40000, (4096, 4), (4096, 1)]]


def _fork_case(seed, lens, children, ps=16):
    c = Cache(seed, list(lens) + [0] * children, 1, 1, ps, spare=children + 3, slots=2, fill=False)
    c.table[len(lens):] = -9
    return c


def _fork(c, sizes, parents, children, fresh, plan=True, **kw):
    host, dev = _buffers(c.P, sizes)
    bt, lens = i32(c.table), i32(c.lens)
    buffers = ts.kv_buffers(dev) if plan else dev
    ts.ts_kv_fork(buffers, bt, lens, i32(parents), i32(children), i32(fresh), c.ps, **kw)
    want, table, lengths = oracle.kv_fork(host, c.table, c.lens, parents, children, fresh, c.ps)
    torch.cuda.synchronize()
    assert _equal(dev, want)
    assert np.array_equal(bt.cpu().numpy(), table) and np.array_equal(lens.cpu().numpy(), lengths)


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("ps", [16, 1, 7])
def test_forks(sizes, ps):
    c = _fork_case(71, [61, 16, 0, 1000, 5], 9, ps)
    parents, children = [0, 0, 1, 2, 3, 3, 4, 0], [7, 5, 6, 13, 8, 9, 10, 12]
    _fork(c, sizes, parents, children, c.free[:8])


def test_more_buffers_than_a_launch_takes():
    c = _fork_case(72, [61, 100], 4)
    _fork(c, [64, 1, 160] * 50, [0, 0, 1], [2, 3, 5], c.free[:3], plan=False)


def test_entries_that_are_skipped():
    c = _fork_case(73, [61, 32, 40, 20], 6)
    c.table[2, 2] = c.P       # the page to copy
    c.lens[3] = 10000         # longer than the table's row
    f = c.free
    parents = [0, 0, 7, -1, 0, 2, 3, 1, 1, 0]
    children = [0, 99, 4, 5, -2, 6, 7, 8, 9, 5]
    fresh = [f[0], f[1], f[2], f[3], f[4], f[0], f[1], -1, c.P + 7, c.P]
    # kept: sequence 1 holds whole pages and needs no fresh one (8, 9); the length 0 of row 7 is forked to 4
    _fork(c, [4096, 20], parents, children, fresh)


def test_forks_of_negative_lengths_and_of_nothing():
    c = _fork_case(74, [30, 30], 3)
    c.lens[1] = -4
    _fork(c, [256], [1, 0], [2, 3], c.free[:2])
    _fork(c, [256], [], [], [])


def test_captured_forks():
    c = _fork_case(75, [61, 32, 40], 4)
    host, dev = _buffers(c.P, [4096, 32])
    plan = ts.kv_buffers(dev)
    bt, lens, parents, children, fresh = (i32(x) for x in (c.table, c.lens, [0, 2], [3, 4], c.free[:2]))
    scratch = bt.clone(), lens.clone()
    graph = torch.cuda.CUDAGraph()
    ts.ts_kv_fork(plan, *scratch, parents, children, fresh, 16)
    with torch.cuda.graph(graph):
        ts.ts_kv_fork(plan, bt, lens, parents, children, fresh, 16)
    for x, y in zip(dev, host):
        x.copy_(torch.from_numpy(y))
    parents.copy_(i32([2, 0]))
    children.copy_(i32([6, 5]))
    graph.replay()
    want, table, lengths = oracle.kv_fork(host, c.table, c.lens, [2, 0], [6, 5], c.free[:2], 16)
    assert _equal(dev, want)
    assert np.array_equal(bt.cpu().numpy(), table) and np.array_equal(lens.cpu().numpy(), lengths)


def _compact(table, lens, P, sizes, ps=16, in_place=False, plan=True, seed=0):
    host, dev = _buffers(P, sizes, seed)
    bt = i32(table)
    got = ts.ts_kv_compact(ts.kv_buffers(dev) if plan else dev, bt, i32(lens), ps, table_out=bt if in_place else None)
    want, want_table, page_map, used = oracle.kv_compact(host, np.asarray(table, dtype=np.int32), lens, ps)
    assert _equal(dev, want)
    assert np.array_equal(got[0].cpu().numpy(), want_table)
    assert np.array_equal(got[1].cpu().numpy(), page_map) and int(got[2]) == used
    assert in_place or np.array_equal(bt.cpu().numpy(), table)
    return used


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_compaction(sizes, in_place):
    c = Cache(81, [61, 16, 0, 1000, 5, 300, 77], 1, 1, spare=30, slots=1, fill=False)
    keep = [1, 2, 3, 6]
    _compact(c.table[keep], c.lens[keep], c.P, sizes, in_place=in_place)


@pytest.mark.parametrize("P", [1, 31, 32, 33, 64, 95, 1000, 1024, 5000])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 0.97, 1.0])
def test_pools_of_any_size_and_filling(P, share):
    rng = np.random.default_rng(P)
    held = rng.permutation(P)[:int(round(share * P))]
    lens = np.array([0, len(held)])
    table = np.full((2, max(1, len(held))), P // 2, dtype=np.int32)
    table[1, :len(held)] = held
    assert _compact(table, lens, P, [32, 5], ps=1) == len(held)


def test_large_pools_with_pages_at_the_end():
    P = 150_001
    rng = np.random.default_rng(82)
    held = np.unique(np.concatenate([rng.integers(0, P, 3000), np.arange(P - 100, P), np.arange(40)]))
    rng.shuffle(held)
    table = held[:len(held) // 7 * 7].reshape(7, -1)
    _compact(table, np.full(7, table.shape[1] * 4 - 3), P, [48], ps=4)


def test_shared_pages_and_ids_out_of_range():
    table = np.array([[9, 8, 7, -4], [9, 8, 5, 1], [12, 11, 9, 30], [3, 2 ** 31 - 1, 0, 0]], dtype=np.int32)
    assert _compact(table, [48, 64, 17, 20], 12, [64, 4], ps=16) == 7  # 9 8 7 5 1 11 3
    _compact(table, [48, 64, -5, 0], 12, [64, 4], ps=16, in_place=True)


def test_more_buffers_than_a_launch_takes_compacted():
    c = Cache(83, [61, 16, 200, 300], 1, 1, spare=5, fill=False)
    _compact(c.table[[0, 3]], c.lens[[0, 3]], c.P, [64, 2, 48] * 60, plan=False)


def test_an_empty_batch_frees_every_page():
    host, dev = _buffers(20, [64])
    empty = torch.zeros(0, 4, dtype=torch.int32, device=DEV)
    table, page_map, used = ts.ts_kv_compact(dev, empty, empty[:, 0].contiguous(), 16)
    assert table.shape == (0, 4) and (page_map == -1).all() and int(used) == 0 and _equal(dev, host)


def test_captured_compaction_with_other_lengths_and_a_stream_of_its_own():
    c = Cache(84, [61, 16, 200, 300], 1, 1, spare=5, fill=False)
    host, dev = _buffers(c.P, [4096, 32])
    plan, bt, lens = ts.kv_buffers(dev), i32(c.table), i32(c.lens)
    out = dict(table_out=torch.zeros_like(bt), page_map=torch.zeros(c.P, dtype=torch.int32, device=DEV),
               used=torch.zeros(1, dtype=torch.int32, device=DEV),
               workspace=ts.new_workspace(ts.ts_kv_compact_workspace_size(c.P)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ts.ts_kv_compact(plan, bt, lens, 16, stream=side, **out)
    side.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ts.ts_kv_compact(plan, bt, lens, 16, **out)
    for new in ([61, 0, 0, 300], [0, 16, 200, 0], [0, 0, 0, 0]):
        for x, y in zip(dev, host):
            x.copy_(torch.from_numpy(y))
        lens.copy_(i32(new))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, table, page_map, used = oracle.kv_compact(host, c.table, new, 16)
        assert _equal(dev, want) and np.array_equal(out["table_out"].cpu().numpy(), table)
        assert np.array_equal(out["page_map"].cpu().numpy(), page_map) and int(out["used"]) == used
