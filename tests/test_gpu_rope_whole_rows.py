"""ts_kv_append_chunk_rope where a warp takes whole rows of many steps, queries, keys and
values in batches of their own: as many rows as leave each warp one row (half of 32 a
multiprocessor and more), more than twelve steps of heads a row."""

import numpy as np
import pytest
import torch

import paged_kv_cache_46_gb300 as ts
from long_context_cases import DEV, i32
from test_gpu_rope_append import Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _whole_rows():
    return 16 * torch.cuda.get_device_properties(0).multi_processor_count + 1


def _steps(H_q, H_kv, D):
    heads = 256 // D
    return -(-H_q // heads) + 2 * -(-H_kv // heads)


# heads that end a section's batches at every remainder of four steps; more kv heads than query heads
@pytest.mark.parametrize("D,H_q,H_kv", [(128, 32, 8), (64, 71, 3), (128, 33, 5), (64, 40, 24), (128, 3, 11), (64, 1, 30)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot,norm,interleaved,fused", [("all", "qk", False, True), ("half", "q", True, False),
                                                       ("few", "", False, False), ("none", "k", False, True)])
def test_whole_rows(D, H_q, H_kv, dtype, rot, norm, interleaved, fused):
    assert _steps(H_q, H_kv, D) > 12
    rng = np.random.default_rng(H_q)
    last = [5, 0, 33, 1]  # sequences that are taken in a call of their own, too
    n = np.concatenate([[1, 0, 40], rng.integers(0, 200, _whole_rows() // 80), last])
    n[3] += max(0, _whole_rows() - n.sum())
    rot = {"all": D, "half": D // 2, "few": 8, "none": 0}[rot]
    case = Rows(21, n, rng.integers(0, 70, len(n)), H_q, H_kv, D, 16, dtype, rot, norm, interleaved, fused, pad=3)
    a = case.args()
    T = case.q.shape[0]
    out = torch.full((T, H_q, D), 7.0, dtype=case.cache.dtype, device=DEV)
    before = out.clone()
    k_pool, v_pool = a["k_pool"].clone(), a["v_pool"].clone()
    ts.ts_kv_append_chunk_rope(**a, q_out=out)
    case.check(out, a["k_pool"], a["v_pool"], before)
    assert torch.equal(out[-3:], before[-3:])

    few = int(np.sum(last))
    rows = slice(T - 3 - few, T - 3)
    small = dict(a, k_pool=k_pool, v_pool=v_pool, block_table=a["block_table"][-4:].contiguous(),
                 seq_lens=a["seq_lens"][-4:].contiguous(), q_indptr=i32(np.concatenate([[0], np.cumsum(last)])),
                 **{name: a[name][rows] for name in ("q", "k_new", "v_new")})
    alone = ts.ts_kv_append_chunk_rope(**small)
    assert torch.equal(alone, out[rows])
    for b, L in enumerate(case.cache.lens[-4:]):
        pages = case.cache.table[len(n) - 4 + b, :(int(L) + 15) // 16].astype(np.int64)
        for pool, whole in ((k_pool, a["k_pool"]), (v_pool, a["v_pool"])):
            assert torch.equal(pool[pages].nan_to_num(9.0), whole[pages].nan_to_num(9.0))

    in_place = case.args()  # the queries' own rows, a part of wider ones where they are fused
    beside = [in_place[name].clone() for name in ("k_new", "v_new")]
    ts.ts_kv_append_chunk_rope(**in_place, q_out=in_place["q"])
    assert torch.equal(in_place["q"][:-3], out[:-3])
    assert torch.equal(in_place["k_new"], beside[0]) and torch.equal(in_place["v_new"], beside[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_whole_rows_of_places_that_take_nothing(dtype):
    T = _whole_rows() + 40
    case = Rows(22, [T - 20, 20], [0, 7], 34, 6, 128, 16, dtype)
    c = case.cache
    c.lens[1] = 12                       # its first eight rows lie in front of the first token
    c.table[0, 3::2] = c.P               # every other page is out of range
    c.table = np.ascontiguousarray(c.table[:, :c.table.shape[1] - 5])  # the last pages have no slot
    a = case.args()
    out = torch.full((T, 34, 128), 7.0, dtype=c.dtype, device=DEV)
    before = out.clone()
    ts.ts_kv_append_chunk_rope(**a, q_out=out)
    case.check(out, a["k_pool"], a["v_pool"], before)
    assert torch.equal(out[T - 20:T - 12], before[T - 20:T - 12])
