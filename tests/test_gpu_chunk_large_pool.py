"""Prompt-chunk operators on pools whose pages lie past 2^31 elements and 2^32
bytes: the same bits as on small pools."""

import numpy as np
import pytest
import torch

import paged_kv_cache_46_gb300 as ts
from chunk_cases import DEV, ChunkCase

pytestmark = pytest.mark.gpu

PS, H_KV, D = 32, 8, 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _case(dtype):
    return ChunkCase(1, [70, 3, 40], [200, 33, 0], 32, H_KV, D, ps=PS, dtype=dtype, spare=0)


def _pages(es):
    """Pages of a pool of more than 2^31 elements and 2^32 bytes (es bytes each)."""
    return max((1 << 31), -(-(1 << 32) // es)) // (PS * H_KV * D) + 100


def _high(small, P):
    """The small pool's pages at the end of one of P pages."""
    pool = torch.empty((P,) + tuple(small.shape[1:]), dtype=small.dtype, device=DEV)
    pool[P - small.shape[0]:] = small
    return pool


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_and_appends_at_the_end_of_a_large_pool(dtype):
    case = _case(dtype)
    a = case.device()
    n_small = a["k_pool"].shape[0]
    P = _pages(a["k_pool"].element_size())
    high = {k: _high(a[k], P) for k in ("k_pool", "v_pool")}
    bt = a["block_table"] + (P - n_small)
    want = ts.ts_paged_prefill_attn(**a, return_lse=True)
    got = ts.ts_paged_prefill_attn(**dict(a, **high, block_table=bt), return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    last = a["q"][:3].contiguous()
    one = lambda kp, vp, b: ts.ts_paged_decode_sink_attn(last, kp, vp, b, a["seq_lens"], case.scale, 20, 3)  # noqa: E731
    assert torch.equal(one(high["k_pool"], high["v_pool"], bt), one(a["k_pool"], a["v_pool"], a["block_table"]))
    g = torch.Generator().manual_seed(2)
    k_new, v_new = (torch.randn(case.T, H_KV, D, generator=g).to(case.q.dtype).to(DEV) for _ in range(2))
    ts.ts_kv_append_chunk(k_new, v_new, a["k_pool"], a["v_pool"], a["block_table"], a["seq_lens"], a["q_indptr"])
    ts.ts_kv_append_chunk(k_new, v_new, high["k_pool"], high["v_pool"], bt, a["seq_lens"], a["q_indptr"])
    for name in ("k_pool", "v_pool"):
        bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
        assert torch.equal(bits(high[name][P - n_small:]), bits(a[name]))


def test_fp8_append_and_read_at_the_end_of_a_large_pool():
    case = _case("bf16")
    a = case.device()
    n_small, P = a["k_pool"].shape[0], _pages(1)
    g = torch.Generator().manual_seed(3)
    k_new, v_new = (torch.randn(case.T, H_KV, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    small = [torch.zeros(n_small, PS, H_KV, D, dtype=torch.uint8, device=DEV) for _ in range(2)] + \
            [torch.zeros(n_small, PS, H_KV, device=DEV) for _ in range(2)]
    high = [_high(x, P) for x in small]
    bt = a["block_table"] + (P - n_small)
    ts.ts_kv_append_chunk_fp8(k_new, v_new, *small, a["block_table"], a["seq_lens"], a["q_indptr"])
    ts.ts_kv_append_chunk_fp8(k_new, v_new, *high, bt, a["seq_lens"], a["q_indptr"])
    for x, y in zip(high, small):
        assert torch.equal(x[P - n_small:], y)
    at = torch.tensor(np.concatenate([[0], np.cumsum(case.L)]), dtype=torch.int32, device=DEV)
    outs = []
    for pools, table in ((small, a["block_table"]), (high, bt)):
        ko, vo = (torch.zeros(int(case.L.sum()), H_KV, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        ts.ts_kv_read_fp8(*pools, table, a["seq_lens"], at, ko, vo)
        outs.append((ko, vo))
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert outs[0][0].abs().sum() > 0
