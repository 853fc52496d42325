"""ts_paged_decode_sparse_attn by each of its ways, in every type, head dimension and number
of queries a head: lists whole in a CTA, cut over warps and joined by small CTAs, cut and
joined by large ones. The launched kernels are asserted, so that a rule that moves takes
these cases along.

The rules: whole up to two items (a query row and kv head) a multiprocessor, if a list's K and
V are 512 KB at most, or 1 MB where the items fill three quarters of them; joined by
small CTAs from a quarter as many items as warps (eight a multiprocessor)."""

import os

import numpy as np
import pytest
import torch

import paged_kv_cache_46_gb300 as ts
from test_gpu_sparse_decode import _case, _check, _run
from traced import kernels_of

pytestmark = pytest.mark.gpu

BYTES = {"bf16": 2, "f32": 4}
FIRST = {"bf16": "sparse_mma_kernel", "f32": "sparse_f32_kernel"}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _both(c, q, idx, names, ctas=None):
    (out, lse, err), launched = kernels_of(lambda: _run(c, q, idx, ctas))
    assert err == 0 and launched == names
    _check(c, q, idx, out, lse)
    again, lse_again, _ = _run(c, q, idx, ctas)  # without the events of a trace between the launches
    assert torch.equal(again, out) and torch.equal(lse_again, lse)


def _pages_above(kilobytes, ps, D, dtype):
    """The shortest lists whose K and V are more than that."""
    return (kilobytes << 10) // (2 * ps * D * BYTES[dtype]) + 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("H_kv", [1, 2])
def test_few_items_of_long_lists(dtype, D, g, H_kv):
    """Cut over many warps, joined by CTAs of 512 threads."""
    ps = 32
    pages = _pages_above(512, ps, D, dtype)
    lens = [pages * ps + 700, 40, 0, 5 * ps + 3, pages * ps // 2 + 1]
    c, q, idx = _case(71, lens, 1, g, H_kv, D, pages, ps, dtype, order="any")
    _both(c, q, idx, [FIRST[dtype], "sparse_merge_kernel"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("ps,pages", [(8, 9), (16, 2), (32, 5)])
def test_many_items(dtype, D, g, ps, pages):
    """Cut, joined by small CTAs; lists of one page to `pages`."""
    B = 2 * _sms() // 8 + 1
    lens = np.random.default_rng(g).integers(0, 12 * ps, B)
    c, q, idx = _case(72, lens, 1, g, 8, D, pages, ps, dtype, order="any")
    _both(c, q, idx, [FIRST[dtype], "sparse_merge_kernel"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pages", [1, 2, 3, 5, 17, 64])
@pytest.mark.parametrize("ctas,B", [(3, 7), (40, 11), (151, 38)])
def test_short_lists_cut_anywhere(dtype, pages, ctas, B):
    lens = np.random.default_rng(pages).integers(0, 900, B)
    lens[-1] = 70 * 8
    c, q, idx = _case(73, lens, 1, 4, 8, 64, pages, 8, dtype, order="any")
    assert 8 * B > 2 * ctas
    _both(c, q, idx, [FIRST[dtype], "sparse_merge_kernel"], ctas)


def test_short_lists_cut_over_a_thousand_ctas():
    B = 251
    lens = np.random.default_rng(3).integers(0, 400, B)
    c, q, idx = _case(74, lens, 1, 2, 8, 64, 40, 8, order="any")
    _both(c, q, idx, ["sparse_mma_kernel", "sparse_merge_kernel"], 1000)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 8])
def test_items_whole_at_both_rules(dtype, D, g):
    ps = 32
    pages = _pages_above(512, ps, D, dtype)
    c, q, idx = _case(75, [pages * ps, 1, 0, 500], 1, g, 2, D, pages - 1, ps, dtype, order="any")
    _both(c, q, idx, [FIRST[dtype]])
    B = -(-3 * _sms() // 32)  # three quarters of the multiprocessors at 8 kv heads
    lens = np.random.default_rng(g).integers(0, 8 * ps, B)
    lens[1] = pages * ps + 9
    c, q, idx = _case(76, lens, 1, g, 8, D, pages, ps, dtype)
    _both(c, q, idx, [FIRST[dtype]])
    c, q, idx = _case(77, lens, 1, g, 8, D, _pages_above(1024, ps, D, dtype), ps, dtype)
    _both(c, q, idx, [FIRST[dtype], "sparse_merge_kernel"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_several_tokens_cut(dtype):
    lens = np.concatenate([[3, 0, 17 * 8 + 2], np.random.default_rng(5).integers(0, 300, 10)])
    c, q, idx = _case(78, lens, 5, 4, 8, 64, 7, 8, dtype, order="any")
    assert len(lens) * 5 * 8 > 2 * _sms()
    _both(c, q, idx, [FIRST[dtype], "sparse_merge_kernel"])


def test_captured_cut_lists_with_other_lengths():
    """Joined by large CTAs, in a graph."""
    assert "TS_PAGED_DECODE_CTAS" not in os.environ
    pages = _pages_above(512, 32, 64, "bf16")
    c, q, idx = _case(79, [2500, 64, 900], 1, 4, 2, 64, pages, 32)
    from long_context_cases import DEV, i32
    from test_gpu_sparse_decode import _lists
    ws = ts.new_workspace(ts.ts_paged_decode_sparse_workspace_size(3, 1, 8, 2, 64, 32, pages))
    a = dict(q=q[:, 0].to(DEV), **c.device(), page_idx=i32(idx[:, 0]), scale=0.125, workspace=ws)
    a["out"], a["lse"] = torch.zeros_like(a["q"]), torch.zeros(3, 8, device=DEV)
    _, launched = kernels_of(lambda: ts.ts_paged_decode_sparse_attn(**a))
    assert launched == ["sparse_mma_kernel", "sparse_merge_kernel"]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ts.ts_paged_decode_sparse_attn(**a)
    for lens in ([2499, 17, 900], [40, 0, 1], [2500, 64, 900]):
        c.lens = np.array(lens)
        idx = _lists(c, 1, pages, "any")
        a["seq_lens"].copy_(i32(lens))
        a["page_idx"].copy_(i32(idx[:, 0]))
        graph.replay()
        torch.cuda.synchronize()
        _check(c, q, idx, a["out"].view(q.shape), a["lse"].view(3, 1, 8))
