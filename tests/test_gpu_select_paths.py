"""ts_select_pages by a CTA of 256 threads an item (more items than multiprocessors, two each at
most, tables of up to 1,024 slots) in every type, head dimension and number of queries a head,
with the launched kernels asserted; and ts_kv_page_bounds where more sequences begin inside a
warp's rows than it looks at in one step. Both are exact."""

import numpy as np
import pytest
import torch

from long_context_cases import Cache
from test_gpu_select_pages import _bounds_args, _check_bounds, _select, _select_case
from traced import kernels_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("H_kv,q_len", [(8, 1), (2, 3)])
def test_items_of_256_threads(dtype, D, g, H_kv, q_len):
    B = _sms() // (H_kv * q_len) + 1
    slots = 1024 if q_len == 1 else 300
    rng = np.random.default_rng(g)
    lens = rng.integers(0, slots // 3 * 4, B)
    lens[3:6] = slots * 4, 19 * 4, 19 * 4 + 1
    c = _select_case(43, lens, q_len, g, H_kv, D, 4, dtype)
    assert c.table.shape[1] == slots and _sms() < B * q_len * H_kv <= 2 * _sms()
    # the same once more in two launches, behind a wider table
    (_, err), launched = kernels_of(lambda: _select(c, 19, 2, 3))
    assert err == 0 and launched == ["page_select_kernel", "page_score_kernel", "page_pick_kernel"]


@pytest.mark.parametrize("pages", [5, 6, 400])
def test_items_of_256_threads_with_ties(pages):
    B = _sms() // 8 + 1
    c = _select_case(44, np.full(B, 700 * 4 - 1), 1, 4, 8, 128, 4)
    c.codes[:] = c.codes[:1]  # five kinds of scores
    c.scale[:] = 0.01
    for i in range(1, 5):
        c.scale[i::5] = 0.01 * i
    (_, err), launched = kernels_of(lambda: _select(c, pages, 2, 3))
    assert err == 0 and launched[0] == "page_select_kernel"


@pytest.mark.parametrize("H_kv,D,dtype", [(2, 64, "bf16"), (3, 128, "f32")])
def test_bounds_of_many_short_and_empty_sequences(H_kv, D, dtype):
    n = [0] * 40
    for run in (31, 32, 33, 40, 100):
        for start in (0, 7, 15):  # rows of a warp's sixteen in front of the run
            for middle in ([0] * run, [1] * run, [0, 1, 0] * run):
                n.append(16 + (start - sum(n)) % 16)
                n += middle
    n += [2100, 1] + [0] * 100
    n = np.array(n)
    assert n.sum() > 2048
    rng = np.random.default_rng(27)
    ctx = rng.integers(0, 40, len(n))
    ctx[rng.random(len(n)) < 0.3] = 0
    c = Cache(27, n + ctx, H_kv, D, 16, dtype)
    _check_bounds(c, _bounds_args(c, n), n)
