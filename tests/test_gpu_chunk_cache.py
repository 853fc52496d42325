"""GPU parity of the chunk appends (plain and quantizing, bit-exact), of the
read-back of a quantized cache, and a run of all of them as a server makes it."""

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


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _batch(seed, n, ctx, H_kv, D, ps, dtype, pad=0, fused=False):
    """(k_new, v_new, block table, seq_lens, indptr, pages)."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    n, L = np.asarray(n), np.asarray(n) + np.asarray(ctx)
    need = (L + ps - 1) // ps
    P = int(need.sum()) + 2
    order = rng.permutation(P)
    bt = np.full((len(n), max(1, int(need.max()))), order[-1], dtype=np.int32)
    at = 0
    for b in range(len(n)):
        bt[b, :need[b]] = order[at:at + need[b]]
        at += int(need[b])
    T = int(n.sum()) + pad
    x = torch.randn(T, 2 * H_kv + (3 if fused else 0), D, generator=g)
    x[:, :, ::9] *= 30
    x = x.to(dtype)
    k, v = x[:, :H_kv], x[:, H_kv:2 * H_kv]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    return k, v, bt, L, np.concatenate([[0], np.cumsum(n)]), P


SHAPES = [
    ([1], [0], 1, 64, 16), ([33], [99], 8, 128, 16), ([5, 0, 17], [3, 9, 0], 2, 64, 8),
    ([130, 1, 64], [0, 31, 100], 4, 128, 32), ([7, 8, 9], [1, 2, 3], 3, 64, 16), ([0, 0, 3, 0], [5, 0, 1, 2], 1, 128, 8),
]


def _bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


@pytest.mark.parametrize("n,ctx,H_kv,D,ps", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fused", [False, True])
def test_append_is_exact_and_touches_nothing_else(n, ctx, H_kv, D, ps, dtype, fused):
    k, v, bt, L, ptr, P = _batch(sum(n) + D, n, ctx, H_kv, D, ps, dtype, pad=5, fused=fused)
    pools = [torch.full((P, ps, H_kv, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2)]
    before = [_bits(p).cpu().numpy() for p in pools]
    ts.ts_kv_append_chunk(k.to(DEV), v.to(DEV), *pools, _i32(bt), _i32(L), _i32(ptr))
    torch.cuda.synchronize()
    ref = oracle.kv_append_chunk(*before, _bits(k).numpy(), _bits(v).numpy(), bt, L, ptr)
    for got, want in zip(pools, ref):
        assert np.array_equal(_bits(got).cpu().numpy(), want)


@pytest.mark.parametrize("n,ctx,H_kv,D,ps", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fused", [False, True])
def test_fp8_append_is_exact_and_touches_nothing_else(n, ctx, H_kv, D, ps, dtype, fused):
    k, v, bt, L, ptr, P = _batch(sum(n) + D, n, ctx, H_kv, D, ps, dtype, pad=5, fused=fused)
    if len(k):
        k[0, 0] = 0.0  # a group of zeros takes the scale's floor
        v[-1, 0] = 1e-30
    pools = [torch.randint(0, 255, (P, ps, H_kv, D), dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.rand(P, ps, H_kv, device=DEV) for _ in range(2)]
    before = [t.cpu().numpy() for t in pools + scales]
    ts.ts_kv_append_chunk_fp8(k.to(DEV), v.to(DEV), *pools, *scales, _i32(bt), _i32(L), _i32(ptr))
    torch.cuda.synchronize()
    ref = oracle.kv_append_chunk_fp8(*before, k.float().numpy(), v.float().numpy(), bt, L, ptr)
    for got, want in zip(pools + scales, ref):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_fp8_append_of_every_bf16_magnitude(dtype):
    """Quotients near every rounding border: all positive bf16 values within 2^-18 .. 1 of the
    group's maximum, and random float32 ones, against the single-token append bit for bit."""
    H_kv, D, ps = 2, 128, 16
    vals = torch.arange(0x3600, 0x3f80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    rows = []
    for top in (1.0, 1.5, 1.0078125, 1.9921875, 7.0, 448.0, 0.33):
        x = vals * top
        x = x[: len(x) // 127 * 127].view(-1, 127)
        rows.append(torch.cat([x, torch.full((len(x), 1), top)], 1))
    x = torch.cat(rows)
    x = torch.cat([x, torch.randn(301, D, generator=torch.Generator().manual_seed(1)).exp()])
    x = x[: len(x) // 2 * 2].view(-1, 2, D).to(dtype).to(DEV)
    T = len(x)
    P = (T + ps - 1) // ps
    bt = torch.arange(P, dtype=torch.int32, device=DEV)[None].contiguous()
    new = [torch.zeros(P, ps, H_kv, D, dtype=torch.uint8, device=DEV) for _ in range(2)]
    new += [torch.zeros(P, ps, H_kv, device=DEV) for _ in range(2)]
    old = [torch.zeros_like(t) for t in new]
    ts.ts_kv_append_chunk_fp8(x, -x, *new, bt, _i32([T]), _i32([0, T]))
    ts.ts_kv_append_fp8(x, -x, *old, bt.expand(T, -1).contiguous(), torch.arange(T, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for a, b in zip(new, old):
        assert torch.equal(a, b)
    ref = oracle.kv_append_chunk_fp8(*[t.cpu().numpy() * 0 for t in new], x.float().cpu().numpy(),
                                     -x.float().cpu().numpy(), bt.cpu().numpy(), [T], [0, T])
    for a, b in zip(new, ref):
        assert np.array_equal(a.cpu().numpy(), b)


def test_appends_skip_rows_without_a_place():
    """Negative positions, slots past the table, page ids out of range, rows outside the
    offsets, offsets out of order: skipped, nothing else written."""
    k, v, bt, L, ptr, P = _batch(4, [20, 20], [30, 30], 2, 64, 16, torch.bfloat16)
    k, v = k.to(DEV), v.to(DEV)
    bt = bt.copy()
    bt[0, 2], bt[1, 3] = -5, P
    for lens, offsets in (([50, 50], [0, 20, 40]), ([10, 0], [0, 20, 40]), ([500, 50], [3, 20, 35]),
                          ([50, 50], [0, 60, 40]), ([50, 50], [40, 20, 0]), ([50, 50], [-8, 20, 4000])):
        room = [torch.zeros(P + 4, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        room8 = [torch.zeros(P + 4, 16, 2, 64, dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.zeros(P + 4, 16, 2, device=DEV) for _ in range(2)]
        inner = lambda ts_: [t[2:-2] for t in ts_]  # noqa: E731
        ts.ts_kv_append_chunk(k, v, *inner(room), _i32(bt), _i32(lens), _i32(offsets))
        ts.ts_kv_append_chunk_fp8(k, v, *inner(room8), *inner(scales), _i32(bt), _i32(lens), _i32(offsets))
        torch.cuda.synchronize()
        for t in room + room8 + scales:
            assert not t[:2].any() and not t[-2:].any()
        if offsets == [0, 20, 40] and lens == [50, 50]:
            good = [(b, j) for b in range(2) for j in range(20) if 0 <= bt[b, (30 + j) // 16] < P]
            want = torch.zeros(P, 16, 2, 64, dtype=torch.bfloat16)
            for b, j in good:
                want[bt[b, (30 + j) // 16], (30 + j) % 16] = k[20 * b + j].cpu()
            assert torch.equal(room[0][2:-2].cpu(), want)


@pytest.mark.parametrize("n,ctx,H_kv,D,ps", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read_back_is_exact_and_touches_nothing_else(n, ctx, H_kv, D, ps, dtype):
    """Every code value, ranges longer than the sequences, rows in front and behind."""
    _, _, bt, L, _, P = _batch(sum(n), n, ctx, H_kv, D, ps, torch.bfloat16)
    g = torch.Generator().manual_seed(1)
    pools = [torch.randint(0, 256, (P, ps, H_kv, D), dtype=torch.uint8, generator=g) for _ in range(2)]
    for p in pools:
        p[(p & 0x7f) == 0x7f] = 0x7e  # no NaN codes: they compare unequal
    scales = [torch.rand(P, ps, H_kv, generator=g) for _ in range(2)]
    ptr = np.concatenate([[3], 3 + np.cumsum(L + np.arange(len(L)) % 3)])
    rows = int(ptr[-1]) + 4
    outs = [torch.full((rows, H_kv, D), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
    ts.ts_kv_read_fp8(*[t.to(DEV) for t in pools + scales], _i32(bt), _i32(L), _i32(ptr), *outs)
    torch.cuda.synchronize()
    for p, s, got in zip(pools, scales, outs):
        ref = oracle.kv_read_fp8(p.numpy(), s.numpy(), bt, L, ptr, np.full((rows, H_kv, D), 7.0))
        assert torch.equal(got.cpu(), torch.from_numpy(ref).to(dtype))


def test_read_back_keeps_rows_without_a_token():
    _, _, bt, L, _, P = _batch(5, [20, 20], [30, 30], 2, 64, 16, torch.bfloat16)
    bt = bt.copy()
    bt[0, 1], bt[1, 0] = -1, P
    pool = torch.full((P, 16, 2, 64), 0x38, dtype=torch.uint8, device=DEV)  # 1.0
    scale = torch.full((P, 16, 2), 2.0, device=DEV)
    for lens, ptr in (([50, 50], [0, 50, 100]), ([-4, 900], [0, 50, 100]), ([50, 50], [0, 70, 20]),
                      ([50, 50], [-9, 50, 5000])):
        outs = [torch.full((100 + 8, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        ts.ts_kv_read_fp8(pool, pool, scale, scale, _i32(bt), _i32(lens), _i32(ptr), *[o[4:-4] for o in outs])
        torch.cuda.synchronize()
        for o in outs:
            assert torch.all(o[:4] == 7.0) and torch.all(o[-4:] == 7.0)
            assert torch.all((o == 7.0) | (o == 2.0))
        if ptr == [0, 50, 100] and lens == [50, 50]:
            there = torch.ones(100, dtype=torch.bool)
            there[16:32] = False
            there[50:66] = False
            assert torch.equal((outs[0][4:-4, 0, 0] == 2.0).cpu(), there)


def test_empty_calls_do_nothing():
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    pool = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    ts.ts_kv_append_chunk(k, k, pool, pool.clone(), _i32([[0]]), _i32([0]), _i32([0, 0]))
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert ts.ts_paged_prefill_attn(q, pool, pool, _i32([[0]]), _i32([0]), _i32([0, 0]), 0.1).shape == (0, 4, 64)
    torch.cuda.synchronize()


@pytest.mark.parametrize("ps", [8, 16])
def test_a_server_run_over_a_quantized_cache(ps):
    """Three steps of two prompts: chunks quantized into the cache, the cache read back as
    consecutive pages, the chunks' attention over those; the same over a bf16 cache; then a
    decode step over each. Held to the oracle over the very values each cache holds."""
    H_q, H_kv, D, B = 8, 2, 64, 2
    g = torch.Generator().manual_seed(3)
    P, slots = 40, 16
    bt = torch.randperm(P, generator=g)[:B * slots].view(B, slots).to(torch.int32)
    chunks = [[60, 7], [33, 0], [1, 90]]
    pools = [torch.full((P, ps, H_kv, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    codes = [torch.full((P, ps, H_kv, D), 0x7f, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.full((P, ps, H_kv), float("nan"), device=DEV) for _ in range(2)]
    scale = D ** -0.5
    L = np.zeros(B, dtype=np.int64)
    for n in chunks:
        L = L + n
        T = sum(n)
        ptr = np.concatenate([[0], np.cumsum(n)])
        qkv = torch.randn(T, H_q + 2 * H_kv, D, generator=g).to(torch.bfloat16).to(DEV)
        q, k, v = qkv[:, :H_q], qkv[:, H_q:H_q + H_kv], qkv[:, H_q + H_kv:]
        dev = (bt.to(DEV), _i32(L), _i32(ptr))
        ts.ts_kv_append_chunk(k, v, *pools, *dev)
        ts.ts_kv_append_chunk_fp8(k, v, *codes, *scales, *dev)
        starts = np.concatenate([[0], np.cumsum((L + ps - 1) // ps * ps)])
        flat = [torch.zeros(int(starts[-1]), H_kv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        ts.ts_kv_read_fp8(*codes, *scales, dev[0], dev[1], _i32(starts), *flat)
        read = [f.view(-1, ps, H_kv, D) for f in flat]
        at = np.arange(slots)[None] + starts[:-1, None] // ps
        at = np.where(at < starts[1:, None] // ps, at, 0).astype(np.int32)
        for pk, pv, table in ((*pools, bt.numpy()), (*read, at)):
            out, lse = ts.ts_paged_prefill_attn(q, pk, pv, _i32(table), dev[1], dev[2], scale, return_lse=True)
            dq = torch.randn(B, H_q, D, generator=g).to(torch.bfloat16)
            d_out, d_lse = ts.ts_paged_decode_sink_attn(dq.to(DEV), pk, pv, _i32(table), dev[1], scale, 20, 3,
                                                        return_lse=True)
            torch.cuda.synchronize()
            kk, vv = pk.double().cpu().numpy(), pv.double().cpu().numpy()
            args = (table, L, ptr, scale)
            qd = q.double().cpu().numpy()
            ref = (*oracle.prefill_attention(qd, kk, vv, *args), oracle.prefill_attention(qd, kk, np.abs(vv), *args)[0],
                   scale * np.nanmax(np.abs(kk).sum(-1)) * np.abs(qd).max())
            check_attention(out, lse, ref, D, int(L.max()), "bf16")
            dd = dq.double().numpy()
            ref = (*oracle.decode_attention_sinks(dd, kk, vv, table, L, scale, 20, 3),
                   oracle.decode_attention_sinks(dd, kk, np.abs(vv), table, L, scale, 20, 3)[0],
                   scale * np.nanmax(np.abs(kk).sum(-1)) * np.abs(dd).max())
            check_attention(d_out, d_lse, ref, D, int(L.max()), "bf16")


def test_appends_and_attention_captured_together():
    """The step of a server as one graph, replayed with new rows and lengths."""
    case = ChunkCase(20, [30, 50], [40, 0], 8, 2, 64)
    a = case.device()
    T = case.T
    kn, vn = (torch.zeros(T, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = ts.new_workspace(ts.ts_paged_prefill_workspace_size(T, 2, 8, 2, 64))
    out = torch.zeros(T, 8, 64, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(T, 8, device=DEV)

    def step():
        ts.ts_kv_append_chunk(kn, vn, a["k_pool"], a["v_pool"], a["block_table"], a["seq_lens"], a["q_indptr"])
        ts.ts_paged_prefill_attn(**a, workspace=ws, out=out, lse=lse)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(1)
    for n in ([30, 50], [45, 35]):
        case.n = np.array(n)
        case.L = np.array([70, 50]) if n[0] == 30 else np.array([60, 45])
        case.indptr = np.array([0, n[0], 80], dtype=np.int32)
        a["seq_lens"].copy_(torch.from_numpy(case.L.astype(np.int32)))
        a["q_indptr"].copy_(torch.from_numpy(case.indptr))
        kn.copy_(torch.randn(T, 2, 64, generator=g).to(torch.bfloat16))
        vn.copy_(torch.randn(T, 2, 64, generator=g).to(torch.bfloat16))
        want = oracle.kv_append_chunk(a["k_pool"].double().cpu().numpy(), a["v_pool"].double().cpu().numpy(),
                                      kn.double().cpu().numpy(), vn.double().cpu().numpy(), case.bt, case.L,
                                      case.indptr)
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((a["k_pool"], a["v_pool"]), want):
            assert np.array_equal(got.double().cpu().numpy(), ref, equal_nan=True)
        assert ts.ts_read_device_error(ws) == 0
        check_attention(out, lse, case.oracle(torch.from_numpy(want[0]), torch.from_numpy(want[1])), 64, 80, "bf16")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_fp8_append_of_infinities_nan_and_extremes_is_the_single_tokens(dtype, D):
    """Groups with infinities, NaN, both, the type's largest and smallest values, all equal."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(40, 3, D, generator=g)
    inf, nan, top = float("inf"), float("nan"), torch.finfo(dtype).max
    for row, (i, value) in enumerate([(0, inf), (5, -inf), (D - 1, nan), (3, -nan), (7, top), (8, -top),
                                      (9, torch.finfo(dtype).tiny)]):
        x[row, 0, i] = value
        x[row + 7, 1] = value
    x[14, 2, 3], x[14, 2, 4] = inf, nan
    x[15], x[16] = 1e-30, -0.0
    x[17] = torch.finfo(dtype).tiny
    x = x.to(dtype).to(DEV)
    bt = torch.randperm(5, generator=g).to(torch.int32)[None].to(DEV)
    new = [torch.zeros(5, 8, 3, D, dtype=torch.uint8, device=DEV) for _ in range(2)]
    new += [torch.zeros(5, 8, 3, device=DEV) for _ in range(2)]
    old = [torch.zeros_like(t) for t in new]
    ts.ts_kv_append_chunk_fp8(x, -x, *new, bt, _i32([40]), _i32([0, 40]))
    ts.ts_kv_append_fp8(x, -x, *old, bt.expand(40, -1).contiguous(), torch.arange(40, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for a, b in zip(new, old):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H_kv,D", [(5, 64), (3, 128), (8, 128)])
def test_fp8_append_of_many_rows_equals_that_of_few(dtype, H_kv, D):
    """From 80 rows per SM on a warp takes a row's K and V; below, one of them."""
    n = 81 * torch.cuda.get_device_properties(0).multi_processor_count
    k, v, bt, L, ptr, P = _batch(H_kv + D, [n - 7, 0, 7], [3, 5, 40], H_kv, D, 16, dtype, fused=True)
    k, v = k.to(DEV), v.to(DEV)
    caches = []
    for parts in (1, 3):
        cache = [torch.full((P, 16, H_kv, D), 0x55, dtype=torch.uint8, device=DEV) for _ in range(2)] + \
                [torch.full((P, 16, H_kv), -1.0, device=DEV) for _ in range(2)]
        at = np.linspace(0, n, parts + 1).astype(int)
        for lo, hi in zip(at[:-1], at[1:]):  # rows lo .. hi of every sequence that has some there
            own = np.clip(ptr, lo, hi)
            ts.ts_kv_append_chunk_fp8(k[lo:hi], v[lo:hi], *cache, _i32(bt), _i32(L - (ptr[1:] - own[1:])),
                                      _i32(own - lo))
        caches.append(cache)
    torch.cuda.synchronize()
    for whole, pieces in zip(*caches):
        assert torch.equal(whole, pieces)
    assert (caches[0][2] >= 0).sum().item() == n * H_kv


def test_more_sequences_than_two_steps_of_the_search():
    """The search over row offsets takes three steps from 1025 sequences on."""
    rng = np.random.default_rng(8)
    n, ctx = rng.integers(0, 3, size=1500), rng.integers(0, 20, size=1500)
    k, v, bt, L, ptr, P = _batch(8, n, ctx, 2, 64, 8, torch.bfloat16)
    pools = [torch.full((P, 8, 2, 64), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    before = [_bits(p).cpu().numpy() for p in pools]
    ts.ts_kv_append_chunk(k.to(DEV), v.to(DEV), *pools, _i32(bt), _i32(L), _i32(ptr))
    torch.cuda.synchronize()
    ref = oracle.kv_append_chunk(*before, _bits(k).numpy(), _bits(v).numpy(), bt, L, ptr)
    for got, want in zip(pools, ref):
        assert np.array_equal(_bits(got).cpu().numpy(), want)


@pytest.mark.parametrize("ps", [1, 7, 24, 100])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pages_of_any_size(ps, dtype):
    """The appends and the read-back take page sizes that are no powers of two (and one row)."""
    n, ctx, H_kv, D = [130, 0, 1, 50], [0, 31, 100, 23], 2, 64
    k, v, bt, L, ptr, P = _batch(ps, n, ctx, H_kv, D, ps, dtype, pad=3)
    dev = (_i32(bt), _i32(L), _i32(ptr))
    pools = [torch.full((P, ps, H_kv, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2)]
    before = [_bits(p).cpu().numpy() for p in pools]
    ts.ts_kv_append_chunk(k.to(DEV), v.to(DEV), *pools, *dev)
    cache = [torch.full((P, ps, H_kv, D), 0x38, dtype=torch.uint8, device=DEV) for _ in range(2)]
    cache += [torch.ones(P, ps, H_kv, device=DEV) for _ in range(2)]
    before8 = [t.cpu().numpy() for t in cache]
    ts.ts_kv_append_chunk_fp8(k.to(DEV), v.to(DEV), *cache, *dev)
    starts = np.concatenate([[2], 2 + np.cumsum(L + 1)])
    outs = [torch.full((int(starts[-1]) + 2, H_kv, D), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
    ts.ts_kv_read_fp8(*cache, dev[0], dev[1], _i32(starts), *outs)
    torch.cuda.synchronize()
    for got, want in zip(pools, oracle.kv_append_chunk(*before, _bits(k).numpy(), _bits(v).numpy(), bt, L, ptr)):
        assert np.array_equal(_bits(got).cpu().numpy(), want)
    ref = oracle.kv_append_chunk_fp8(*before8, k.float().numpy(), v.float().numpy(), bt, L, ptr)
    for got, want in zip(cache, ref):
        assert np.array_equal(got.cpu().numpy(), want)
    for i, got in enumerate(outs):
        want = oracle.kv_read_fp8(ref[i], ref[2 + i], bt, L, starts, np.full(outs[i].shape, 7.0))
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(dtype))


def _quantized(x):
    """Codes and scales of rows x [T, H_kv, D] as both quantizing appends store them, in order of the rows."""
    T, H_kv, D = x.shape
    bt = torch.arange(T, dtype=torch.int32, device=DEV)
    made = []
    for chunk in (True, False):
        cache = [torch.zeros(T, 1, H_kv, D, dtype=torch.uint8, device=DEV) for _ in range(2)]
        cache += [torch.zeros(T, 1, H_kv, device=DEV) for _ in range(2)]
        if chunk:
            ts.ts_kv_append_chunk_fp8(x, -x, *cache, bt[None].contiguous(), _i32([T]), _i32([0, T]))
        else:
            ts.ts_kv_append_fp8(x, -x, *cache, bt[:, None].contiguous(), torch.zeros_like(bt))
        torch.cuda.synchronize()
        assert torch.equal(cache[0] ^ 0x80, cache[1]) and torch.equal(cache[2], cache[3])
        made.append((cache[0][:, 0].cpu().numpy(), cache[2][:, 0].cpu().numpy()))
    return made


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_fp8_append_of_every_bf16_ratio_up_to_the_maximum(dtype):
    """All 2432 bf16 values of 2^-18 up to the group's maximum, times tops of many significands: the last
    ones are the quotients beside the clamp."""
    vals = torch.arange(0x3600, 0x3f81, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    assert len(vals) == 2433 and vals[-1] == 1.0
    vals = torch.cat([vals, vals[-1:].expand(-len(vals) % 127)]).view(-1, 127)
    tops = (1.0, 1.5, 1.0078125, 1.9921875, 7.0, 448.0, 0.33, 3e-10, 2.0 ** 100)
    x = torch.stack([torch.cat([vals * top, torch.full((len(vals), 1), top)], 1) for top in tops], 1).to(dtype)
    codes, scales = oracle.quantize_token_groups(x.float().numpy())
    for got in _quantized(x.to(DEV)):
        assert np.array_equal(got[0], codes) and np.array_equal(got[1], scales)


def test_fp8_append_of_float32_values_beside_every_border():
    """float32 values within four units in the last place of every border between two codes, and of every
    code, times scales of random significands, of all ones and of powers of two, over the type's range:
    the quotients' rounding decides the code."""
    rng = np.random.default_rng(9)
    grid = oracle.fp8.e4m3_decode(np.arange(0x7f))  # 0 .. 448
    borders = np.concatenate([grid[1:], (grid[1:] + grid[:-1]) / 2])
    ones = np.float32(2.0) - np.float32(2.0 ** -23)
    rows, exact = [], 0
    for i in range(700):
        e = rng.integers(-44, 118)
        m = (1 + rng.random(), ones, 1.0)[0 if i % 7 > 1 else 1 + i % 7]
        scale = np.float32(float(m) * 2.0 ** e)
        top = np.float32(np.float64(scale) * 448)
        scale = np.float32(max(top, np.float32(1e-10))) / np.float32(448)
        exact += ((~scale.view(np.uint32)) & 0x7fffff) == 0
        x = np.abs(borders * np.float64(scale)).astype(np.float32)
        off = rng.integers(-4, 5, size=x.shape, dtype=np.int32)
        x = (x.view(np.int32) + off).view(np.float32)
        x = np.minimum(x, top)
        x = np.concatenate([x, x[:-len(x) % 127]]).reshape(-1, 127)
        rows.append(np.concatenate([x, np.full((len(x), 1), top)], 1))
    assert exact > 50
    x = np.stack(rows, 1)[:, :, rng.permutation(128)]  # [rows, scales, 128]: four scales a row of the cache
    x = np.ascontiguousarray(x.reshape(-1, 4, 128))
    codes, scales = oracle.quantize_token_groups(x)
    for got in _quantized(torch.from_numpy(x).to(DEV)):
        assert np.array_equal(got[1], scales)
        assert np.array_equal(got[0], codes), np.argwhere(got[0] != codes)[:5]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_padding_rows_may_hold_anything(dtype):
    """NaN in the input rows in front of the first sequence and behind the last: the results are those of
    the rows alone, and no padding row of a result is written."""
    n, ctx, H_q, H_kv, D, ps, front, back = [70, 0, 20], [0, 9, 300], 8, 2, 64, 16, 9, 30
    k, v, bt, L, ptr, P = _batch(11, n, ctx, H_kv, D, ps, dtype)
    T, g = len(k), torch.Generator().manual_seed(12)
    q = torch.randn(T, H_q, D, generator=g).to(dtype)
    cached = [torch.randn(P, ps, H_kv, D, generator=g).to(dtype) for _ in range(2)]
    runs = []
    for pad in (False, True):
        def rows(t):
            t = t.to(DEV)
            nan = lambda count: torch.full((count, *t.shape[1:]), float("nan"), dtype=dtype, device=DEV)  # noqa: E731
            return torch.cat([nan(front), t, nan(back)]) if pad else t
        meta = (_i32(bt), _i32(L), _i32(ptr + front if pad else ptr))
        pools = [c.to(DEV) for c in cached]
        cache = [torch.zeros(P, ps, H_kv, D, dtype=torch.uint8, device=DEV) for _ in range(2)]
        cache += [torch.zeros(P, ps, H_kv, device=DEV) for _ in range(2)]
        ts.ts_kv_append_chunk(rows(k), rows(v), *pools, *meta)
        ts.ts_kv_append_chunk_fp8(rows(k), rows(v), *cache, *meta)
        total = T + (front + back if pad else 0)
        out = torch.full((total, H_q, D), 7.0, dtype=dtype, device=DEV)
        lse = torch.full((total, H_q), 7.0, device=DEV)
        ts.ts_paged_prefill_attn(rows(q), *pools, *meta, D ** -0.5, out=out, lse=lse)
        torch.cuda.synchronize()
        if pad:
            for t in (out, lse):
                assert torch.all(t[:front] == 7.0) and torch.all(t[front + T:] == 7.0)
            out, lse = out[front:front + T], lse[front:front + T]
        runs.append(pools + cache)
        kk, vv, qd = (t.double().cpu().numpy() for t in (*pools, q))
        args = (bt, L, ptr, D ** -0.5)
        ref = (*oracle.prefill_attention(qd, kk, vv, *args), oracle.prefill_attention(qd, kk, np.abs(vv), *args)[0],
               D ** -0.5 * np.abs(kk).sum(-1).max() * np.abs(qd).max())
        check_attention(out, lse, ref, D, int(L.max()), "bf16" if dtype == torch.bfloat16 else "f32", f"padding {pad}")
    for alone, padded in zip(*runs):
        assert torch.equal(alone, padded)
