"""Refusals of the long-context entry points, on the host (no GPU)."""

import ctypes

import pytest
import torch

import paged_kv_cache_46_gb300 as ts

VP = ctypes.c_void_p(256)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_46_gb300 import build
    build.build()
    return ts.lib()


def _call(fn, good, **over):
    assert set(over) <= set(good)
    return fn(*{**good, **over}.values())


INVALID, UNSUPPORTED, WORKSPACE, OK = (ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED, ts.TS_ERR_WORKSPACE, ts.TS_OK)


def test_rope_append_refuses_on_the_host(lib):
    good = dict(q=VP, q_stride=32 * 128, k=VP, v=VP, step=8 * 128, qw=VP, kw=None, eps=1e-6, freq=VP, rot=128, inter=0,
                kp=VP, vp=VP, bt=VP, bts=4, lens=VP, ptr=VP, T=5, B=2, H_q=32, H_kv=8, D=128, ps=16, P=8, dt=1, out=VP,
                out_stride=32 * 128, stream=None)
    call = lambda **o: _call(lib.ts_kv_append_chunk_rope, good, **o)  # noqa: E731
    for bad in (dict(T=-1), dict(B=-1), dict(H_q=0), dict(H_kv=0), dict(ps=0), dict(P=0), dict(bts=0), dict(dt=2),
                dict(rot=-8), dict(rot=136), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(q_stride=32 * 128 - 8), dict(step=8 * 128 - 8), dict(out_stride=8), dict(q=None), dict(v=None),
                dict(freq=None), dict(lens=None), dict(out=None), dict(qw=ctypes.c_void_p(8)),
                dict(out=ctypes.c_void_p(264)), dict(freq=ctypes.c_void_p(258))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D=96, rot=96), dict(rot=12), dict(q_stride=32 * 128 + 4), dict(step=8 * 128 + 4),
                dict(out_stride=32 * 128 + 4), dict(H_q=4097, q_stride=1 << 20, out_stride=1 << 20)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(T=0, q=None, out=None) == call(B=0, q=None) == OK


def test_page_bounds_refuse_on_the_host(lib):
    good = dict(k=VP, bounds=VP, scale=VP, bt=VP, bts=4, lens=VP, ptr=VP, T=5, B=2, H_kv=8, D=128, ps=16, P=8, dt=1,
                stream=None)
    call = lambda **o: _call(lib.ts_kv_page_bounds, good, **o)  # noqa: E731
    for bad in (dict(T=-1), dict(B=-1), dict(H_kv=0), dict(ps=0), dict(P=0), dict(bts=0), dict(dt=2), dict(k=None),
                dict(scale=None), dict(ptr=None), dict(bounds=ctypes.c_void_p(8)), dict(scale=ctypes.c_void_p(6))):
        assert call(**bad) == INVALID, bad
    assert call(D=96) == call(H_kv=4097) == UNSUPPORTED
    assert call(T=0, k=None) == call(B=0, k=None) == OK


def test_select_pages_refuses_on_the_host(lib):
    good = dict(q=VP, bounds=VP, scale=VP, bt=VP, bts=40, lens=VP, B=2, q_len=1, H_q=32, H_kv=8, D=128, ps=16, P=8,
                pages=8, first=1, last=1, dt=1, idx=VP, ws=VP, wsb=1 << 40, stream=None)
    call = lambda **o: _call(lib.ts_select_pages, good, **o)  # noqa: E731
    for bad in (dict(B=-1), dict(q_len=0), dict(H_q=30), dict(H_kv=0), dict(ps=0), dict(P=0), dict(bts=0), dict(dt=2),
                dict(pages=0), dict(first=-1), dict(last=0), dict(first=5, last=4), dict(q=None), dict(idx=None),
                dict(lens=None), dict(q=ctypes.c_void_p(8)), dict(bounds=ctypes.c_void_p(8)),
                dict(first=2 ** 31 - 1, last=2 ** 31 - 1)):
        assert call(**bad) == INVALID, bad
    assert call(D=96) == call(H_q=24) == call(H_kv=3, H_q=12) == call(H_kv=16) == call(B=(1 << 24) + 1) == UNSUPPORTED
    assert call(B=0, q=None, ws=None, wsb=0) == OK
    size = lib.ts_select_pages_workspace_size
    assert size(2, 1, 8, 40) >= 256 + 2 * 8 * 40 * 4
    assert size(-1, 1, 8, 40) == size(2, 0, 8, 40) == size(2, 1, 9, 40) == size(2, 1, 8, 0) == 0
    assert call(wsb=size(2, 1, 8, 40) - 1) == call(ws=None) == call(ws=ctypes.c_void_p(128)) == WORKSPACE


def test_sparse_decode_refuses_on_the_host(lib, monkeypatch):
    monkeypatch.setenv("TS_PAGED_DECODE_CTAS", "8")  # the size follows the CTAs
    good = dict(q=VP, k=VP, v=VP, bt=VP, bts=40, lens=VP, idx=VP, pages=32, B=1, q_len=1, H_q=8, H_kv=2, D=64, ps=16,
                P=8, scale=1.0, dt=1, out=VP, lse=None, ws=VP, wsb=1 << 40, stream=None)
    call = lambda **o: _call(lib.ts_paged_decode_sparse_attn, good, **o)  # noqa: E731
    for bad in (dict(B=-1), dict(q_len=0), dict(H_q=7), dict(H_kv=0), dict(ps=0), dict(P=0), dict(bts=0), dict(dt=2),
                dict(pages=0), dict(P=1 << 27), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None),
                dict(idx=None), dict(out=None), dict(k=ctypes.c_void_p(8)), dict(out=ctypes.c_void_p(8))):
        assert call(**bad) == INVALID, bad
    assert call(D=96) == call(H_q=6) == call(H_kv=16, H_q=16) == call(ps=64) == call(ps=24) == UNSUPPORTED
    assert call(B=(1 << 24) + 1) == UNSUPPORTED
    assert call(B=0, q=None, ws=None, wsb=0) == OK
    size = lib.ts_paged_decode_sparse_workspace_size
    need = size(1, 1, 8, 2, 64, 16, 32)
    assert 256 < need <= size(4096, 1, 8, 2, 64, 16, 32) < 1 << 20  # two states for each warp of the grid at most
    assert size(-1, 1, 8, 2, 64, 16, 32) == size(1, 1, 8, 2, 96, 16, 32) == size(1, 1, 8, 2, 64, 16, 0) == 0
    assert call(wsb=need - 1) == call(ws=None) == call(ws=ctypes.c_void_p(128)) == WORKSPACE


def _buffers(*sizes, null=False):
    n = max(1, len(sizes))
    data, size = (ctypes.c_void_p * n)(*([None if null else 256] * len(sizes))), (ctypes.c_int64 * n)(*sizes)
    return ctypes.addressof(data), ctypes.addressof(size), (data, size)


def test_forks_and_compaction_refuse_on_the_host(lib):
    data, size, keep = _buffers(4096, 32)
    fork = dict(data=data, size=size, nb=2, bt=VP, bts=4, lens=VP, B=4, parents=VP, children=VP, fresh=VP, n=2, ps=16,
                P=8, stream=None)
    call = lambda **o: _call(lib.ts_kv_fork, fork, **o)  # noqa: E731
    zero, null, huge = _buffers(4096, 0), _buffers(4096, null=True), _buffers((1 << 30) + 1)
    shared = [dict(data=None), dict(size=None), dict(nb=-1), dict(data=zero[0], size=zero[1]),
              dict(data=null[0], size=null[1], nb=1), dict(data=huge[0], size=huge[1], nb=1), dict(B=-1), dict(bts=0),
              dict(ps=0), dict(P=0), dict(bt=None), dict(lens=None)]
    for bad in shared + [dict(n=-1), dict(parents=None), dict(children=None), dict(fresh=None)]:
        assert call(**bad) == INVALID, bad
    assert call(n=0, bt=None) == call(B=0, bt=None) == OK
    large = _buffers(1 << 30)
    assert call(data=large[0], size=large[1], nb=1, n=1 << 20) == UNSUPPORTED
    many = _buffers(*[16] * 200, 1 << 30)  # the last buffers alone are too many pieces: nothing of the call runs
    assert call(data=many[0], size=many[1], nb=201, n=1 << 20) == UNSUPPORTED
    compact = dict(data=data, size=size, nb=2, bt=VP, out=VP, bts=4, lens=VP, B=4, ps=16, P=8, page_map=VP, used=VP,
                   ws=VP, wsb=1 << 40, stream=None)
    call = lambda **o: _call(lib.ts_kv_compact, compact, **o)  # noqa: E731
    for bad in shared + [dict(out=None), dict(page_map=None), dict(used=None)]:
        assert call(**bad) == INVALID, bad
    need = lib.ts_kv_compact_workspace_size(8)
    assert need > 512 and lib.ts_kv_compact_workspace_size(0) == 0
    assert call(wsb=need - 1) == call(ws=None) == call(ws=ctypes.c_void_p(128)) == WORKSPACE


def _refuses(fn, good, *cases):
    for over, error in (*cases, (dict(), ValueError)):  # the last: tensors that are on no GPU
        with pytest.raises(error):
            fn(**{**good, **over})


def test_binding_refuses_what_it_would_have_to_guess():
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    bf = torch.bfloat16
    bt, lens, ptr = torch.zeros(2, 2, dtype=torch.int32), i32(4, 2), i32(0, 4, 6)
    pool, k, q = torch.zeros(3, 16, 2, 64), torch.zeros(6, 2, 64), torch.zeros(6, 4, 64)
    _refuses(ts.ts_kv_append_chunk_rope,
             dict(q=q, k_new=k, v_new=k, k_pool=pool, v_pool=pool, block_table=bt, seq_lens=lens, q_indptr=ptr,
                  inv_freq=torch.ones(32)),
             (dict(q=q.to(bf)), TypeError), (dict(k_pool=pool.to(bf)), TypeError), (dict(q=q[:5]), ValueError),
             (dict(q=torch.zeros(6, 4, 128)), ValueError), (dict(q=q.transpose(1, 2)), ValueError),
             (dict(q_weight=torch.ones(32)), ValueError), (dict(k_weight=torch.ones(64).to(bf)), ValueError),
             (dict(inv_freq=torch.ones(32).double()), TypeError), (dict(inv_freq=torch.ones(4, 8)), TypeError),
             (dict(q_out=q[:5]), ValueError), (dict(q_out=q.to(bf)), ValueError),
             (dict(q_indptr=ptr.long()), TypeError),
             (dict(v_new=torch.zeros(6, 5, 64)[:, :2]), ValueError), (dict(q_indptr=i32(0, 6)), ValueError))
    bounds, scale = torch.zeros(3, 2, 2, 64, dtype=torch.int8), torch.zeros(3, 2)
    shapes = ((dict(bounds=bounds.float()), TypeError), (dict(bound_scale=scale.double()), TypeError),
              (dict(bounds=bounds[:, :, :1]), ValueError), (dict(bound_scale=scale[:2]), ValueError),
              (dict(seq_lens=lens.long()), TypeError), (dict(block_table=bt[:1]), ValueError))
    _refuses(ts.ts_kv_page_bounds,
             dict(k_pool=pool, bounds=bounds, bound_scale=scale, block_table=bt, seq_lens=lens, q_indptr=ptr, rows=6),
             *shapes, (dict(bounds=bounds[:2], bound_scale=scale[:2]), ValueError))
    q = torch.zeros(2, 4, 64)
    _refuses(ts.ts_select_pages,
             dict(q=q, bounds=bounds, bound_scale=scale, block_table=bt, seq_lens=lens, page_size=16, pages=4), *shapes,
             (dict(q=q[:1]), ValueError), (dict(q=q[0]), ValueError),
             (dict(page_idx=torch.zeros(2, 2, 3, dtype=torch.int32)), ValueError),
             (dict(page_idx=torch.zeros(2, 2, 4)), ValueError))
    idx = torch.zeros(2, 2, 4, dtype=torch.int32)
    _refuses(ts.ts_paged_decode_sparse_attn,
             dict(q=q, k_pool=pool, v_pool=pool, block_table=bt, seq_lens=lens, page_idx=idx, scale=0.1),
             (dict(q=q.to(bf)), TypeError), (dict(v_pool=pool[:2]), ValueError), (dict(q=q[:1]), ValueError),
             (dict(q=torch.zeros(2, 4, 128)), ValueError), (dict(page_idx=idx.long()), ValueError),
             (dict(page_idx=idx[:, :1]), ValueError), (dict(q=torch.zeros(2, 1, 4, 64)), ValueError),
             (dict(out=q[:1]), ValueError), (dict(lse=torch.zeros(2, 5)), ValueError))
    with pytest.raises(ValueError):
        ts.kv_buffers([pool])  # on no GPU
    with pytest.raises(ValueError):
        ts.kv_buffers([pool, pool[:2]])
    with pytest.raises(ValueError):
        ts.ts_kv_fork([], bt, lens, i32(0), i32(1), i32(2), 16)
    with pytest.raises(ValueError):
        ts.ts_kv_compact([], bt, lens, 16)
