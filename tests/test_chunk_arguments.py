"""Refusals of the entry points for prompt chunks, on the host (no GPU)."""

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


def _prefill(lib, **o):
    a = dict(q=VP, q_stride=32 * 128, k=VP, v=VP, bt=VP, bts=4, lens=VP, ptr=VP, T=5, B=2, H_q=32, H_kv=8, D=128,
             ps=16, P=8, window=0, sinks=0, scale=1.0, dt=1, out=VP, lse=None, ws=VP, wsb=1 << 40, stream=None)
    a.update(o)
    return lib.ts_paged_prefill_attn(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), "TS_ERR_INVALID_ARG"), (dict(B=-1), "TS_ERR_INVALID_ARG"), (dict(H_kv=0), "TS_ERR_INVALID_ARG"),
    (dict(H_q=30), "TS_ERR_INVALID_ARG"), (dict(bts=0), "TS_ERR_INVALID_ARG"), (dict(P=1 << 27), "TS_ERR_INVALID_ARG"),
    (dict(T=(1 << 30) + 1), "TS_ERR_INVALID_ARG"), (dict(window=-1), "TS_ERR_INVALID_ARG"),
    (dict(sinks=-1), "TS_ERR_INVALID_ARG"), (dict(dt=2), "TS_ERR_INVALID_ARG"),
    (dict(scale=float("nan")), "TS_ERR_INVALID_ARG"), (dict(scale=float("inf")), "TS_ERR_INVALID_ARG"),
    (dict(q_stride=32 * 128 - 8), "TS_ERR_INVALID_ARG"), (dict(q=None), "TS_ERR_INVALID_ARG"),
    (dict(ptr=None), "TS_ERR_INVALID_ARG"), (dict(out=None), "TS_ERR_INVALID_ARG"),
    (dict(q=ctypes.c_void_p(264)), "TS_ERR_INVALID_ARG"), (dict(out=ctypes.c_void_p(260)), "TS_ERR_INVALID_ARG"),
    (dict(q_stride=32 * 128 + 4), "TS_ERR_UNSUPPORTED"), (dict(D=96), "TS_ERR_UNSUPPORTED"),
    (dict(ps=64), "TS_ERR_UNSUPPORTED"), (dict(ps=24), "TS_ERR_UNSUPPORTED"),
    (dict(H_q=65, H_kv=1, q_stride=65 * 128), "TS_ERR_UNSUPPORTED"),
    (dict(T=0, q=None, out=None, ws=None, wsb=0), "TS_OK"), (dict(B=0, q=None, ws=None, wsb=0), "TS_OK"),
])
def test_prefill_refuses_on_the_host(lib, over, status):
    assert _prefill(lib, **over) == getattr(ts, status), lib.ts_last_error_detail()


def test_prefill_workspace(lib, monkeypatch):
    # the size follows the CTAs, which this variable sets without a GPU
    monkeypatch.setenv("TS_PAGED_DECODE_CTAS", "4")
    size = lib.ts_paged_prefill_workspace_size
    small, large = size(20, 1, 32, 8, 128), size(4096, 1, 32, 8, 128)
    assert 0 < small < large and small % 256 == 0
    assert large >= 2 * 4 * 256 * 129 * 4
    for bad in ((-1, 1, 32, 8, 128), (5, -1, 32, 8, 128), (5, 1, 30, 8, 128), (5, 1, 32, 8, 96), (5, 1, 65, 1, 64)):
        assert size(*bad) == 0
    assert _prefill(lib, wsb=small - 1, T=20) == ts.TS_ERR_WORKSPACE
    assert _prefill(lib, ws=None, T=20) == ts.TS_ERR_WORKSPACE
    assert _prefill(lib, ws=ctypes.c_void_p(128), T=20) == ts.TS_ERR_WORKSPACE


def test_sink_decode_refuses_on_the_host(lib):
    def call(**o):
        a = dict(q=VP, k=VP, v=VP, bt=VP, bts=4, lens=VP, B=2, H_q=32, H_kv=8, D=128, ps=16, P=8, window=64, sinks=4,
                 scale=1.0, dt=1, out=VP, lse=None, ws=VP, wsb=1 << 40, stream=None)
        a.update(o)
        return lib.ts_paged_decode_sink_attn(*a.values())

    assert call(window=0) == call(window=-5) == call(sinks=-1) == ts.TS_ERR_INVALID_ARG
    assert call(scale=float("nan")) == call(q=None) == call(H_q=30) == call(B=-1) == ts.TS_ERR_INVALID_ARG
    assert call(H_q=24) == call(D=96) == call(ps=64) == ts.TS_ERR_UNSUPPORTED
    assert call(B=0, q=None, ws=None, wsb=0) == ts.TS_OK


def test_chunk_appends_refuse_on_the_host(lib):
    def plain(**o):
        a = dict(k=VP, v=VP, kp=VP, vp=VP, bt=VP, bts=4, lens=VP, ptr=VP, step=8 * 128, T=5, B=2, H_kv=8, D=128, ps=16,
                 P=8, dt=1, stream=None)
        a.update(o)
        return lib.ts_kv_append_chunk(*a.values())

    def fp8(**o):
        a = dict(k=VP, v=VP, kp=VP, vp=VP, ks=VP, vs=VP, bt=VP, bts=4, lens=VP, ptr=VP, step=8 * 128, T=5, B=2, H_kv=8,
                 D=128, ps=16, P=8, dt=1, stream=None)
        a.update(o)
        return lib.ts_kv_append_chunk_fp8(*a.values())

    for call in (plain, fp8):
        for bad in (dict(T=-1), dict(B=-1), dict(H_kv=0), dict(ps=0), dict(P=0), dict(bts=0), dict(dt=3),
                    dict(step=8 * 128 - 8), dict(k=None), dict(lens=None), dict(ptr=None), dict(kp=ctypes.c_void_p(8)),
                    dict(v=ctypes.c_void_p(24))):
            assert call(**bad) == ts.TS_ERR_INVALID_ARG, bad
        assert call(step=8 * 128 + 4) == ts.TS_ERR_UNSUPPORTED
        assert call(T=0, k=None) == call(B=0, k=None) == ts.TS_OK
    assert plain(D=3, H_kv=1, step=8) == ts.TS_ERR_UNSUPPORTED
    assert fp8(D=96) == ts.TS_ERR_UNSUPPORTED
    assert fp8(ks=None) == fp8(vs=ctypes.c_void_p(258)) == ts.TS_ERR_INVALID_ARG


def test_read_back_refuses_on_the_host(lib):
    def call(**o):
        a = dict(kp=VP, vp=VP, ks=VP, vs=VP, bt=VP, bts=4, lens=VP, ptr=VP, rows=5, B=2, H_kv=8, D=128, ps=16, P=8, dt=1,
                 k=VP, v=VP, stream=None)
        a.update(o)
        return lib.ts_kv_read_fp8(*a.values())

    for bad in (dict(rows=-1), dict(B=-1), dict(H_kv=0), dict(ps=0), dict(P=0), dict(bts=0), dict(dt=3), dict(kp=None),
                dict(ks=None), dict(ptr=None), dict(k=None), dict(v=ctypes.c_void_p(24)), dict(vs=ctypes.c_void_p(2))):
        assert call(**bad) == ts.TS_ERR_INVALID_ARG, bad
    assert call(D=96) == ts.TS_ERR_UNSUPPORTED
    assert call(rows=0, k=None) == call(B=0, k=None) == ts.TS_OK


def test_binding_refuses_what_it_would_have_to_guess():
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    q, pool = torch.zeros(6, 4, 64), torch.zeros(3, 16, 2, 64)
    bt, lens, ptr = torch.zeros(2, 2, dtype=torch.int32), i32(4, 2), i32(0, 4, 6)
    good = dict(q=q, k_pool=pool, v_pool=pool, block_table=bt, seq_lens=lens, q_indptr=ptr, scale=0.1)
    for over, error in ((dict(q_indptr=ptr.long()), TypeError), (dict(seq_lens=lens.long()), TypeError),
                        (dict(q_indptr=i32(0, 6)), ValueError), (dict(block_table=bt[:1]), ValueError),
                        (dict(k_pool=pool.bfloat16()), TypeError), (dict(v_pool=pool[:2]), ValueError),
                        (dict(q=torch.zeros(6, 4, 128)), ValueError), (dict(q=q.transpose(1, 2)), ValueError),
                        (dict(out=torch.zeros(6, 4, 64).bfloat16()), ValueError), (dict(out=q[:5]), ValueError),
                        (dict(lse=torch.zeros(6, 5)), ValueError), (dict(lse=torch.zeros(6, 4).double()), ValueError),
                        (dict(), ValueError)):  # the last: tensors that are on no GPU
        with pytest.raises(error):
            ts.ts_paged_prefill_attn(**{**good, **over})
    k = torch.zeros(6, 2, 64)
    good = dict(k_new=k, v_new=k, k_pool=pool, v_pool=pool, block_table=bt, seq_lens=lens, q_indptr=ptr)
    for over, error in ((dict(v_new=k[:5]), ValueError), (dict(k_new=k.bfloat16(), v_new=k.bfloat16()), TypeError),
                        (dict(k_new=torch.zeros(6, 3, 64), v_new=torch.zeros(6, 3, 64)), ValueError),
                        (dict(v_new=torch.zeros(6, 5, 64)[:, :2]), ValueError), (dict(), ValueError)):
        with pytest.raises(error):
            ts.ts_kv_append_chunk(**{**good, **over})
    codes, scales = torch.zeros(3, 16, 2, 64, dtype=torch.uint8), torch.zeros(3, 16, 2)
    for over, error in ((dict(k_pool=pool), TypeError), (dict(k_scale=scales[:2]), ValueError), (dict(), ValueError)):
        a = dict(k_new=k, v_new=k, k_pool=codes, v_pool=codes, k_scale=scales, v_scale=scales, block_table=bt,
                 seq_lens=lens, q_indptr=ptr)
        with pytest.raises(error):
            ts.ts_kv_append_chunk_fp8(**{**a, **over})
    for over, error in ((dict(k_out=torch.zeros(6, 2, 128)), ValueError),
                        (dict(v_out=torch.zeros(5, 2, 64)), ValueError), (dict(), ValueError)):
        a = dict(k_pool=codes, v_pool=codes, k_scale=scales, v_scale=scales, block_table=bt, seq_lens=lens,
                 kv_indptr=ptr, k_out=k, v_out=k.clone())
        with pytest.raises(error):
            ts.ts_kv_read_fp8(**{**a, **over})
    with pytest.raises(ValueError):
        ts.ts_paged_decode_sink_attn(q[:2], pool, pool, bt, lens, 0.1, 8, 2)
