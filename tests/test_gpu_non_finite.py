"""Scores that are not finite: a query that sees one has no softmax, so its O and LSE are NaN, and
every other row keeps its bounds. LSE = -inf is for rows that see nothing, which a merge drops."""

import os

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


def _spoil(case, b, t, head, value):
    """A copy of the key pool whose column 0 of token t, kv head `head`, of sequence b is `value`."""
    k = case.k_pool.clone()
    page, row = case.bt[b, t // case.ps], t % case.ps
    assert torch.isfinite(k[page, row, head]).all()
    k[page, row, head, 0] = value
    return k


def _reach(case):
    """Largest scaled sum |q k| of finite keys and queries, as ChunkCase.oracle gives it."""
    return case.scale * np.nanmax(case.k_pool.double().abs().sum(-1).numpy()) * case.q.double().abs().max().item()


def _check(out, lse, ref, qk, case, what):
    """Rows whose LSE is NaN in float64 are NaN, the others within their bounds (qk: see _reach)."""
    o_ref, l_ref, a_ref = (x.copy() for x in ref[:3])
    bad = np.isnan(l_ref)
    assert bad.any() and not bad.all(), what
    where = torch.from_numpy(bad).to(DEV)
    assert torch.isnan(lse[where]).all(), f"{what}: {lse[where][~torch.isnan(lse[where])][:5]}"
    assert torch.isnan(out[where]).all(), what
    o_ref[bad], l_ref[bad], a_ref[bad] = 0.0, 0.0, 0.0
    check_attention(out.masked_fill(where[..., None], 0.0), lse.masked_fill(where, 0.0), (o_ref, l_ref, a_ref, qk),
                    case.D, int(case.L.max()), case.dtype, what)


@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_prompt_attention_of_keys_that_are_not_finite(dtype, D, value, window, sinks):
    """Column 0 of a key is infinite or NaN: scores of both signs, for the rows that see the key. Items
    whole and cut between CTAs, where the merge has to keep them too."""
    case = ChunkCase(3, [200, 3, 70], [900, 260, 0], 8, 2, D, ps=16, dtype=dtype, window=window, sinks=sinks)
    k = _spoil(case, 0, 1030, 1, value)
    with np.errstate(invalid="ignore"):
        ref = case.oracle(k_pool=k)
    a = case.device()
    a["k_pool"] = k.to(DEV)
    for ctas in (152, 1):
        os.environ["TS_PAGED_DECODE_CTAS"] = str(ctas)
        try:
            out, lse = ts.ts_paged_prefill_attn(**a, return_lse=True)
        finally:
            os.environ.pop("TS_PAGED_DECODE_CTAS", None)
        torch.cuda.synchronize()
        _check(out, lse, ref, _reach(case), case, f"{value} W {window} {ctas} CTAs")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(dtype):
    case = ChunkCase(4, [140], [300], 8, 2, 64, dtype=dtype)
    a, qk = case.device(), _reach(case)
    case.q[77, 3, 5] = float("nan")
    a["q"] = case.q.to(DEV)
    with np.errstate(invalid="ignore"):
        ref = case.oracle()
    out, lse = ts.ts_paged_prefill_attn(**a, return_lse=True)
    torch.cuda.synchronize()
    assert np.isnan(ref[1]).sum() == 1
    _check(out, lse, ref, qk, case, "query")


@pytest.mark.parametrize("window,sinks", [(300, 20), (1000, 4)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_decode_with_first_tokens_of_keys_that_are_not_finite(dtype, D, value, window, sinks):
    """The key is the first one, the window's last but one, one in front of the window; sequences whole
    and cut between CTAs."""
    L = np.array([700, 640, 900, 1])
    case = ChunkCase(5, [1] * 4, L - 1, 8, 2, D, dtype=dtype, window=window, sinks=sinks)
    k = case.k_pool.clone()
    for b, t in ((0, 2), (1, 638), (2, 30)):
        page, row = case.bt[b, t // 16], t % 16
        k[page, row, b % 2, 0] = value
    args = (case.bt, case.L, case.scale, window, sinks)
    q, kd, v = (x.double().numpy() for x in (case.q, k, case.v_pool))
    with np.errstate(invalid="ignore"):
        ref = (*oracle.decode_attention_sinks(q, kd, v, *args),
               oracle.decode_attention_sinks(q, kd, np.abs(v), *args)[0])
    a = case.device()
    for ctas in (152, 1):
        os.environ["TS_PAGED_DECODE_CTAS"] = str(ctas)
        try:
            out, lse = ts.ts_paged_decode_sink_attn(a["q"], k.to(DEV), a["v_pool"], a["block_table"], a["seq_lens"],
                                                    case.scale, window, sinks, return_lse=True)
        finally:
            os.environ.pop("TS_PAGED_DECODE_CTAS", None)
        torch.cuda.synchronize()
        _check(out, lse, ref, _reach(case), case, f"{value} W {window} {ctas} CTAs")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_merge_keeps_a_state_whose_lse_is_nan(dtype):
    """Beside a finite state, an empty one and another NaN; an empty side's O does not count."""
    nan, none, D = float("nan"), -float("inf"), 64
    la = torch.tensor([nan, nan, 0.5, none, nan, none, none, 0.5], device=DEV)
    lb = torch.tensor([0.5, none, nan, nan, nan, none, 0.5, none], device=DEV)
    o = [torch.randn(8, D, generator=torch.Generator().manual_seed(i)).to(dtype).to(DEV) for i in range(2)]
    o[0][torch.isnan(la)], o[1][torch.isnan(lb)] = nan, nan
    o[0][5:7], o[1][5], o[1][7] = nan, nan, nan  # of empty states
    out, lse = ts.ts_merge_states(o[0], la, o[1], lb)
    torch.cuda.synchronize()
    assert torch.isnan(out[:5]).all() and torch.isnan(lse[:5]).all()
    assert (out[5] == 0).all() and lse[5].item() == none
    assert torch.equal(out[6], o[1][6]) and torch.equal(out[7], o[0][7]) and lse[6:].tolist() == [0.5, 0.5]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_quantized_groups_that_are_not_finite_read_back_as_nan(dtype, D):
    """Codes and scales are the definition's in IEEE arithmetic, from both appends: a NaN spoils its
    group (max and quotients are NaN), an infinity's own quotient is NaN and the others are zeros of
    an infinite scale. The groups beside them in the warp are exact."""
    g = torch.Generator().manual_seed(6)
    T, H_kv, ps = 24, 3, 8
    x = torch.randn(T, H_kv, D, generator=g)
    for t, values in enumerate([(float("inf"),), (-float("inf"),), (float("nan"),), (-float("nan"),),
                                (float("inf"), float("nan")), (float("inf"), -float("inf"))]):
        for i, value in enumerate(values):
            x[2 * t, t % 3, (7 * t + 3 * i) % D] = value
    x[21] = float("nan")
    x = x.to(dtype)
    xs = x.float().numpy()
    with np.errstate(invalid="ignore"):
        scale = (np.maximum(np.abs(xs).max(-1), np.float32(1e-10)) / np.float32(448)).astype(np.float32)
        y = (xs / scale[..., None]).astype(np.float32)
    nan = np.isnan(y)
    code = oracle.fp8.e4m3_encode(np.clip(np.where(nan, 0, y), -448, 448))
    assert nan.any() and np.isnan(scale).sum() == 6 and np.isinf(scale).sum() == 3
    bt = torch.randperm(T // ps, generator=g).to(torch.int32)[None]
    where = (bt[0].numpy()[np.arange(T) // ps], np.arange(T) % ps)
    x = x.to(DEV)
    lens, ptr = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([T], [0, T]))
    for chunk in (True, False):
        cache = [torch.zeros(T // ps, ps, H_kv, D, dtype=torch.uint8, device=DEV) for _ in range(2)]
        cache += [torch.zeros(T // ps, ps, H_kv, device=DEV) for _ in range(2)]
        if chunk:
            ts.ts_kv_append_chunk_fp8(x, -x, *cache, bt.to(DEV), lens, ptr)
        else:
            ts.ts_kv_append_fp8(x, -x, *cache, bt.expand(T, -1).contiguous().to(DEV),
                                torch.arange(T, dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        for i, flip in ((0, 0), (1, 0x80)):
            got = cache[i].cpu().numpy()[where]
            assert np.array_equal((got & 0x7f) == 0x7f, nan)
            assert np.array_equal(got[~nan], code[~nan] ^ flip)
            assert np.array_equal(cache[2 + i].cpu().numpy()[where], scale, equal_nan=True)
    out = [torch.zeros(T, H_kv, D, device=DEV) for _ in range(2)]
    ts.ts_kv_read_fp8(*cache, bt.to(DEV), lens, ptr, *out)
    torch.cuda.synchronize()
    for o in out:
        assert np.array_equal(torch.isnan(o).cpu().numpy(), np.repeat(~np.isfinite(scale)[..., None], D, -1))


def _cache(B, lens, H_kv, D, ps=16, shared=0, seed=7):
    """(K pool, V pool, block table [B, slots]) with the first `shared` pages of all sequences the same,
    and one more of two of them."""
    g = torch.Generator().manual_seed(seed)
    slots = (max(lens) + ps - 1) // ps
    bt = torch.arange(B * slots, dtype=torch.int32).view(B, slots)
    bt[:, :shared] = bt[0, :shared]
    if shared:
        bt[3, shared] = bt[2, shared]  # a deeper node of the last two
    pools = [torch.randn(B * slots, ps, H_kv, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    return *pools, bt.to(DEV)


def _q(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).to(DEV)


def _codes(t):
    """e4m3 codes and per-row scales of t."""
    code, scale = oracle.quantize_token_groups(t.float().cpu().numpy())
    return torch.from_numpy(code).to(DEV), torch.from_numpy(scale).to(DEV)


LENS = [1500, 33, 700, 64]


def _runs(which):
    """A query [..., heads, D] (last but one dimension: heads) and the call over it."""
    lens = torch.tensor(LENS, dtype=torch.int32, device=DEV)
    args = dict(seq_lens=lens, scale=0.1, return_lse=True)
    if which.startswith("mla"):
        pool, _, bt = _cache(4, LENS, 1, 576, ps=64)
        pool = pool.view(-1, 64, 576)
        q = _q(4, *((2,) if which.endswith("multi") else ()), 128, 576)
        if which == "mla_fp8":
            kv, scale = _codes(pool)
            q_code, q_scale = _codes(q)
            # NaN of the query's row reaches the kernel as its scale
            return q, lambda x: ts.ts_mla_paged_decode_fp8(
                q_code, torch.where(torch.isnan(x).any(-1), torch.full_like(q_scale, float("nan")), q_scale), kv,
                scale, bt, **args)
        fn = ts.ts_mla_paged_decode_multi if which.endswith("multi") else ts.ts_mla_paged_decode
        return q, lambda x: fn(x, pool, bt, **args)
    D, shared = (64, 2) if which.startswith("cascade") else (128, 0)
    k, v, bt = _cache(4, LENS, 8, D, shared=shared)
    if which.startswith("multi"):
        return _q(4, 4, 32, 128), lambda x: ts.ts_paged_decode_multi_attn(x, k, v, bt, **args)
    q = _q(4, 32, D)
    if which.startswith("fp8"):
        kc, vc, ks, vs = (c for pair in zip(*(_codes(t) for t in (k, v))) for c in pair)
        return q, lambda x: ts.ts_paged_decode_fp8_attn(x, kc, vc, ks, vs, bt, **args)
    host = (bt.cpu().numpy(), np.array(LENS, dtype=np.int32), 16)
    if which == "cascade":
        groups = ts.groups_to_device(ts.ts_group_prefixes(*host), DEV)
        return q, lambda x, key=k: ts.ts_cascade_decode_attn(x, key, v, groups, bt, **args)
    forest = ts.forest_to_device(ts.ts_group_prefixes_nested(*host), DEV)
    return q, lambda x, key=k: ts.ts_cascade_nested_decode_attn(x, key, v, forest, bt, **args)


PATHS = {"multi_cuda": ("TS_MULTI_QUERY_PATH", "cuda"), "multi_tensor": ("TS_MULTI_QUERY_PATH", "tensor"),
         "fp8_cuda": ("TS_FP8_DECODE_PATH", "cuda"), "fp8_tensor": ("TS_FP8_DECODE_PATH", "tensor"),
         "fp8_mma": ("TS_FP8_DECODE_PATH", "mma")}


@pytest.mark.parametrize("which", [*PATHS, "cascade", "cascade_nested", "mla", "mla_multi", "mla_fp8"])
def test_other_decode_calls_give_nan_for_a_query_that_is_not_finite(which, monkeypatch):
    """That row's O and LSE are NaN; the others are those of the clean query. Both runs round the weights
    (bf16, 2^-8 of each at most, the sum of weighted |V| below the largest |V|) and the output (2^-8)."""
    if which in PATHS:
        monkeypatch.setenv(*PATHS[which])
    q, call = _runs(which)
    clean, clean_lse = call(q)
    spoiled = q.clone()
    rows = [(0, 5), (1, 0), (2, 31)]
    for b, h in rows:
        spoiled[b, ..., h, 3] = float("nan")
    out, lse = call(spoiled)
    torch.cuda.synchronize()
    bad = torch.isnan(spoiled).any(-1)
    assert torch.isnan(lse[bad]).all(), lse[bad]
    assert torch.isnan(out[bad]).all()
    top = 5.5  # |V| of 10^6 standard normal values
    assert ((out[~bad].float() - clean[~bad].float()).abs() <= 2.0 ** -7 * (top + clean[~bad].float().abs())).all()
    assert ((lse[~bad] - clean_lse[~bad]).abs() <= 2.0 ** -20 * clean_lse[~bad].abs().clamp(min=16)).all()


@pytest.mark.parametrize("which", ["cascade", "cascade_nested"])
def test_a_shared_prefix_that_is_not_finite_is_not_dropped(which):
    """A NaN key of a shared page reaches every member of the group, at the heads of its kv head."""
    q, call = _runs(which)
    k, _, bt = _cache(4, LENS, 8, 64, shared=2)
    k[bt[0, 1].item(), 7, 2, 0] = float("nan")
    out, lse = call(q, k)
    torch.cuda.synchronize()
    assert torch.isnan(out[:, 8:12]).all() and torch.isnan(lse[:, 8:12]).all()
    for heads in (slice(0, 8), slice(12, 32)):
        assert torch.isfinite(out[:, heads]).all() and torch.isfinite(lse[:, heads]).all()
