"""GPU parity of ts_kv_append_chunk_rope.

Bounds, from the formats (half a step of bf16 is 2^-8 of the value, of float32
2^-24): the normalised row is off by at most 12 * 2^-24 of itself (a sum of
squares over 12 additions a lane, halved by the root; rsqrtf 2 units = 4 half
steps; two products), a cosine or sine by 4 * 2^-24 (the angle's rounding,
2^-24 * pi / 4; sincospif, 2 units of a value below 1), a rotated value by the
sum over its two terms of both and of two more roundings: 20 * 2^-24 * (|y1| +
|y2|), with 2 to spare; then the output's own rounding."""

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_46_gb300 as ts
from long_context_cases import DEV, DTYPES, Cache, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _freq(rot, base=10000.0):
    return torch.from_numpy(base ** (-np.arange(rot // 2) / max(1, rot // 2))).float()


class Rows:
    def __init__(self, seed, n, ctx, H_q, H_kv, D, ps=16, dtype="bf16", rot=None, norm="qk", interleaved=False,
                 fused=False, pad=0):
        n = np.asarray(n)
        self.cache = Cache(seed, n + np.asarray(ctx), H_kv, D, ps, dtype)
        self.indptr = np.concatenate([[0], np.cumsum(n)])
        T = int(n.sum()) + pad
        self.q, self.k, self.v = (self.cache.normal(T, H, D) for H in (H_q, H_kv, H_kv))
        self.q[:, :, ::37] *= 12
        self.rot, self.interleaved, self.fused = D if rot is None else rot, interleaved, fused
        self.freq = _freq(self.rot)
        self.weights = {f"{x}_weight": (1 + 0.3 * self.cache.normal(D).float()).to(self.cache.dtype)
                        for x in "qk" if x in norm}

    def args(self):
        c = self.cache.device()
        q, k, v = (x.to(DEV) for x in (self.q, self.k, self.v))
        if self.fused:
            H_q, H_kv = q.shape[1], k.shape[1]
            q, k, v = torch.cat([q, k, v], 1).split([H_q, H_kv, H_kv], 1)
        return dict(q=q, k_new=k, v_new=v, **c, q_indptr=i32(self.indptr),
                    inv_freq=self.freq.to(DEV) if self.rot else None, eps=1e-5, interleaved=self.interleaved,
                    **{name: w.to(DEV) for name, w in self.weights.items()})

    def check(self, q_out, k_pool, v_pool, before, what=""):
        c, f = self.cache, lambda x: x.detach().double().cpu().numpy()  # noqa: E731
        w = {name: f(x) for name, x in self.weights.items()}
        want = oracle.kv_append_chunk_rope(f(self.q), f(self.k), f(self.v), f(c.k_pool), f(c.v_pool), c.table, c.lens,
                                           self.indptr, f(self.freq), eps=1e-5, interleaved=self.interleaved,
                                           q_out=f(before), **w)
        # |y1| + |y2| of a rotated value is at most sqrt(2) of its pair's length, which the rotation keeps
        half = 2.0 ** -8 if c.dtype == torch.bfloat16 else 2.0 ** -24
        for name, got, ref in zip("qk", (q_out, k_pool), want[:2]):
            pair = np.abs(ref).copy()
            r = self.rot // 2
            i = np.arange(r)
            one, two = (2 * i, 2 * i + 1) if self.interleaved else (i, i + r)
            pair[..., one] = pair[..., two] = np.sqrt(2 * (ref[..., one] ** 2 + ref[..., two] ** 2))
            got = f(got)
            same = np.isnan(ref) & np.isnan(got)
            err = np.where(same, 0, np.abs(got - ref))
            bound = np.where(same, 1, 1.01 * (22 * 2.0 ** -24 * pair + half * np.abs(ref)) + 1e-30)
            assert np.all(err <= bound), f"{what} {name}: off by {np.max(err / bound):.2f} of its bound"
        assert np.array_equal(f(v_pool), want[2], equal_nan=True), f"{what}: V"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rot,norm,interleaved,fused", [
    ("all", "qk", False, True), ("all", "", False, False), ("half", "q", True, True), ("half", "k", False, False),
    ("few", "qk", True, False), ("few", "", False, True), ("none", "qk", False, True), ("none", "", False, False)])
def test_rows(dtype, D, rot, norm, interleaved, fused):
    rot = {"all": D, "half": D // 2, "few": 8, "none": 0}[rot]
    case = Rows(11, [3, 0, 1, 17, 40], [0, 5, 900, 15, 130], 8, 2, D, 16, dtype, rot, norm, interleaved, fused, pad=3)
    a = case.args()
    out = torch.full((case.q.shape[0], 8, D), 7.0, dtype=case.cache.dtype, device=DEV)
    before = out.clone()
    got = ts.ts_kv_append_chunk_rope(**a, q_out=out)
    assert got is out
    case.check(out, a["k_pool"], a["v_pool"], before)
    assert torch.equal(out[-3:], before[-3:])  # rows of no sequence
    if rot == 0 and not norm:
        assert torch.equal(out[:-3], a["q"][:-3])


@pytest.mark.parametrize("H_q,H_kv", [(1, 1), (3, 1), (32, 8), (5, 5), (71, 3)])
@pytest.mark.parametrize("ps", [1, 7, 32])
def test_heads_and_page_sizes(H_q, H_kv, ps):
    case = Rows(12, [5, 1, 30], [20, 0, 3], H_q, H_kv, 64, ps)
    a = case.args()
    out = ts.ts_kv_append_chunk_rope(**a)
    case.check(out, a["k_pool"], a["v_pool"], torch.zeros_like(out))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_and_strided_queries(dtype):
    case = Rows(13, [9, 4], [100, 3], 4, 2, 128, 16, dtype, fused=True)
    a = case.args()
    rows = a["q"]  # a part of the projection's rows
    others = a["k_new"].clone()
    wide = torch.full((13, 6, 128), 3.0, dtype=case.cache.dtype, device=DEV)
    ts.ts_kv_append_chunk_rope(**a, q_out=wide[:, 1:5])
    assert (wide[:, 0] == 3).all() and (wide[:, 5] == 3).all()
    case.check(wide[:, 1:5], a["k_pool"], a["v_pool"], torch.zeros(13, 4, 128))
    ts.ts_kv_append_chunk_rope(**a, q_out=rows)
    assert torch.equal(rows, wide[:, 1:5]) and torch.equal(others, a["k_new"])


@pytest.mark.parametrize("dtype,last", [("bf16", 3_000_017), ("f32", 3_000_017), ("f32", 1_000_000_007)])
def test_far_positions(dtype, last):
    """Angles of far positions, where a float32 product would be off by whole turns' fractions."""
    case = Rows(14, [5], [0], 2, 1, 64, 16, dtype, norm="")
    c = case.cache
    c.ps = ps = 1 << 16
    c.lens = np.array([last + 1])
    c.table = np.full((1, last // ps + 1), -1, dtype=np.int32)
    c.table[0, -1] = 1
    c.k_pool, c.v_pool = (torch.full((2, ps, 1, 64), float("nan"), dtype=c.dtype) for _ in "kv")
    a = case.args()
    out = ts.ts_kv_append_chunk_rope(**a)
    case.check(out, a["k_pool"], a["v_pool"], torch.zeros_like(out))


def test_places_that_take_nothing():
    case = Rows(15, [6, 4, 4], [30, 0, 60], 4, 2, 64)
    c = case.cache
    c.lens[1] = 2           # two of its four rows are in front of the first token
    c.table[0, 2] = c.P     # the page of positions 32 ..
    c.table = c.table[:, :4]
    c.lens[2] = 66          # positions 62 .. 65: the table's row ends at 64
    a = case.args()
    out = torch.full((14, 4, 64), 7.0, dtype=c.dtype, device=DEV)
    before = out.clone()
    ts.ts_kv_append_chunk_rope(**a, q_out=out)
    case.check(out, a["k_pool"], a["v_pool"], before)
    assert torch.equal(out[6:8], before[6:8]) and not torch.equal(out[0], before[0])
    a["block_table"].fill_(-1)
    a["k_pool"].fill_(5), a["v_pool"].fill_(5)
    again = ts.ts_kv_append_chunk_rope(**a)
    assert torch.equal(again[0:6], out[0:6]) and (a["k_pool"] == 5).all() and (a["v_pool"] == 5).all()


def test_values_that_are_not_finite_stay_in_their_rows():
    case = Rows(16, [4], [12], 4, 2, 128, rot=64, norm="q")
    clean = case.args()
    want = ts.ts_kv_append_chunk_rope(**clean)
    for value in (float("nan"), float("inf")):
        a = case.args()
        a["q"][1, 2, 70] = value
        a["k_new"][2, 1, 100] = value  # a column that nothing touches
        a["k_new"][3, 0, 3] = value    # one that turns with column 35
        a["v_new"][0, 0, 5] = value
        out = ts.ts_kv_append_chunk_rope(**a)
        assert not torch.isfinite(out[1, 2]).all()
        out[1, 2] = want[1, 2]
        assert torch.equal(out, want)
        page = int(case.cache.table[0, 0])
        k, ref = a["k_pool"][page, 12:], clean["k_pool"][page, 12:].clone()
        ref[2, 1, 100] = value
        assert not torch.isfinite(k[3, 0, [3, 35]]).any()
        k[3, 0, [3, 35]] = ref[3, 0, [3, 35]]
        assert torch.equal(k.nan_to_num(9.0), ref.nan_to_num(9.0))
        assert torch.equal(a["v_pool"][page, 12:].nan_to_num(9.0), a["v_new"].nan_to_num(9.0))


def test_a_row_does_not_depend_on_its_batch():
    """One row a call, and the same rows among thousands: the heads of a row are shared out differently."""
    one = Rows(17, [3], [500], 8, 2, 128)
    many = Rows(18, [40] * 500 + [3], [0] * 500 + [500], 8, 2, 128)
    a, m = one.args(), many.args()
    for name in ("q", "k_new", "v_new"):
        m[name][-3:] = a[name]
    m.update(q_weight=a["q_weight"], k_weight=a["k_weight"])
    x, y = ts.ts_kv_append_chunk_rope(**a), ts.ts_kv_append_chunk_rope(**m)
    assert torch.equal(x, y[-3:])
    t = np.arange(500, 503)
    rows = [(int(c.table[-1, p // 16]), p % 16) for c in (one.cache, many.cache) for p in t]
    k = [a["k_pool"][r] for r in rows[:3]] + [m["k_pool"][r] for r in rows[3:]]
    assert all(torch.equal(k[i], k[i + 3]) for i in range(3))


def test_captured_steps_with_other_lengths_and_a_stream_of_its_own():
    case = Rows(19, [1] * 6, [3, 90, 31, 200, 15, 0], 8, 2, 64)
    a = case.args()
    pools = [a[name].clone() for name in ("k_pool", "v_pool")]
    out = torch.zeros_like(a["q"])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ts.ts_kv_append_chunk_rope(**a, q_out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ts.ts_kv_append_chunk_rope(**a, q_out=out)
    torch.cuda.synchronize()
    case.check(out, a["k_pool"], a["v_pool"], torch.zeros_like(out))
    for name, pool in zip(("k_pool", "v_pool"), pools):
        a[name].copy_(pool)
    case.cache.lens = case.cache.lens - np.array([1, 5, 0, 30, 3, 0])
    a["seq_lens"].copy_(i32(case.cache.lens))
    graph.replay()
    torch.cuda.synchronize()
    case.check(out, a["k_pool"], a["v_pool"], torch.zeros_like(out))
    x = ts.ts_kv_append_chunk_rope(**a, stream=side)
    side.synchronize()
    assert torch.equal(x, out)
