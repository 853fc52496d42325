"""Ragged chunk batches over a paged cache for the GPU tests, and the bounds
their outputs are held to.

Bounds of an attention row, from the formats (half a step of bf16 is 2^-8 of
the value, of float32 2^-24) and the oracle's A = sum_t softmax_t |V_t|:

* score: a D-term float32 dot product of exact products is off by at most
  D * 2^-24 * sum |q k|, scaled; e^x turns an absolute error d of x into a
  relative one, d to first order. With exp's own error (2 units in the last
  place) a weight is off by at most w = 2 d + 2^-21 of its value after the
  normalisation, O by w A.
* the float32 sum over L weights and values: (L + D) 2^-24 A at most.
* bf16 path: each weight is rounded to bf16 for the product (2^-8 of itself):
  2^-8 A; the output's own rounding 2^-8 |O|.
* float32 output: 2^-24 |O|.
* LSE: d + the relative error of the sum, (L + 16) 2^-24, + 2^-24 |LSE|.

Each bound is taken once more by a hundredth for the second-order terms."""

from __future__ import annotations

import numpy as np
import torch

import oracle

DEV = "cuda"


class ChunkCase:
    """New tokens n[b] after ctx[b] cached ones. Rows that no query may read are NaN: unused
    pages, rows past a sequence's end, and (windowed) everything between the first tokens
    and the first query's window."""

    def __init__(self, seed, n, ctx, H_q, H_kv, D, ps=16, dtype="bf16", window=0, sinks=0, fused=False, pad_rows=0,
                 spare=3):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        n, L = np.asarray(n), np.asarray(n) + np.asarray(ctx)
        self.n, self.L, self.window, self.sinks, self.dtype, self.ps = n, L, window, sinks, dtype, ps
        need = (L + ps - 1) // ps
        P = int(need.sum()) + spare
        order = rng.permutation(P)
        bt = np.full((len(n), max(1, int(need.max()))), order[-1], dtype=np.int32)
        k = torch.full((P, ps, H_kv, D), float("nan"), dtype=dt)
        v = torch.full((P, ps, H_kv, D), float("nan"), dtype=dt)
        at = 0
        for b in range(len(n)):
            own = order[at:at + need[b]]
            at += int(need[b])
            bt[b, :need[b]] = own
            t = np.arange(int(L[b]))
            first = int(L[b] - n[b])  # position of the first query
            if window:
                t = t[(t > first - window) | (t < sinks)]
            k[own[t // ps], t % ps] = torch.randn(len(t), H_kv, D, generator=g).to(dt)
            v[own[t // ps], t % ps] = torch.randn(len(t), H_kv, D, generator=g).to(dt)
            if window:  # slots without a visible token hold a placeholder
                seen = np.unique(t // ps)
                gone = np.setdiff1d(np.arange(int(need[b])), seen)
                bt[b, gone] = order[-1]
        self.k_pool, self.v_pool, self.bt = k, v, bt
        self.T = int(n.sum()) + pad_rows
        self.indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.H_q, self.H_kv, self.D, self.scale = H_q, H_kv, D, D ** -0.5
        self.q = torch.randn(self.T, H_q + (2 * H_kv if fused else 0), D, generator=g).to(dt)
        self.fused = fused

    def device(self):
        q = self.q.to(DEV)[:, :self.H_q]
        return dict(q=q, k_pool=self.k_pool.to(DEV), v_pool=self.v_pool.to(DEV),
                    block_table=torch.from_numpy(self.bt).to(DEV),
                    seq_lens=torch.from_numpy(self.L.astype(np.int32)).to(DEV),
                    q_indptr=torch.from_numpy(self.indptr).to(DEV), scale=self.scale, window=self.window,
                    sinks=self.sinks)

    def oracle(self, k_pool=None, v_pool=None):
        """(O, LSE, A, largest scaled sum |q k|) in float64."""
        q = self.q[:, :self.H_q].double().numpy()
        k = (self.k_pool if k_pool is None else k_pool).double().numpy()
        v = (self.v_pool if v_pool is None else v_pool).double().numpy()
        args = (self.bt, self.L, self.indptr, self.scale, self.window, self.sinks)
        o, lse = oracle.prefill_attention(q, k, v, *args)
        a, _ = oracle.prefill_attention(q, k, np.abs(v), *args)
        reach = np.nanmax(np.abs(k).sum(-1)) if np.isfinite(k).any() else 0.0
        return o, lse, a, abs(self.scale) * reach * np.abs(q).max()


def check_attention(out, lse, ref, D, L, dtype, what=""):
    """Hold O and LSE to the bounds of the module's docstring."""
    o_ref, l_ref, a, qk = ref
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(np.isfinite(o)), f"{what}: non-finite output"
    d = D * 2.0 ** -24 * qk
    w = 2 * d + 2.0 ** -21 + (L + D) * 2.0 ** -24
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    bound = 1.01 * ((w + (half if dtype == "bf16" else 0.0)) * a + half * np.abs(o_ref)) + 1e-30
    err = np.abs(o - o_ref)
    assert np.all(err <= bound), f"{what}: O off by {err.max():.3e}, {np.max(err / bound):.2f} of its bound"
    none = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(l), none), f"{what}: -inf LSE mismatch"
    l_bound = 1.01 * (d + 2.0 ** -21 + (L + 16) * 2.0 ** -24 + 2.0 ** -24 * np.abs(l_ref[~none]))
    l_err = np.abs(l[~none] - l_ref[~none])
    assert np.all(l_err <= l_bound), f"{what}: LSE off by {l_err.max():.3e}"
