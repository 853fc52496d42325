"""Operators that serve a prompt in chunks over a paged cache, as measurable cases.

Five operators: the attention of a ragged batch of prompt chunks over a paged
cache (`prefill`), decode attention that sees a sliding window and a few first
tokens (`sinks`), writing a chunk's K/V rows into the pages (`append`), the
same while quantizing them to e4m3 codes (`append_fp8`), and reading a
quantized cache back into rows (`read_fp8`).

`run` computes a case in elementary torch operations where `own` is false, and
through the library's entry points where it is true.
"""

import math

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_E4M3_MAX = 448.0


def listed():
    return [
        # the last, short chunk of one user's prompt: latency counts
        dict(name="prefill_tail", op="prefill", dtype="bf16", B=1, H_q=32, H_kv=8, D=128, ps=16, lo=33, hi=33,
             ctx_lo=999, ctx_hi=999, window=0, sinks=0, fused=True, lengths=1),
        # a scheduler's step: 16 prompts of mixed lengths, some fresh, some continued
        dict(name="prefill_ragged", op="prefill", dtype="bf16", B=16, H_q=32, H_kv=8, D=128, ps=16, lo=1, hi=1024,
             ctx_lo=0, ctx_hi=4096, window=0, sinks=0, fused=True, lengths=2),
        # the last 4096-token chunk of a 32k-token document
        dict(name="prefill_long", op="prefill", dtype="bf16", B=1, H_q=32, H_kv=8, D=128, ps=16, lo=4096, hi=4096,
             ctx_lo=28672, ctx_hi=28672, window=0, sinks=0, fused=False, lengths=3),
        # streaming prompts: a window of 1024 tokens and 16 first tokens stay visible, head dim 64
        dict(name="prefill_sinks", op="prefill", dtype="bf16", B=6, H_q=32, H_kv=8, D=64, ps=16, lo=500, hi=2048,
             ctx_lo=0, ctx_hi=8192, window=1024, sinks=16, fused=False, lengths=4),
        # one streaming user, a small fp32 model: latency counts
        dict(name="sinks_one", op="sinks", dtype="f32", B=1, H_q=8, H_kv=2, D=64, ps=16, ctx_lo=1501, ctx_hi=1501,
             window=250, sinks=4, lengths=5),
        # a batch of long conversations at the Llama-3-8B layer's shape
        dict(name="sinks_batch", op="sinks", dtype="bf16", B=64, H_q=32, H_kv=8, D=128, ps=16, ctx_lo=4096,
             ctx_hi=32768, window=4096, sinks=64, lengths=6),
        # K/V rows of a short chunk, taken from a fused projection's output
        dict(name="append_tail", op="append", dtype="bf16", B=1, H_kv=8, D=128, ps=16, lo=33, hi=33, ctx_lo=999,
             ctx_hi=999, fused=True, lengths=7),
        # a full step of a prefill server: 32 chunks
        dict(name="append_batch", op="append", dtype="bf16", B=32, H_kv=8, D=128, ps=16, lo=1, hi=1024, ctx_lo=0,
             ctx_hi=4096, fused=True, lengths=8),
        # the same two into a quantized cache
        dict(name="append_fp8_tail", op="append_fp8", dtype="f32", B=1, H_kv=8, D=128, ps=16, lo=33, hi=33,
             ctx_lo=999, ctx_hi=999, fused=False, lengths=9),
        dict(name="append_fp8_batch", op="append_fp8", dtype="bf16", B=32, H_kv=8, D=128, ps=16, lo=1, hi=1024,
             ctx_lo=0, ctx_hi=4096, fused=True, lengths=10),
        # one user's quantized context, read back for the attention of its next chunk
        dict(name="read_fp8_one", op="read_fp8", dtype="bf16", B=1, H_kv=8, D=128, ps=16, ctx_lo=999, ctx_hi=999,
             lengths=11),
        # a batch's whole quantized cache, read back to be moved or attended
        dict(name="read_fp8_batch", op="read_fp8", dtype="bf16", B=64, H_kv=8, D=128, ps=16, ctx_lo=512,
             ctx_hi=4096, lengths=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "sinks", "append", "append_fp8", "read_fp8"])
    D, ps = rng.choice([64, 128]), rng.choice([8, 16, 16, 32])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    lengths = rng.randrange(1, 1 << 20)
    if op == "prefill":
        H_kv = rng.choice([1, 2, 4, 8])
        H_q = H_kv * rng.choice([1, 2, 4, 4, 8])
        B = _log(rng, 1, 24)
        hi = _log(rng, 1, 4096)
        ctx = _log(rng, 1, 28672)
        # the padded scores of all rows stay within a quarter of the longest listed chunk's
        most = 4096 * 32768 * 32 // 4 // (4 if dtype == "f32" else 1)
        while B * H_q * hi * (hi + ctx) > most:
            B, hi, ctx = max(1, B * 3 // 4), max(1, hi * 3 // 4), max(1, ctx * 3 // 4)
        win = rng.random() < 0.5
        return dict(op=op, dtype=dtype, B=B, H_q=H_q, H_kv=H_kv, D=D, ps=ps, lo=rng.randint(1, hi), hi=hi,
                    ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, window=_log(rng, 1, 4096) if win else 0,
                    sinks=rng.randint(0, 64) if win else 0, fused=rng.random() < 0.5, lengths=lengths)
    H_kv = rng.choice([2, 4, 8])
    if op == "sinks":
        ctx = _log(rng, 16, 32768)
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 64), H_q=H_kv * rng.choice([1, 2, 4, 8]), H_kv=H_kv, D=D,
                    ps=ps, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, window=_log(rng, 1, 4096),
                    sinks=rng.randint(0, 64), lengths=lengths)
    if op == "read_fp8":
        ctx = _log(rng, 1, 4096)
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 64), H_kv=H_kv, D=D, ps=ps, ctx_lo=rng.randint(0, ctx),
                    ctx_hi=ctx, lengths=lengths)
    hi = _log(rng, 1, 1024)
    return dict(op=op, dtype=dtype, B=_log(rng, 1, 32), H_kv=H_kv, D=D, ps=ps, lo=rng.randint(0, hi), hi=hi, ctx_lo=0,
                ctx_hi=_log(rng, 1, 4096), fused=rng.random() < 0.5, lengths=lengths)


def _sizes(case):
    """(new tokens, total tokens) of each sequence: of the case alone, so that its work is known."""
    r = np.random.default_rng(case["lengths"])
    ctx = r.integers(case["ctx_lo"], case["ctx_hi"] + 1, size=case["B"])
    if case["op"] in ("sinks", "read_fp8"):
        ctx[0] = max(1, ctx[0])  # a batch holds one token at least
        return np.zeros_like(ctx), ctx
    n = r.integers(case["lo"], case["hi"] + 1, size=case["B"])
    n[0] = max(1, n[0])
    return n, n + ctx


def _round_up(x, m):
    return (x + m - 1) // m * m


def prepare(case, seed):
    dev = "cuda"
    n, L = _sizes(case)
    B, ps, H_kv, D = case["B"], case["ps"], case["H_kv"], case["D"]
    r = np.random.default_rng(seed)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    pages = (L + ps - 1) // ps
    P = int(pages.sum()) + 8
    order = r.permutation(P)
    table = np.full((B, max(1, int(pages.max()))), P - 1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += int(pages[b])
    dt = _T[case["dtype"]]
    T = int(n.sum())
    s = dict(case=case, n_max=max(1, int(n.max())), L_max=max(1, int(L.max())), scale=D ** -0.5,
             table=torch.from_numpy(table).to(dev), lens=torch.from_numpy(L.astype(np.int32)).to(dev),
             indptr=torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(dev))

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    op = case["op"]
    if op in ("prefill", "sinks"):
        H_q = case["H_q"]
        s["k_pool"], s["v_pool"] = normal(P, ps, H_kv, D), normal(P, ps, H_kv, D)
        rows = T if op == "prefill" else B
        if op == "prefill" and case["fused"]:  # the query part of a fused projection's rows
            s["q"] = normal(rows, (H_q + 2 * H_kv), D)[:, :H_q]
        else:
            s["q"] = normal(rows, H_q, D)
        s["out"] = torch.zeros(rows, H_q, D, dtype=dt, device=dev)
        s["lse"] = torch.zeros(rows, H_q, dtype=torch.float32, device=dev)
        if own:
            import paged_kv_cache_46_gb300 as ts
            size = (ts.ts_paged_prefill_workspace_size(rows, B, H_q, H_kv, D) if op == "prefill"
                    else ts.ts_paged_decode_workspace_size(B, H_q, D))
            s["ws"] = ts.new_workspace(size)
        return s
    if op in ("append", "append_fp8"):
        # rows of a fused projection, or tensors of their own; activations have outlying channels
        x = normal(T, 2 * H_kv, D, dtype=torch.float32)
        x[:, :, ::37] *= 12.0
        x = x.to(dt)
        s["k_new"], s["v_new"] = x[:, :H_kv], x[:, H_kv:]
        if not case["fused"]:
            s["k_new"], s["v_new"] = s["k_new"].contiguous(), s["v_new"].contiguous()
    if op == "append":
        s["k_pool"], s["v_pool"] = normal(P, ps, H_kv, D), normal(P, ps, H_kv, D)
        return s
    for name in ("k", "v"):
        s[name + "_pool"] = normal(P, ps, H_kv, D, dtype=torch.float32).mul_(100).clamp_(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_scale"] = torch.rand(P, ps, H_kv, generator=g, device=dev) * 0.02 + 0.001
    if op == "read_fp8":
        # each sequence's rows begin at a whole page, so that the result can be taken as pages again
        starts = np.concatenate([[0], np.cumsum(_round_up(L, ps))]).astype(np.int32)
        s["indptr"] = torch.from_numpy(starts).to(dev)
        for name in ("k_out", "v_out"):
            s[name] = torch.zeros(int(starts[-1]), H_kv, D, dtype=dt, device=dev)
    return s


def _new_rows(s):
    """(chunk row of the batch, its row in the pool) of every new token."""
    ptr, ps = s["indptr"].long(), s["case"]["ps"]
    row = torch.arange(s["k_new"].shape[0], device=ptr.device)
    seq = torch.searchsorted(ptr, row, right=True) - 1
    pos = s["lens"].long()[seq] - ptr[seq + 1] + row
    return s["table"].long()[seq, pos // ps] * ps + pos % ps


def _gather(s, name, pos):
    """Cache rows of positions pos [B, K], in fp32, as [B, H_kv, K, D]."""
    ps, pool = s["case"]["ps"], s[name]
    row = s["table"].long().gather(1, pos // ps) * ps + pos % ps
    return pool.view(-1, *pool.shape[2:])[row].float().transpose(1, 2)


def _attend(s, q, k, v, seen):
    """Softmax attention of q [B, n, H_q, D] over k, v [B, H_kv, K, D] where seen [B, n, K]."""
    B, n, H_q, D = q.shape
    H_kv = k.shape[1]
    g = H_q // H_kv
    q = q.float().view(B, n, H_kv, g, D).permute(0, 2, 3, 1, 4).reshape(B, H_kv, g * n, D)
    x = torch.matmul(q * s["scale"], k.transpose(2, 3)).view(B, H_kv, g, n, -1)
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, H_kv, g * n, -1), v).view(B, H_kv, g, n, D)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + total.log()).squeeze(-1)
    return (o.permute(0, 3, 1, 2, 4).reshape(B, n, H_q, D), lse.permute(0, 3, 1, 2).reshape(B, n, H_q))


def _plain_prefill(s):
    c, ptr, lens = s["case"], s["indptr"].long(), s["lens"].long()
    n_max, L_max, q = s["n_max"], s["L_max"], s["q"]
    n = ptr[1:] - ptr[:-1]
    j = torch.arange(n_max, device=q.device)
    row = torch.minimum(ptr[:-1, None] + j, ptr[1:, None] - 1).clamp_(min=0)
    pos = torch.arange(L_max, device=q.device).expand(c["B"], -1)
    k, v = _gather(s, "k_pool", pos), _gather(s, "v_pool", pos)
    at = (lens - n)[:, None] + j  # position of each query
    seen = pos[:, None] <= at[:, :, None]
    if c["window"]:
        seen &= (pos[:, None] > at[:, :, None] - c["window"]) | (pos[:, None] < c["sinks"])
    o, lse = _attend(s, q[row], k, v, seen)
    real = j < n[:, None]
    s["out"].copy_(o[real])
    s["lse"].copy_(lse[real])
    return s["out"], s["lse"]


def _plain_sinks(s):
    c, lens = s["case"], s["lens"].long()[:, None]
    S, W = c["sinks"], c["window"]
    i = torch.arange(S + W, device=lens.device)
    pos = torch.where(lens > S + W, torch.where(i < S, i, lens - W - S + i), i)
    ok = pos < lens
    pos = torch.where(ok, pos, torch.zeros_like(pos))
    o, lse = _attend(s, s["q"][:, None], _gather(s, "k_pool", pos), _gather(s, "v_pool", pos), ok[:, None])
    s["out"].copy_(o[:, 0])
    s["lse"].copy_(lse[:, 0])
    return s["out"], s["lse"]


def _plain_append(s):
    row = _new_rows(s)
    for name in ("k", "v"):
        pool = s[name + "_pool"]
        pool.view(-1, *pool.shape[2:])[row] = s[name + "_new"]
    return s["k_pool"], s["v_pool"]


def _values(s):
    """A quantized cache as the values that its codes stand for, and their scales."""
    return (s["k_pool"].view(torch.float8_e4m3fn), s["v_pool"].view(torch.float8_e4m3fn), s["k_scale"], s["v_scale"])


def _plain_append_fp8(s):
    row = _new_rows(s)
    for name in ("k", "v"):
        pool, scales = s[name + "_pool"], s[name + "_scale"]
        x = s[name + "_new"].float()
        scale = x.abs().amax(-1).clamp(min=1e-10) / _E4M3_MAX
        code = (x / scale[..., None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn)
        pool.view(-1, *pool.shape[2:])[row] = code.view(torch.uint8)
        scales.view(-1, scales.shape[2])[row] = scale
    return _values(s)


def _plain_read_fp8(s):
    ptr, lens, ps = s["indptr"].long(), s["lens"].long(), s["case"]["ps"]
    out = torch.arange(s["k_out"].shape[0], device=ptr.device)
    seq = torch.searchsorted(ptr, out, right=True) - 1
    pos = out - ptr[seq]
    real = pos < lens[seq]
    row = torch.where(real, s["table"].long()[seq, pos // ps] * ps + pos % ps, torch.zeros_like(pos))
    for name in ("k", "v"):
        pool, scales = s[name + "_pool"], s[name + "_scale"]
        code = pool.view(-1, *pool.shape[2:])[row].view(torch.float8_e4m3fn).float()
        x = code * scales.view(-1, scales.shape[2])[row][..., None]
        to = s[name + "_out"]
        to.copy_(torch.where(real[:, None, None], x, to.float()))
    return s["k_out"], s["v_out"]


def _own(s):
    import paged_kv_cache_46_gb300 as ts
    c, op = s["case"], s["case"]["op"]
    if op == "prefill":
        ts.ts_paged_prefill_attn(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["indptr"], s["scale"],
                                 window=c["window"], sinks=c["sinks"], out=s["out"], lse=s["lse"], workspace=s["ws"])
        return s["out"], s["lse"]
    if op == "sinks":
        ts.ts_paged_decode_sink_attn(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["scale"],
                                     c["window"], c["sinks"], out=s["out"], lse=s["lse"], workspace=s["ws"])
        return s["out"], s["lse"]
    if op == "append":
        ts.ts_kv_append_chunk(s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["indptr"])
        return s["k_pool"], s["v_pool"]
    if op == "append_fp8":
        ts.ts_kv_append_chunk_fp8(s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                  s["table"], s["lens"], s["indptr"])
        return _values(s)
    ts.ts_kv_read_fp8(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"], s["lens"], s["indptr"],
                      s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


_PLAIN = dict(prefill=_plain_prefill, sinks=_plain_sinks, append=_plain_append, append_fp8=_plain_append_fp8,
              read_fp8=_plain_read_fp8)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


def _pairs(case, n, L):
    """(visible query-key pairs, cache rows that some query sees), over the batch."""
    W, S = case["window"], case["sinks"]
    pairs = rows = 0
    for nb, Lb in zip(n.tolist(), L.tolist()):
        if Lb == 0:
            continue
        at = np.arange(Lb - nb, Lb, dtype=np.int64) if case["op"] == "prefill" else np.array([Lb - 1])
        if W == 0:
            pairs += int((at + 1).sum())
            rows += Lb
        else:
            pairs += int((np.minimum(at + 1, W) + np.minimum(S, np.maximum(0, at + 1 - W))).sum())
            first = max(0, int(at[0]) + 1 - W) if at.size else Lb
            rows += Lb - first + min(S, first)
    return pairs, rows


def work(case):
    n, L = _sizes(case)
    es = 2 if case["dtype"] == "bf16" else 4
    H_kv, D, op = case["H_kv"], case["D"], case["op"]
    T = int(n.sum())
    if op in ("prefill", "sinks"):
        H_q = case["H_q"]
        rows = T if op == "prefill" else case["B"]
        pairs, seen = _pairs(case, n, L)
        return {"bytes": rows * H_q * (2 * D * es + 4) + seen * 2 * H_kv * D * es, "flops": 4 * D * H_q * pairs}
    if op == "append":
        return {"bytes": T * 2 * H_kv * D * 2 * es, "flops": 0}
    if op == "append_fp8":  # the values in; codes and scales out; maximum, quotient and rounding of each value
        return {"bytes": T * 2 * H_kv * (D * es + D + 4), "flops": T * 2 * H_kv * D * 3}
    tokens = int(L.sum())
    return {"bytes": tokens * 2 * H_kv * (D + 4 + D * es), "flops": tokens * 2 * H_kv * D}


def _cache_rows(s, name, b, positions):
    """Cache rows of sequence b at `positions`, as stored."""
    pool, ps = s[name], s["case"]["ps"]
    page = s["table"][b].long()[positions // ps]
    return pool[page, positions % ps]


def exact(case, seed):
    s = prepare(case, seed)
    n, L = _sizes(case)
    op, ps, dev = case["op"], case["ps"], s["table"].device
    if op in ("prefill", "sinks"):
        H_kv, D = case["H_kv"], case["D"]
        g = case["H_q"] // H_kv
        W, S = case["window"], case["sinks"]
        outs, lses = [], []
        at = 0
        for b in range(case["B"]):
            nb, Lb = (int(n[b]), int(L[b])) if op == "prefill" else (1, int(L[b]))
            q = s["q"][at:at + nb].double()
            at += nb
            o = torch.zeros(nb, H_kv * g, D, dtype=torch.float64, device=dev)
            lse = torch.full((nb, H_kv * g), float("-inf"), dtype=torch.float64, device=dev)
            if nb and Lb:
                t = torch.arange(Lb, device=dev)
                mine = torch.arange(Lb - nb, Lb, device=dev)
                hidden = t[None] > mine[:, None]
                if W:
                    hidden |= (t[None] <= mine[:, None] - W) & (t[None] >= S)
                for h in range(H_kv):
                    k = _cache_rows(s, "k_pool", b, t)[:, h].double()
                    v = _cache_rows(s, "v_pool", b, t)[:, h].double()
                    for i in range(h * g, (h + 1) * g):
                        x = (q[:, i] @ k.T) * s["scale"]
                        x[hidden] = float("-inf")
                        lse[:, i] = torch.logsumexp(x, 1)
                        o[:, i] = torch.exp(x - lse[:, i:i + 1]) @ v
            outs.append(o)
            lses.append(lse)
        return torch.cat(outs), torch.cat(lses)
    if op == "read_fp8":
        made = []
        for name in ("k", "v"):
            to = s[name + "_out"].double()
            for b in range(case["B"]):
                t, at = torch.arange(int(L[b]), device=dev), int(s["indptr"][b])
                code = _cache_rows(s, name + "_pool", b, t).view(torch.float8_e4m3fn).double()
                to[at:at + int(L[b])] = code * _cache_rows(s, name + "_scale", b, t).double()[..., None]
            made.append(to)
        return tuple(made)
    pools = {}
    for name in ("k", "v"):
        x = s[name + "_new"].double()
        pool = s[name + "_pool"]
        pool = pool.double() if op == "append" else pool.view(torch.float8_e4m3fn).double()
        if op == "append_fp8":
            step = x.abs().max(-1).values.clamp(min=1e-10) / 448.0
            scales = s[name + "_scale"].double()
            x = x / step[..., None]  # before the rounding to 8 bits
        at = 0
        for b in range(case["B"]):
            t = torch.arange(int(L[b] - n[b]), int(L[b]), device=dev)
            page = s["table"][b].long()[t // ps]
            pool[page, t % ps] = x[at:at + int(n[b])]
            if op == "append_fp8":
                scales[page, t % ps] = step[at:at + int(n[b])]
                pools[name + "_scale"] = scales
            at += int(n[b])
        pools[name] = pool
    if op == "append":
        return pools["k"], pools["v"]
    return pools["k"], pools["v"], pools["k_scale"], pools["v_scale"]
