"""Operators of a long-context serving step over a paged cache, as measurable cases.

Six operators: normalising and rotating the queries and keys of a ragged batch
of chunks while K and V are written into their pages (`rope`), the bounds of
each page's keys (`bounds`), choosing the pages whose bounds promise most for a
query (`select`), decode attention over the chosen pages (`sparse`), forking
sequences (`fork`), and moving the pages in use to the front of the pool
(`compact`).

`run` computes a case in elementary torch operations where `own` is false, and
through the library's entry points where it is true.
"""

import math

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_STEP = 1.0 / 127.0


def listed():
    return [
        # one user's next token at the Llama-3-8B layer's shape: latency counts
        dict(name="rope_one", op="rope", dtype="bf16", B=1, H_q=32, H_kv=8, D=128, ps=16, lo=1, hi=1, ctx_lo=1000,
             ctx_hi=1000, norm=True, rot=128, interleaved=False, fused=True, lengths=1),
        # a full step of a prefill server: 32 chunks, rows of a fused projection
        dict(name="rope_batch", op="rope", dtype="bf16", B=32, H_q=32, H_kv=8, D=128, ps=16, lo=1, hi=1024, ctx_lo=0,
             ctx_hi=4096, norm=True, rot=128, interleaved=False, fused=True, lengths=2),
        # after a decode step of 64 long conversations: the page of each one's new token
        dict(name="bounds_step", op="bounds", dtype="bf16", B=64, H_kv=8, D=128, ps=16, lo=1, hi=1, ctx_lo=4096,
             ctx_hi=32767, lengths=3),
        # after a prefill step of 32 chunks
        dict(name="bounds_batch", op="bounds", dtype="bf16", B=32, H_kv=8, D=128, ps=16, lo=1, hi=1024, ctx_lo=0,
             ctx_hi=4096, lengths=4),
        # one user over a context of 131,072 tokens: latency counts
        dict(name="select_one", op="select", dtype="bf16", B=1, q_len=1, H_q=32, H_kv=8, D=128, ps=16, ctx_lo=131072,
             ctx_hi=131072, pages=128, first=1, last=2, lengths=5),
        # 64 long conversations, 2048 tokens of each kept
        dict(name="select_batch", op="select", dtype="bf16", B=64, q_len=1, H_q=32, H_kv=8, D=128, ps=16, ctx_lo=4096,
             ctx_hi=32768, pages=128, first=1, last=2, lengths=6),
        # one streaming user, a small fp32 model: latency counts
        dict(name="sparse_one", op="sparse", dtype="f32", B=1, q_len=1, H_q=8, H_kv=2, D=64, ps=16, ctx_lo=20001,
             ctx_hi=20001, pages=32, lengths=7),
        # the attention of select_batch's step
        dict(name="sparse_batch", op="sparse", dtype="bf16", B=64, q_len=1, H_q=32, H_kv=8, D=128, ps=16, ctx_lo=4096,
             ctx_hi=32768, pages=128, lengths=8),
        # one conversation gets a second continuation, one layer's K and V
        dict(name="fork_one", op="fork", cache="bf16", layers=1, parents=1, each=1, H_kv=8, D=128, ps=16, ctx_lo=999,
             ctx_hi=999, lengths=9),
        # 16 prompts sampled four times each: K, V and page bounds of 12 layers
        dict(name="fork_batch", op="fork", cache="bounds", layers=12, parents=16, each=4, H_kv=8, D=128, ps=16,
             ctx_lo=100, ctx_hi=1000, lengths=10),
        # a small quantized cache after some conversations ended
        dict(name="compact_one", op="compact", cache="fp8", layers=1, B=4, gone=4, H_kv=2, D=64, ps=16, ctx_lo=50,
             ctx_hi=500, lengths=11),
        # half of 64 conversations ended: K, V and page bounds of 12 layers
        dict(name="compact_batch", op="compact", cache="bounds", layers=12, B=32, gone=32, H_kv=8, D=128, ps=16,
             ctx_lo=100, ctx_hi=1000, lengths=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "bounds", "select", "select", "sparse", "sparse", "fork", "compact"])
    D, ps = rng.choice([64, 128]), rng.choice([8, 16, 16, 32])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    lengths = rng.randrange(1, 1 << 20)
    H_kv = rng.choice([1, 2, 4, 8])
    if op in ("rope", "bounds"):
        hi = _log(rng, 1, 1024)
        case = dict(op=op, dtype=dtype, B=_log(rng, 1, 32), H_kv=H_kv, D=D, ps=ps, lo=rng.randint(0, hi), hi=hi,
                    ctx_lo=0, ctx_hi=_log(rng, 1, 4096), lengths=lengths)
        if dtype == "f32":
            case["B"] = max(1, case["B"] // 2)
        if op == "rope":
            case.update(H_q=H_kv * rng.choice([1, 2, 4]), norm=rng.random() < 0.5,
                        rot=rng.choice([D, D, D, D // 2, D // 4]), interleaved=rng.random() < 0.3,
                        fused=rng.random() < 0.5)
        return case
    if op in ("select", "sparse"):
        q_len = rng.choice([1, 1, 1, 2, 4])
        ctx = _log(rng, 16, 32768)
        case = dict(op=op, dtype=dtype, B=max(1, _log(rng, 1, 64) // q_len), q_len=q_len,
                    H_q=H_kv * rng.choice([1, 2, 4, 8]), H_kv=H_kv, D=D, ps=ps, ctx_lo=rng.randint(q_len, ctx),
                    ctx_hi=ctx, pages=_log(rng, 4, 128 * 16 // ps), lengths=lengths)
        if dtype == "f32":
            case["B"] = max(1, case["B"] // 2)
        if op == "select":
            case["H_q"] = H_kv * rng.choice([1, 2, 4])
            if ps == 8:
                case["B"] = max(1, case["B"] // 2)
            # more pages than are chosen in one sequence at least
            case["ctx_hi"] = max(ctx, 16 * ps)
            case["pages"] = _log(rng, 5, min(128 * 16 // ps, case["ctx_hi"] // (2 * ps)))
            case["first"] = rng.randint(0, 1)
            case["last"] = rng.randint(1, 3)
        return case
    case = dict(op=op, cache=rng.choice(["bf16", "f32", "fp8", "bounds"]), layers=_log(rng, 1, 8), H_kv=H_kv, D=D,
                ps=ps, ctx_lo=rng.randint(1, 100), ctx_hi=rng.randint(100, 1000), lengths=lengths)
    if op == "fork":
        case.update(parents=_log(rng, 1, 16), each=rng.randint(1, 4))
    else:
        case.update(B=_log(rng, 1, 32), gone=_log(rng, 1, 32))
    return case


def _sizes(case):
    """(new tokens, total tokens) of each sequence: of the case alone, so that its work is known."""
    r = np.random.default_rng(case["lengths"])
    if case["op"] == "fork":
        rows = case["parents"]
    elif case["op"] == "compact":
        rows = case["B"] + case["gone"]
    else:
        rows = case["B"]
    ctx = r.integers(case["ctx_lo"], case["ctx_hi"] + 1, size=rows)
    if case["op"] == "select":
        ctx[0] = case["ctx_hi"]
    if case["op"] not in ("rope", "bounds"):
        return np.zeros_like(ctx), ctx
    n = r.integers(case["lo"], case["hi"] + 1, size=rows)
    n[0] = max(1, n[0])
    return n, n + ctx


def _buffers(case):
    """(type, elements of a page) of each buffer of a layer's cache."""
    H, D, ps = case["H_kv"], case["D"], case["ps"]
    kv = ps * H * D
    return {"bf16": [("bf16", kv)] * 2, "f32": [("f32", kv)] * 2, "fp8": [("e4m3", kv)] * 2 + [("f32", ps * H)] * 2,
            "bounds": [("bf16", kv)] * 2 + [("i8", 2 * H * D), ("f32", H)]}[case["cache"]]


_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1, "i8": 1}


def prepare(case, seed):
    dev = "cuda"
    n, L = _sizes(case)
    op, ps, H_kv, D = case["op"], case["ps"], case["H_kv"], case["D"]
    r = np.random.default_rng(seed)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    pages = (L + ps - 1) // ps
    children = case["parents"] * case["each"] if op == "fork" else 0
    P = int(pages.sum()) + children + 8
    order = r.permutation(P)
    table = np.full((len(L) + children, max(1, int(pages.max()))), order[-1], dtype=np.int32)
    at = 0
    for b in range(len(L)):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += int(pages[b])

    def i32(x):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)

    s = dict(case=case, L_max=max(1, int(L.max())), scale=D ** -0.5)

    def normal(*shape, dtype):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    if op in ("fork", "compact"):
        s["buffers"] = []
        for _ in range(case["layers"]):
            for kind, size in _buffers(case):
                if kind == "e4m3":
                    x = normal(P, size, dtype=torch.float32).mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
                elif kind == "i8":
                    x = torch.randint(-127, 128, (P, size), generator=g, device=dev, dtype=torch.int8)
                else:
                    x = normal(P, size, dtype=_T[kind])
                s["buffers"].append(x)
        if own:
            import paged_kv_cache_46_gb300 as ts
        if op == "fork":
            s["parents"] = i32(np.repeat(np.arange(len(L)), case["each"]))
            s["children"] = i32(len(L) + r.permutation(children))
            s["fresh"] = i32(order[at:at + children])
            s["lens"] = i32(np.concatenate([L, np.zeros(children, dtype=L.dtype)]))
            s["table"] = i32(table)
            if own:
                s["plan"] = ts.kv_buffers(s["buffers"])
            return s
        stay = np.sort(r.permutation(len(L))[:case["B"]])  # the rest ended
        s["table"], s["lens"] = i32(table[stay]), i32(L[stay])
        s["table_out"] = torch.empty_like(s["table"])
        if own:
            s["plan"] = ts.kv_buffers(s["buffers"])
            s["used"] = torch.zeros(1, dtype=torch.int32, device=dev)
            s["page_map"] = torch.zeros(P, dtype=torch.int32, device=dev)
            s["ws"] = ts.new_workspace(ts.ts_kv_compact_workspace_size(P))
        return s

    dt = _T[case["dtype"]]
    s["table"], s["lens"] = i32(table), i32(L)
    if op in ("rope", "bounds"):
        s["indptr"] = i32(np.concatenate([[0], np.cumsum(n)]))
        s["T"] = T = int(n.sum())
    if op == "rope":
        H_q = case["H_q"]
        rows = normal(T, H_q + 2 * H_kv, D, dtype=torch.float32)
        rows[:, :, ::37] *= 12.0  # activations have outlying channels
        rows = rows.to(dt)
        s["q"], s["k_new"], s["v_new"] = rows[:, :H_q], rows[:, H_q:H_q + H_kv], rows[:, H_q + H_kv:]
        if not case["fused"]:
            s["q"], s["k_new"], s["v_new"] = (x.contiguous() for x in (s["q"], s["k_new"], s["v_new"]))
        s["k_pool"], s["v_pool"] = normal(P, ps, H_kv, D, dtype=dt), normal(P, ps, H_kv, D, dtype=dt)
        half = case["rot"] // 2
        s["inv_freq"] = torch.from_numpy(500000.0 ** (-np.arange(half) / half)).to(torch.float32).to(dev)
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = ((1 + 0.2 * normal(D, dtype=torch.float32)).to(dt) for _ in "qk")
        s["q_out"] = torch.zeros(T, H_q, D, dtype=dt, device=dev)
        return s
    if op == "bounds":
        s["k_pool"] = normal(P, ps, H_kv, D, dtype=dt)
        s["bounds"] = torch.randint(-127, 128, (P, H_kv, 2, D), generator=g, device=dev, dtype=torch.int8)
        s["bound_scale"] = torch.rand(P, H_kv, generator=g, device=dev) * 0.02 + 0.01
        return s
    H_q, q_len = case["H_q"], case["q_len"]
    q = normal(len(L), q_len, H_q, D, dtype=dt)
    s["q"] = q if q_len > 1 else q[:, 0].contiguous()
    if op == "select":
        # the keys of a page lie around a centre of its own
        middle = normal(P, H_kv, D, dtype=torch.float32)
        reach = normal(P, H_kv, D, dtype=torch.float32).abs() + 0.3
        s["bounds"], s["bound_scale"] = _quantize_bounds(middle + reach, middle - reach)
        shape = (len(L), q_len, H_kv, case["pages"]) if q_len > 1 else (len(L), H_kv, case["pages"])
        s["page_idx"] = torch.zeros(shape, dtype=torch.int32, device=dev)
        if own:
            import paged_kv_cache_46_gb300 as ts
            s["ws"] = ts.new_workspace(ts.ts_select_pages_workspace_size(len(L), q_len, H_kv, table.shape[1]))
        return s
    s["k_pool"], s["v_pool"] = normal(P, ps, H_kv, D, dtype=dt), normal(P, ps, H_kv, D, dtype=dt)
    # lists as a selection makes them: ascending, the first and the last page among them
    K, N = case["pages"], table.shape[1]
    have = ((s["lens"][:, None] - q_len + torch.arange(q_len, device=dev)) // ps + 1)[:, :, None, None]
    i = torch.arange(N, device=dev)
    rank = torch.rand(len(L), q_len, H_kv, N, generator=g, device=dev)
    rank = torch.where((i == 0) | (i == have - 1), 2.0, rank).masked_fill(i >= have, -1.0)
    rank, idx = rank.topk(min(K, N), dim=-1)
    idx = torch.where(rank >= 0, idx, N).sort(-1).values
    idx = torch.cat([idx, idx.new_full((*idx.shape[:3], K - idx.shape[3]), N)], -1)
    idx = torch.where(idx < N, idx, -1).to(torch.int32)
    s["page_idx"] = idx if q_len > 1 else idx[:, 0].contiguous()
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(s["q"].shape[:-1], dtype=torch.float32, device=dev)
    if own:
        import paged_kv_cache_46_gb300 as ts
        s["ws"] = ts.new_workspace(ts.ts_paged_decode_sparse_workspace_size(len(L), q_len, H_q, H_kv, D, ps, K))
    return s


def _new_rows(s):
    """(position, row in the pool) of every new token."""
    ptr, ps = s["indptr"].long(), s["case"]["ps"]
    row = torch.arange(s["T"], device=ptr.device)
    seq = torch.searchsorted(ptr, row, right=True) - 1
    pos = s["lens"].long()[seq] - ptr[seq + 1] + row
    return pos, s["table"].long()[seq, pos // ps] * ps + pos % ps


def _rotate(s, x, weight, cos, sin):
    """x [T, H, D], normalised where there is a weight, its first columns rotated; in fp32."""
    x, rot = x.float(), s["case"]["rot"]
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    else:
        x = x.clone()
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    new_a, new_b = a * cos - b * sin, b * cos + a * sin
    a.copy_(new_a)
    b.copy_(new_b)
    return x


def _plain_rope(s):
    pos, row = _new_rows(s)
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    s["q_out"].copy_(_rotate(s, s["q"], s["q_weight"], cos, sin))
    k = _rotate(s, s["k_new"], s["k_weight"], cos, sin)
    for name, x in (("k_pool", k), ("v_pool", s["v_new"])):
        pool = s[name]
        pool.view(-1, *pool.shape[2:])[row] = x.to(pool.dtype)
    return s["q_out"], s["k_pool"], s["v_pool"]


def _quantize_bounds(top, low):
    """Codes [P, H_kv, 2, D] and scale [P, H_kv] of channel bounds [P, H_kv, D], rounded outward."""
    scale = torch.maximum(top.abs(), low.abs()).amax(-1).clamp(min=1e-10) * _STEP
    top = (top / scale[..., None]).ceil().clamp(-127, 127)
    low = (low / scale[..., None]).floor().clamp(-127, 127)
    return torch.stack([top, low], 2).to(torch.int8), scale


def _plain_bounds(s):
    lens, ps = s["lens"].long(), s["case"]["ps"]
    n = s["indptr"].long().diff()
    N = s["table"].shape[1]
    slot = torch.arange(N, device=lens.device)
    # pages that hold a new token
    touched = (slot >= ((lens - n) // ps)[:, None]) & (slot * ps < lens[:, None]) & (n > 0)[:, None]
    seq, slot = touched.nonzero(as_tuple=True)
    page = s["table"].long()[seq, slot]
    real = (slot[:, None] * ps + torch.arange(ps, device=lens.device) < lens[seq, None])[:, :, None, None]
    k = s["k_pool"][page].float()
    top = torch.where(real, k, float("-inf")).amax(1)
    low = torch.where(real, k, float("inf")).amin(1)
    s["bounds"][page], s["bound_scale"][page] = _quantize_bounds(top, low)
    return s["bounds"], s["bound_scale"]


def _plain_select(s):
    c = s["case"]
    ps, H_kv, D, K, first, last = c["ps"], c["H_kv"], c["D"], c["pages"], c["first"], c["last"]
    q_len, N = c["q_len"], s["table"].shape[1]
    q = s["q"].float().view(c["B"], q_len, H_kv, -1, D)
    q_scale = q.abs().amax(-1).clamp(min=1e-10) * _STEP
    code = (q / q_scale[..., None]).round().clamp(-127, 127)
    have = (s["lens"].long()[:, None] - q_len + torch.arange(q_len, device=q.device)) // ps + 1  # pages of each query
    i = torch.arange(N, device=q.device)
    at = s["table"].long()
    bounds, scale = s["bounds"], s["bound_scale"]
    rank = torch.empty(c["B"], q_len, H_kv, N, device=q.device)
    step = max(1, (1 << 28) // (N * H_kv * 2 * D))
    for b in range(0, c["B"], step):  # the bounds of some sequences at a time
        mine = at[b:b + step]
        B = mine.shape[0]
        lim = bounds[mine].permute(0, 2, 3, 4, 1).float()  # [B, H_kv, 2, D, N]
        both = torch.stack([code[b:b + step].clamp(min=0), code[b:b + step].clamp(max=0)], -2)  # .., 2, D
        both = both.permute(0, 2, 1, 3, 4, 5).reshape(B, H_kv, -1, 2 * D)
        dot = torch.matmul(both, lim.reshape(B, H_kv, 2 * D, N)).view(B, H_kv, q_len, -1, N)  # whole numbers
        score = dot * q_scale[b:b + step].permute(0, 2, 1, 3)[..., None]
        score = score * scale[mine].permute(0, 2, 1)[:, :, None, None]
        rank[b:b + step] = score.amax(3).transpose(1, 2)
    have = have[:, :, None, None]
    rank = torch.where((i < first) | (i >= have - last), float("inf"), rank).masked_fill(i >= have, float("-inf"))
    idx = rank.sort(dim=-1, descending=True, stable=True).indices[..., :K]
    idx = torch.where(torch.arange(idx.shape[-1], device=q.device) < have, idx, N).sort(-1).values
    s["page_idx"].fill_(-1)
    s["page_idx"].view(c["B"], q_len, H_kv, K)[..., :idx.shape[-1]] = torch.where(idx < N, idx, -1)
    return s["page_idx"]


def _plain_sparse(s):
    c = s["case"]
    ps, H_kv, D, q_len, K = c["ps"], c["H_kv"], c["D"], c["q_len"], c["pages"]
    B = c["B"]
    q = s["q"].float().view(B, q_len, H_kv, -1, D)
    idx = s["page_idx"].long().view(B, q_len, H_kv, K)
    at = s["lens"].long()[:, None] - q_len + torch.arange(q_len, device=q.device)  # position of each query
    out, lse = s["out"].view(q.shape), s["lse"].view(q.shape[:-1])
    t = torch.arange(ps, device=q.device)
    for j in range(q_len):
        page = s["table"].long()[torch.arange(B, device=q.device)[:, None, None], idx[:, j].clamp(min=0)]
        head = torch.arange(H_kv, device=q.device)[:, None]
        seen = (idx[:, j, :, :, None] >= 0) & (idx[:, j, :, :, None] * ps + t <= at[:, j, None, None, None])
        seen = seen.view(B, H_kv, 1, K * ps)
        k = s["k_pool"].transpose(1, 2)[page, head].view(B, H_kv, K * ps, D).float()
        x = torch.matmul(q[:, j] * s["scale"], k.transpose(2, 3)).masked_fill(~seen, float("-inf"))
        m = x.amax(-1, keepdim=True)
        m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
        x = (x - m).exp()
        total = x.sum(-1, keepdim=True)
        v = s["v_pool"].transpose(1, 2)[page, head].view(B, H_kv, K * ps, D).float()
        out[:, j] = torch.matmul(x, v) / torch.where(total > 0, total, torch.ones_like(total))
        lse[:, j] = (m + total.log()).squeeze(-1)
    return s["out"], s["lse"]


def _plain_fork(s):
    ps, table, lens = s["case"]["ps"], s["table"], s["lens"]
    parents, children, fresh = s["parents"].long(), s["children"].long(), s["fresh"].long()
    L = lens[parents].long()
    slots = (L + ps - 1) // ps
    slot = torch.arange(table.shape[1], device=L.device)
    row = torch.where(slot < slots[:, None], table[parents], table[children])
    cut = (L % ps != 0).nonzero(as_tuple=True)[0]
    source = row[cut, slots[cut] - 1].long()
    for x in s["buffers"]:
        x = x.view(torch.uint8)
        x[fresh[cut]] = x[source]
    row[cut, slots[cut] - 1] = s["fresh"][cut]
    table[children] = row
    lens[children] = L.to(torch.int32)
    return s["buffers"], table, lens


def _plain_compact(s):
    ps, table = s["case"]["ps"], s["table"]
    P = s["buffers"][0].shape[0]
    slot = torch.arange(table.shape[1], device=table.device)
    live = slot * ps < s["lens"].long()[:, None]
    used = torch.zeros(P, dtype=torch.bool, device=table.device)
    used[table[live].long()] = True
    count = used.sum()
    page = torch.arange(P, device=table.device)
    source = (used & (page >= count)).nonzero(as_tuple=True)[0]
    target = (~used & (page < count)).nonzero(as_tuple=True)[0]
    page_map = torch.where(used, page, -1)
    page_map[source] = target
    for x in s["buffers"]:
        x = x.view(torch.uint8)
        x[target] = x[source]
    s["table_out"].copy_(torch.where(live, page_map[table.long()], table.long()))
    return s["buffers"], s["table_out"], page_map.to(torch.int32), count.to(torch.int32).view(1)


def _own(s):
    import paged_kv_cache_46_gb300 as ts
    c, op = s["case"], s["case"]["op"]
    if op == "rope":
        ts.ts_kv_append_chunk_rope(s["q"], s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], s["table"], s["lens"],
                                   s["indptr"], s["inv_freq"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                   eps=1e-6, interleaved=c["interleaved"], q_out=s["q_out"])
        return s["q_out"], s["k_pool"], s["v_pool"]
    if op == "bounds":
        ts.ts_kv_page_bounds(s["k_pool"], s["bounds"], s["bound_scale"], s["table"], s["lens"], s["indptr"], s["T"])
        return s["bounds"], s["bound_scale"]
    if op == "select":
        return ts.ts_select_pages(s["q"], s["bounds"], s["bound_scale"], s["table"], s["lens"], c["ps"], c["pages"],
                                  first=c["first"], last=c["last"], page_idx=s["page_idx"], workspace=s["ws"])
    if op == "sparse":
        ts.ts_paged_decode_sparse_attn(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["page_idx"],
                                       s["scale"], out=s["out"], lse=s["lse"], workspace=s["ws"])
        return s["out"], s["lse"]
    if op == "fork":
        ts.ts_kv_fork(s["plan"], s["table"], s["lens"], s["parents"], s["children"], s["fresh"], c["ps"])
        return s["buffers"], s["table"], s["lens"]
    ts.ts_kv_compact(s["plan"], s["table"], s["lens"], c["ps"], table_out=s["table_out"], page_map=s["page_map"],
                     used=s["used"], workspace=s["ws"])
    return s["buffers"], s["table_out"], s["page_map"], s["used"]


_PLAIN = dict(rope=_plain_rope, bounds=_plain_bounds, select=_plain_select, sparse=_plain_sparse, fork=_plain_fork,
              compact=_plain_compact)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


def work(case):
    n, L = _sizes(case)
    op, ps, H_kv, D = case["op"], case["ps"], case["H_kv"], case["D"]
    pages = (L + ps - 1) // ps
    if op in ("fork", "compact"):
        size = case["layers"] * sum(_BYTES[kind] * elements for kind, elements in _buffers(case))
        if op == "fork":
            copied, moved = int((L % ps != 0).sum()), int(pages.sum())
            return {"bytes": case["each"] * (copied * 2 * size + moved * 8), "flops": 0}
        # of `used` pages spread over the pool, those beyond its first `used` move
        held = int(pages.sum()) * case["B"] // (case["B"] + case["gone"])
        P = int(pages.sum()) + 8
        return {"bytes": held * (P - held) // P * 2 * size + held * 8 + P * 4, "flops": 0}
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "rope":  # mean of squares, scale and weight, rotation
        T, H_q = int(n.sum()), case["H_q"]
        return {"bytes": T * (H_q + 2 * H_kv) * D * 2 * es, "flops": T * (H_q + H_kv) * D * 7}
    if op == "bounds":
        touched = np.where(n > 0, (L + ps - 1) // ps - (L - n) // ps, 0)
        rows = np.where(n > 0, L - (L - n) // ps * ps, 0)
        return {"bytes": int(rows.sum()) * H_kv * D * es + int(touched.sum()) * H_kv * (2 * D + 4),
                "flops": int(rows.sum()) * H_kv * D * 2}
    H_q, q_len, K = case["H_q"], case["q_len"], case["pages"]
    data = flops = 0
    for Lb in L.tolist():
        at = Lb - q_len + np.arange(q_len)
        have = at // ps + 1
        if op == "select":
            data += int(have.max()) * H_kv * (2 * D + 4) if have.max() > K else 0
            flops += int(np.where(have > K, have, 0).sum()) * H_q * 2 * D
        else:
            tokens = np.where(have <= K, at + 1, (K - 1) * ps + at % ps + 1)
            data += min(int(tokens.sum()), Lb) * 2 * H_kv * D * es
            flops += int(tokens.sum()) * H_q * 4 * D
    rows = len(L) * q_len
    data += rows * H_q * D * es + rows * H_kv * K * 4
    if op == "sparse":
        data += rows * H_q * (D * es + 4)
    return {"bytes": data, "flops": flops}


def exact(case, seed):
    op = case["op"]
    if op in ("select", "fork", "compact"):  # whole numbers, and copies
        return None
    s = prepare(case, seed)
    n, L = _sizes(case)
    ps, H_kv, D = case["ps"], case["H_kv"], case["D"]
    if op == "rope":
        dev, rot = s["q"].device, case["rot"]
        made = {"q": s["q_out"].double(), "k_pool": s["k_pool"].double(), "v_pool": s["v_pool"].double()}
        at = 0
        for b in range(case["B"]):
            rows = slice(at, at + int(n[b]))
            at += int(n[b])
            t = torch.arange(int(L[b] - n[b]), int(L[b]), device=dev)
            turn = torch.polar(torch.ones(1, dtype=torch.float64, device=dev),
                               torch.outer(t.double(), s["inv_freq"].double()))[:, None]
            done = []
            for x, w in ((s["q"][rows], s["q_weight"]), (s["k_new"][rows], s["k_weight"])):
                x = x.double()
                if w is not None:
                    x = x / (x.square().sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
                head, tail = x[..., :rot], x[..., rot:]
                if case["interleaved"]:
                    z = torch.complex(head[..., 0::2].contiguous(), head[..., 1::2].contiguous()) * turn
                    head = torch.stack([z.real, z.imag], -1).flatten(-2)
                else:
                    z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
                    head = torch.cat([z.real, z.imag], -1)
                done.append(torch.cat([head, tail], -1))
            made["q"][rows] = done[0]
            page = s["table"][b].long()[t // ps]
            made["k_pool"][page, t % ps] = done[1]
            made["v_pool"][page, t % ps] = s["v_new"][rows].double()
        return made["q"], made["k_pool"], made["v_pool"]
    if op == "bounds":
        scale = s["bound_scale"].double()
        for b in range(case["B"]):
            for slot in range(int(L[b] - n[b]) // ps, int(L[b] + ps - 1) // ps if n[b] else 0):
                page = int(s["table"][b, slot])
                keys = s["k_pool"][page, :int(L[b]) - slot * ps].double()
                scale[page] = keys.abs().amax((0, 2)).clamp(min=1e-10) / 127
        return None, scale
    H_q, q_len = case["H_q"], case["q_len"]
    g = H_q // H_kv
    idx = s["page_idx"].view(case["B"], q_len, H_kv, -1).cpu().numpy()
    q = s["q"].view(case["B"], q_len, H_q, D)
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:-1], dtype=torch.float64, device=q.device)
    for b in range(case["B"]):
        for j in range(q_len):
            for h in range(H_kv):
                listed_pages = idx[b, j, h][idx[b, j, h] >= 0]
                t = (listed_pages[:, None].astype(np.int64) * ps + np.arange(ps)).ravel()
                t = torch.from_numpy(t[t <= int(L[b]) - q_len + j]).to(q.device)
                page = s["table"][b].long()[t // ps]
                k, v = s["k_pool"][page, t % ps, h].double(), s["v_pool"][page, t % ps, h].double()
                x = q[b, j, h * g:(h + 1) * g].double() @ k.T * s["scale"]
                lse[b, j, h * g:(h + 1) * g] = torch.logsumexp(x, 1)
                out[b, j, h * g:(h + 1) * g] = torch.softmax(x, 1) @ v
    return out.view(s["q"].shape), lse.view(s["lse"].shape)
