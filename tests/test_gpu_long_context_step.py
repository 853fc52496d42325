"""The long-context calls together, as a server uses them: a prompt is appended, its
page bounds made, decode steps select and attend, a conversation forks, others end,
the pool is compacted, and decoding goes on. Each step is held to the oracle on the
cache as the device holds it."""

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_46_gb300 as ts
from chunk_cases import check_attention
from long_context_cases import DEV, DTYPES, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_46_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class Server:
    """One layer's cache, `rows` sequences at most, pages handed out from a list on the host."""

    def __init__(self, dtype, H_q, H_kv, D, ps, P, rows, slots):
        self.dt, self.H_q, self.H_kv, self.D, self.ps, self.P = DTYPES[dtype], H_q, H_kv, D, ps, P
        self.dtype = dtype
        nan = float("nan")
        self.k, self.v = (torch.full((P, ps, H_kv, D), nan, dtype=self.dt, device=DEV) for _ in "kv")
        self.bounds = torch.zeros(P, H_kv, 2, D, dtype=torch.int8, device=DEV)
        self.scale = torch.full((P, H_kv), nan, device=DEV)
        self.plan = ts.kv_buffers([self.k, self.v, self.bounds, self.scale])
        self.table = np.zeros((rows, slots), dtype=np.int32)
        self.lens = np.zeros(rows, dtype=np.int32)
        rng = np.random.default_rng(5)
        self.free = list(rng.permutation(P))
        self.gen = torch.Generator(device=DEV).manual_seed(5)
        self.freq = torch.from_numpy(10000.0 ** (-np.arange(D // 2) / (D // 2))).float().to(DEV)
        self.weight = (1 + 0.2 * self.normal(D).float()).to(self.dt)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gen, device=DEV).to(self.dt)

    def append(self, n):
        """n[b] new tokens of each sequence: pages, rows, bounds. Returns the rotated queries."""
        for b, more in enumerate(n):
            have, need = -(-int(self.lens[b]) // self.ps), -(-int(self.lens[b] + more) // self.ps)
            for slot in range(have, need):
                self.table[b, slot] = self.free.pop()
        self.lens = (self.lens + np.asarray(n)).astype(np.int32)
        T = int(np.sum(n))
        x = self.normal(T, self.H_q + 2 * self.H_kv, self.D)
        self.bt, self.len_dev = i32(self.table), i32(self.lens)
        ptr = i32(np.concatenate([[0], np.cumsum(n)]))
        q, k, v = x.split([self.H_q, self.H_kv, self.H_kv], 1)
        q = ts.ts_kv_append_chunk_rope(q, k, v, self.k, self.v, self.bt, self.len_dev, ptr, self.freq,
                                       q_weight=self.weight, k_weight=self.weight)
        ts.ts_kv_page_bounds(self.k, self.bounds, self.scale, self.bt, self.len_dev, ptr, T)
        return q

    def decode(self, pages, q_len=1):
        B = len(self.lens)
        q = self.append([q_len] * B).view(B, q_len, self.H_q, self.D)
        idx = ts.ts_select_pages(q, self.bounds, self.scale, self.bt, self.len_dev, self.ps, pages, first=1, last=2)
        out, lse = ts.ts_paged_decode_sparse_attn(q, self.k, self.v, self.bt, self.len_dev, idx, self.D ** -0.5,
                                                  return_lse=True)
        k, v, qd = (x.double().cpu().numpy() for x in (self.k, self.v, q))
        codes, scale = self.bounds.cpu().numpy(), self.scale.cpu().numpy()
        for b in range(B):  # the bounds are those of the keys that the cache holds
            for slot in range(-(-int(self.lens[b]) // self.ps)):
                page = self.table[b, slot]
                want = oracle.page_bounds(k[page, :int(self.lens[b]) - slot * self.ps])
                assert np.array_equal(codes[page], want[0]) and np.array_equal(scale[page], want[1])
        want = oracle.select_pages(qd, codes, scale, self.table, self.lens, self.ps, pages, 1, 2)
        assert np.array_equal(idx.cpu().numpy(), want)
        o, l = oracle.sparse_decode_attention(qd, k, v, self.table, self.lens, want, self.D ** -0.5)
        a, _ = oracle.sparse_decode_attention(qd, k, np.abs(v), self.table, self.lens, want, self.D ** -0.5)
        qk = self.D ** -0.5 * np.nanmax(np.abs(k).sum(-1)) * np.abs(qd).max()
        check_attention(out, lse, (o, l, a, qk), self.D, pages * self.ps, self.dtype)

    def fork(self, parents, children):
        fresh = [self.free.pop() for _ in parents]
        self.bt, self.len_dev = i32(self.table), i32(self.lens)
        ts.ts_kv_fork(self.plan, self.bt, self.len_dev, i32(parents), i32(children), i32(fresh), self.ps)
        self.table, self.lens = self.bt.cpu().numpy(), self.len_dev.cpu().numpy()

    def compact(self, keep):
        self.table, self.lens = self.table[keep], self.lens[keep]
        before = [oracle.gather_sequence(self.k.double().cpu().numpy(), t, int(n), self.ps)
                  for t, n in zip(self.table, self.lens)]
        table, page_map, used = ts.ts_kv_compact(self.plan, i32(self.table), i32(self.lens), self.ps)
        self.table = table.cpu().numpy()
        k = self.k.double().cpu().numpy()
        assert all(np.array_equal(x, oracle.gather_sequence(k, t, int(n), self.ps))
                   for x, t, n in zip(before, self.table, self.lens))
        self.free = list(range(int(used), self.P))[::-1]
        assert int(used) == (page_map >= 0).sum()


@pytest.mark.parametrize("dtype,H_q,H_kv,D,ps", [("bf16", 8, 2, 128, 16), ("f32", 4, 2, 64, 8), ("bf16", 8, 1, 64, 32)])
def test_a_served_run(dtype, H_q, H_kv, D, ps):
    s = Server(dtype, H_q, H_kv, D, ps, P=260, rows=5, slots=60)
    s.append([300, 17, 150, 0, 0])
    s.append([33, 1, 0, 0, 0])
    s.fork([0, 2], [3, 4])
    for _ in range(2):
        s.decode(7)
    s.decode(6, q_len=3)
    s.compact([0, 3, 4])
    s.decode(7)
    s.decode(9, q_len=2)
    s.compact([2, 1])
    s.decode(5)
