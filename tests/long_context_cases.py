"""A paged cache in use for the long-context GPU tests: sequences of given lengths on
shuffled pages, with NaN in every row that no sequence holds."""

from __future__ import annotations

import numpy as np
import torch

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


class Cache:
    """Host tensors k_pool, v_pool [P, ps, H_kv, D], table and lengths; `spare` pages more, and
    table rows `slots` longer than the longest sequence (pointing at an unused page)."""

    def __init__(self, seed, lens, H_kv, D, ps=16, dtype="bf16", spare=4, slots=0, fill=True):
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator().manual_seed(seed)
        self.lens = np.asarray(lens, dtype=np.int64)
        self.H_kv, self.D, self.ps, self.dtype = H_kv, D, ps, DTYPES[dtype]
        need = (self.lens + ps - 1) // ps
        self.P = int(need.sum()) + spare
        order = self.rng.permutation(self.P)
        self.table = np.full((len(self.lens), max(1, int(need.max()) + slots)), order[-1], dtype=np.int32)
        self.free = order[int(need.sum()):-1] if spare > 1 else order[:0]
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += int(n)
        shape = (self.P, ps, H_kv, D)
        self.k_pool, self.v_pool = (torch.full(shape, float("nan"), dtype=self.dtype) for _ in "kv")
        if fill:
            for b, L in enumerate(self.lens):
                t = np.arange(int(L))
                for pool in (self.k_pool, self.v_pool):
                    pool[self.table[b, t // ps], t % ps] = self.normal(int(L), H_kv, D)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gen).to(self.dtype)

    def device(self):
        return dict(k_pool=self.k_pool.to(DEV), v_pool=self.v_pool.to(DEV), block_table=i32(self.table),
                    seq_lens=i32(self.lens))

    def bounds(self):
        """Bounds of every page from the oracle's definition, whole pages' rows counted as held."""
        import oracle
        made = [oracle.page_bounds(np.nan_to_num(page)) for page in self.k_pool.float().numpy()]
        return np.stack([c for c, _ in made]), np.stack([s for _, s in made])
