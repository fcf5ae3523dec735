"""Seeded paged caches for the paged operator tests."""
from __future__ import annotations

import numpy as np
import torch

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def table_for(lens, page, seed=0, spare=2, max_pages=None, shared=0):
    """A page table with scattered pages for sequences of the given capacities;
    the first `shared` pages are the same for all.  Unused entries are -7: no
    call may look at them.  Returns (table, pages of the pool)."""
    need = [-(-n // page) for n in lens]
    width = max_pages or max(1, max(need, default=1))
    pool = sum(need) + spare
    order = np.random.default_rng(seed).permutation(pool).astype(np.int32)
    table, at = np.full((len(lens), width), -7, np.int32), shared
    for b, n in enumerate(need):
        for i in range(n):
            if i < shared:
                table[b, i] = order[i]
            else:
                table[b, i] = order[at]
                at += 1
    return table, pool


def owned(table, lens, page, pool):
    """True for every row of the pool that some sequence holds: [pool][page]."""
    mine = np.zeros((pool, page), bool)
    for b, n in enumerate(lens):
        for l in range(max(0, n)):
            mine[table[b, l // page], l % page] = True
    return mine


def randn(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(TYPES[dtype]).cuda()


def rope_table(max_pos, rot, base=10000.0):
    half = rot // 2
    angle = np.arange(max_pos)[:, None] * base ** (-np.arange(half) / half)
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)).cuda()


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()
