"""Seeded synthetic inputs for the paged cache operators (qk_norm_rope, kv_append,
paged_attention). One numpy PCG64 generator per workload; 16-bit tensors are
stored as uint16 bit patterns. Nothing here computes any part of an operator.
"""

from __future__ import annotations

import dataclasses
from typing import Optional, Sequence

import numpy as np

from .nsa import _bits


@dataclasses.dataclass
class PagedInputs:
    dtype: str
    page: int
    q: np.ndarray            # uint16 [T, Hq, D]
    k: np.ndarray            # uint16 [T, Hk, D]
    v: np.ndarray            # uint16 [T, Hk, D]
    k_cache: np.ndarray      # uint16 [blocks, page, Hk, D]
    v_cache: np.ndarray
    block_table: np.ndarray  # int32 [B, pages], -1 past a sequence's rows
    cu_seqlens: np.ndarray   # int32 [B + 1]
    start_pos: np.ndarray    # int32 [B]
    weight: np.ndarray       # uint16 [D]
    sin: Optional[np.ndarray]  # float32 [T, R]
    cos: Optional[np.ndarray]


def make_paged_inputs(*, seed: int, lens: Sequence[int], ctx: Sequence[int], Hq: int, Hk: int, D: int, page: int,
                      dtype: str = "bf16", rope: int = 0, extra_tokens: int = 0, rows: Optional[Sequence[int]] = None,
                      spare_blocks: int = 2) -> PagedInputs:
    """Sequences of lens[b] new tokens after ctx[b] positions; ``rows``: cache rows each
    sequence holds (default ctx + len). ``extra_tokens`` rows follow the last sequence.
    Blocks are drawn from a random permutation; table entries past a sequence's rows
    are -1. Table angles are those of the tokens' positions (base 10000)."""
    rng = np.random.Generator(np.random.PCG64(seed))
    B = len(lens)
    cu = np.concatenate([[0], np.cumsum(np.asarray(lens, dtype=np.int64))]).astype(np.int32)
    T = int(cu[-1]) + extra_tokens
    held = [l + c for l, c in zip(lens, ctx)] if rows is None else list(rows)
    need = [-(-h // page) for h in held]
    pool = sum(need) + spare_blocks
    perm = rng.permutation(pool).astype(np.int32)
    table = np.full((B, max(need + [1])), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    sin = cos = None
    if rope:
        pos = np.zeros(T)
        for b in range(B):
            pos[cu[b]:cu[b + 1]] = ctx[b] + np.arange(lens[b])
        ang = pos[:, None] * 10000.0 ** (-np.arange(0, rope, 2) / rope)[None]
        # the two halves hold different angles, so that a test sees which column is read
        sin = np.concatenate([np.sin(ang), np.sin(ang + 0.25)], 1).astype(np.float32)
        cos = np.concatenate([np.cos(ang), np.cos(ang + 0.25)], 1).astype(np.float32)
    weight = np.abs(rng.standard_normal(D)).astype(np.float32) * 0.2 + 0.9
    w16 = weight.astype(np.float16).view(np.uint16) if dtype == "fp16" else (
        (weight.view(np.uint32) >> 16).astype(np.uint16))
    return PagedInputs(dtype=dtype, page=page, q=_bits(rng, (T, Hq, D), dtype, 2.0), k=_bits(rng, (T, Hk, D), dtype),
                       v=_bits(rng, (T, Hk, D), dtype), k_cache=_bits(rng, (pool, page, Hk, D), dtype),
                       v_cache=_bits(rng, (pool, page, Hk, D), dtype), block_table=table, cu_seqlens=cu,
                       start_pos=np.asarray(ctx, dtype=np.int32), weight=w16, sin=sin, cos=cos)
