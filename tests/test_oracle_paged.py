"""The paged operators' oracle against closed forms and element-by-element restatements (CPU)."""

import math

import numpy as np
import pytest

from oracle import paged
from oracle.nsa import to_f64
from workloads import make_paged_inputs


def test_visible_keys():
    assert [paged.visible(p)[1] for p in range(4)] == [1, 2, 3, 4]
    # the Compressor's rows: row w stands for positions w*r .. w*r + r - 1
    for r in (2, 4, 128):
        for p in range(300):
            assert paged.visible(p, r, r)[1] == sum((w + 1) * r - 1 <= p for w in range(400))
    # NSA's rows: row j stands for positions j*stride .. j*stride + block - 1
    for p in range(200):
        assert paged.visible(p, 32, 16)[1] == sum(j * 16 + 31 <= p for j in range(50))
        assert paged.visible(p, 1, 1, 7) == (max(0, p - 6), p + 1)


@pytest.mark.parametrize("pairs", ["interleaved", "halves"])
def test_norm_rope_closed_forms(pairs):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 32))
    y, mag = paged.norm_rope(x, np.ones(32), None, None, pairs, 0.0)
    assert np.allclose((y ** 2).mean(-1), 1.0) and np.allclose(mag, np.abs(y))
    one, zero = np.ones((3, 16)), np.zeros((3, 16))
    assert np.array_equal(paged.norm_rope(x, None, zero, one, pairs, 0.0)[0], x)       # angle 0
    q, _ = paged.norm_rope(x, None, one, zero, pairs, 0.0)                              # a quarter turn
    a, b = ((x[..., 16::2], x[..., 17::2]) if pairs == "interleaved" else (x[..., 16:24], x[..., 24:]))
    qa, qb = ((q[..., 16::2], q[..., 17::2]) if pairs == "interleaved" else (q[..., 16:24], q[..., 24:]))
    assert np.array_equal(qa, -b) and np.array_equal(qb, a) and np.array_equal(q[..., :16], x[..., :16])


@pytest.mark.parametrize("kb,ks,window", [(1, 1, 0), (1, 1, 3), (4, 4, 0), (32, 16, 2)])
def test_attention_is_the_sum_over_keys(kb, ks, window):
    lens, ctx, page, Hq, Hk, D = [3, 0, 2], [10, 4, 37], 16, 4, 2, 16
    rows = [paged.visible(c + n - 1, kb, ks)[1] if n else 0 for n, c in zip(lens, ctx)]
    i = make_paged_inputs(seed=1, lens=lens, ctx=ctx, Hq=Hq, Hk=Hk, D=D, page=page, rows=rows)
    q, kc, vc = (to_f64(a, "bf16") for a in (i.q, i.k_cache, i.v_cache))
    res = paged.paged_attention(q, kc, vc, i.block_table, i.cu_seqlens, i.start_pos, 0.3, key_block=kb, key_stride=ks,
                                window=window)
    for b in range(3):
        for t in range(lens[b]):
            tok, p = int(i.cu_seqlens[b]) + t, ctx[b] + t
            seen = [j for j in range(200) if j * ks + kb - 1 <= p]
            seen = seen[-window:] if window else seen
            for h in range(Hq):
                num, den = np.zeros(D), 0.0
                for j in seen:
                    blk = int(i.block_table[b][j // page])
                    e = math.exp(0.3 * sum(q[tok, h, d] * kc[blk, j % page, h // 2, d] for d in range(D)))
                    den += e
                    num += e * vc[blk, j % page, h // 2]
                if not seen:
                    assert np.all(res.out[tok, h] == 0) and res.lse[tok, h] == -np.inf
                else:
                    assert np.allclose(res.out[tok, h], num / den, rtol=1e-12, atol=1e-13)
                    assert abs(res.lse[tok, h] - math.log(den)) < 1e-12


def test_cache_rows():
    table = np.array([[2, 0], [1, -1]])
    assert paged.cache_rows(table, [0, 3, 3 + 2], [15, 0], 16) == [(0, 47), (1, 0), (2, 1), (3, 16), (4, 17)]
