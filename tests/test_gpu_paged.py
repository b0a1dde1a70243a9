"""The paged cache operators on a B200 against their oracle (oracle/paged.py):
qk_norm_rope, kv_append and paged_attention, each alone and as they run together."""

import numpy as np
import pytest

from oracle import paged as oracle
from oracle.nsa import to_f64
from tests.paged_helpers import assert_attention, assert_normed, b16, bits, dev
from workloads import make_paged_inputs

pytestmark = pytest.mark.gpu


# ---- qk_norm_rope ------------------------------------------------------------


def norm_case(lib, i, pairs, *, packed=False, tables=None, eps=1e-6, in_place=False):
    import torch
    T, Hq, D = i.q.shape
    Hk = i.k.shape[1]
    q, k = b16(i.q, i.dtype), b16(i.k, i.dtype)
    if packed:  # parts of one projection's output
        qkv = torch.cat([q, k, b16(i.v, i.dtype)], 1)
        q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        before = bits(qkv[:, Hq + Hk:])
    sin, cos = dev(i.sin), dev(i.cos)
    if tables == "bf16" and sin is not None:
        sin, cos = sin.bfloat16(), cos.bfloat16()
    w = b16(i.weight, i.dtype)
    w2 = w.flip(0).contiguous()
    qo, ko = lib.qk_norm_rope(q, k, w, w2, sin=sin, cos=cos, rope_pairs=pairs, eps=eps,
                              q_out=q if in_place else None, k_out=k if in_place else None)
    assert lib.get_error() == 0
    s64 = None if sin is None else sin.float().cpu().numpy()
    c64 = None if cos is None else cos.float().cpu().numpy()
    wv = to_f64(i.weight, i.dtype)
    for got, src, wt in ((qo, i.q, wv), (ko, i.k, wv[::-1])):
        ref, mag = oracle.norm_rope(to_f64(src, i.dtype), wt, s64, c64, pairs, eps)
        assert_normed(bits(got), ref, mag, i.dtype)
    if packed:
        assert np.array_equal(bits(qkv[:, Hq + Hk:]), before)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("pairs", ["interleaved", "halves"])
@pytest.mark.parametrize("T,Hq,Hk,D,rope", [(1, 1, 1, 16, 16), (5, 3, 1, 64, 32), (33, 7, 5, 80, 48),
                                            (17, 32, 8, 128, 128), (3, 40, 24, 192, 64), (9, 5, 2, 256, 256),
                                            (7, 4, 2, 144, 0), (700, 9, 3, 32, 16)])
def test_norm_shapes(lib, dtype, pairs, T, Hq, Hk, D, rope):
    i = make_paged_inputs(seed=T + D, lens=[T], ctx=[3], Hq=Hq, Hk=Hk, D=D, page=16, dtype=dtype, rope=rope)
    norm_case(lib, i, pairs)


@pytest.mark.parametrize("pairs", ["interleaved", "halves"])
@pytest.mark.parametrize("tables", ["f32", "bf16"])
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_of_a_packed_projection(lib, pairs, tables, in_place):
    i = make_paged_inputs(seed=5, lens=[40], ctx=[100000], Hq=12, Hk=4, D=128, page=16, rope=64)
    norm_case(lib, i, pairs, packed=True, tables=tables, in_place=in_place)


def test_norm_queries_only_and_zero_rows(lib):
    import torch
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out, none = lib.qk_norm_rope(q, None, w, eps=1e-6)
    assert none is None and torch.equal(out, q)
    big = torch.full((1, 1, 64), 3e38, dtype=torch.bfloat16, device="cuda")  # the sum of squares overflows
    out, _ = lib.qk_norm_rope(big, None, w)
    assert not torch.isnan(out).any()
    out, _ = lib.qk_norm_rope(q[:0], None, w)
    assert out.shape == (0, 2, 64)


@pytest.mark.parametrize("D", [16, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_over_the_whole_range(lib, D, eps):
    """Heads whose squares leave the range of fp32: up to bf16's largest value, and with eps = 0
    down to its smallest ones; ordinary heads beside them are what they are without them."""
    import torch
    from workloads.synth import bf16_bits
    mags = np.float32([1.0, 3.3e38, 1e30, 2e19, 1.7e19, 1e18, 1e-3] + ([1e-19, 1e-25, 1e-38] if eps == 0 else [1e-3]))
    rng = np.random.default_rng(D)
    x = rng.uniform(-1, 1, (9, len(mags), D)).astype(np.float32)
    x[..., 0] = 1.0
    xb = bf16_bits(x * mags[None, :, None])
    i = make_paged_inputs(seed=D, lens=[9], ctx=[3], Hq=1, Hk=1, D=D, page=16, rope=16)
    w, sin, cos = b16(i.weight, "bf16"), dev(i.sin), dev(i.cos)
    q = b16(xb, "bf16")
    out, none = lib.qk_norm_rope(q, None, w, sin=sin, cos=cos, eps=eps)
    ref, mag = oracle.norm_rope(to_f64(xb, "bf16"), to_f64(i.weight, "bf16"), i.sin, i.cos, "interleaved", eps)
    assert_normed(bits(out), ref, mag, "bf16")
    one, none = lib.qk_norm_rope(q[:, :1], None, w, sin=sin, cos=cos, eps=eps)
    assert torch.equal(one, out[:, :1])
    # the same keys appended
    H = len(mags)
    kc, vc = (torch.zeros(1, 16, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.kv_append(q, q, kc, vc, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), dev(i.cu_seqlens), None,
                  norm_weight=w, sin=sin, cos=cos, eps=eps)
    assert lib.get_error() == 0
    assert torch.equal(kc[0, :9], out) and torch.equal(vc[0, :9], q)


def test_norm_of_infinities_and_zeros(lib):
    """As the formula has it: beside an infinity finite channels are 0 and the infinity is NaN; a
    NaN makes its head NaN; a head of zeros is 0, and NaN (0 / 0) without eps. Other heads stay."""
    import torch
    x = torch.ones(4, 3, 64, dtype=torch.bfloat16, device="cuda")
    x[1, 1, 5] = float("inf")
    x[2, 1, 5] = float("nan")
    x[3, 1] = 0
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for eps in (0.0, 1e-6):
        y, _ = lib.qk_norm_rope(x, None, w, eps=eps)
        assert torch.all(y[:, ::2] == 1) and torch.all(y[0, 1] == 1)
        assert torch.isnan(y[1, 1, 5]) and torch.all(y[1, 1, :5] == 0) and torch.all(y[1, 1, 6:] == 0)
        assert torch.isnan(y[2, 1]).all()
        assert torch.isnan(y[3, 1]).all() if eps == 0 else torch.all(y[3, 1] == 0)


# ---- kv_append ---------------------------------------------------------------


def append_case(lib, i, pairs="interleaved", norm=True, stream=None):
    import torch
    kc, vc = b16(i.k_cache, i.dtype), b16(i.v_cache, i.dtype)
    w = b16(i.weight, i.dtype) if norm else None
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    lib.kv_append(b16(i.k, i.dtype), b16(i.v, i.dtype), kc, vc, dev(i.block_table), dev(i.cu_seqlens),
                  dev(i.start_pos), norm_weight=w, sin=dev(i.sin), cos=dev(i.cos), rope_pairs=pairs, stream=stream)
    torch.cuda.synchronize()
    assert lib.get_error() == 0
    D = i.k.shape[2]
    ref, mag = oracle.norm_rope(to_f64(i.k, i.dtype), to_f64(i.weight, i.dtype) if norm else None, i.sin, i.cos, pairs,
                                1e-6)
    at = oracle.cache_rows(i.block_table, i.cu_seqlens, i.start_pos, i.page)
    tok, row = np.asarray(at, dtype=np.int64).reshape(-1, 2).T
    gk, gv = bits(kc).reshape(-1, *i.k.shape[1:]), bits(vc).reshape(-1, *i.k.shape[1:])
    if i.sin is None and not norm:
        assert np.array_equal(gk[row], i.k[tok])
    else:
        assert_normed(gk[row], ref[tok], mag[tok], i.dtype)
    assert np.array_equal(gv[row], i.v[tok])
    left = np.ones(gk.shape[0], dtype=bool)
    left[row] = False
    assert np.array_equal(gk[left], i.k_cache.reshape(-1, *i.k.shape[1:])[left])
    assert np.array_equal(gv[left], i.v_cache.reshape(-1, *i.k.shape[1:])[left])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("pairs", ["interleaved", "halves"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("lens,ctx,Hk,D,page,rope", [
    ([1], [0], 1, 16, 16, 16),
    ([1] * 40, list(range(0, 400, 10)), 8, 128, 64, 64),
    ([0, 5, 0, 0, 129, 1, 0], [7, 0, 9, 0, 63, 16, 5], 3, 80, 16, 0),
    ([300, 17], [1000, 31], 5, 192, 128, 192),
    ([33, 64, 2], [0, 1, 2], 2, 256, 1, 32),
    ([50], [5], 24, 64, 100, 48),
])
def test_append_shapes(lib, dtype, pairs, norm, lens, ctx, Hk, D, page, rope):
    i = make_paged_inputs(seed=sum(lens) + D, lens=lens, ctx=ctx, Hq=1, Hk=Hk, D=D, page=page, dtype=dtype, rope=rope)
    append_case(lib, i, pairs, norm)


def test_append_many_sequences_and_padding(lib):
    """2000 sequences (three rounds of the sequence search), most of them empty, and
    tokens behind the last one, which are not stored."""
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 3, 2000)]
    i = make_paged_inputs(seed=2, lens=lens, ctx=[int(x) for x in rng.integers(0, 40, 2000)], Hq=1, Hk=2, D=32, page=16,
                          rope=32, extra_tokens=77)
    append_case(lib, i)


def test_append_bad_entries_are_reported(lib):
    import torch
    i = make_paged_inputs(seed=3, lens=[20, 20, 4], ctx=[0, 0, 0], Hq=1, Hk=2, D=64, page=16)
    tbl = i.block_table.copy()
    tbl[0, 1] = -1
    tbl[1, 0] = i.k_cache.shape[0]
    kc, vc = b16(i.k_cache, i.dtype), b16(i.v_cache, i.dtype)
    args = (b16(i.k, i.dtype), b16(i.v, i.dtype), kc, vc)
    lib.kv_append(*args, dev(tbl), dev(i.cu_seqlens), dev(i.start_pos))
    assert lib.get_error() == 5 and lib.get_error() == 0
    gk = bits(kc).reshape(-1, 2, 64)
    stored = 0
    for t, row in oracle.cache_rows(tbl, i.cu_seqlens, i.start_pos, 16):
        if 0 <= row < gk.shape[0]:
            assert np.array_equal(gk[row], i.k[t])
            stored += 1
    assert stored == 16 + 4 + 4
    for cu, sp in (([0, 20, 10, 44], [0, 0, 0]), ([0, 20, 40, 60], [0, 0, 0]), ([3, 20, 40, 44], [0, 0, 0]),
                   ([0, 20, 40, 44], [0, -3, 0]), ([0, 20, 40, 44], [0, 0, 2 ** 31 - 2])):
        lib.kv_append(*args, dev(i.block_table), dev(np.asarray(cu, np.int32)), dev(np.asarray(sp, np.int32)))
        assert lib.get_error() == 5, (cu, sp)
    torch.cuda.synchronize()


def test_append_on_another_stream(lib):
    import torch
    i = make_paged_inputs(seed=4, lens=[100, 3], ctx=[5, 6], Hq=1, Hk=4, D=128, page=32, rope=64)
    append_case(lib, i, stream=torch.cuda.Stream())


# ---- paged_attention ---------------------------------------------------------


def attn_inputs(seed, lens, ctx, Hq, Hk, D, page, dtype="bf16", key_block=1, key_stride=1, **kw):
    rows = [oracle.visible(c + n - 1, key_block, key_stride)[1] if n else 0 for n, c in zip(lens, ctx)]
    return make_paged_inputs(seed=seed, lens=lens, ctx=ctx, Hq=Hq, Hk=Hk, D=D, page=page, dtype=dtype, rows=rows, **kw)


def attn_case(lib, i, *, key_block=1, key_stride=1, window=0, scale=None, stale=None, max_len="exact", stream=None):
    """``stale``: what every cache row that no token of the call sees holds (a number, NaN included)."""
    import torch
    D = i.q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    kc, vc = i.k_cache.copy(), i.v_cache.copy()
    tbl = i.block_table.copy()
    if stale is not None:
        seen = np.zeros(kc.shape[0] * i.page, dtype=bool)
        for b in range(len(i.start_pos)):
            n = int(i.cu_seqlens[b + 1] - i.cu_seqlens[b])
            span = [oracle.visible(int(i.start_pos[b]) + t, key_block, key_stride, window) for t in range(n)]
            keys = {j for lo, hi in span for j in (range(lo, hi) if n <= 2 else ())}
            if n > 2:
                keys = range(min(s[0] for s in span), max(s[1] for s in span))
            used = set()
            for j in keys:
                seen[int(tbl[b][j // i.page]) * i.page + j % i.page] = True
                used.add(j // i.page)
            for c in range(tbl.shape[1]):
                if c not in used:
                    tbl[b, c] = -1
        fill = np.float16(stale).view(np.uint16) if i.dtype == "fp16" else (
            np.uint16(0x7FC0) if np.isnan(stale) else np.uint16(np.float32(stale).view(np.uint32) >> 16))
        kc.reshape(-1, *kc.shape[2:])[~seen] = fill
        vc.reshape(-1, *vc.shape[2:])[~seen] = fill
    lens = np.diff(i.cu_seqlens)
    if max_len == "exact":
        max_len = max(1, int(lens.max(initial=0)))
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    out = torch.full(i.q.shape, 7.0, dtype=torch.float16 if i.dtype == "fp16" else torch.bfloat16, device="cuda")
    lse = torch.full(i.q.shape[:2], 7.0, device="cuda")
    args = (b16(i.q, i.dtype), b16(kc, i.dtype), b16(vc, i.dtype), dev(tbl), dev(i.cu_seqlens), dev(i.start_pos))
    torch.cuda.synchronize()
    lib.paged_attention(*args, scale=scale, max_len=max_len, window=window or None, key_block=key_block,
                        key_stride=key_stride, out=out, lse=lse, stream=stream)
    torch.cuda.synchronize()
    assert lib.get_error() == 0
    res = oracle.paged_attention(to_f64(i.q, i.dtype), to_f64(i.k_cache, i.dtype), to_f64(i.v_cache, i.dtype),
                                 i.block_table, i.cu_seqlens, i.start_pos, scale, key_block=key_block,
                                 key_stride=key_stride, window=window)
    assert_attention(bits(out), lse.cpu().numpy(), res, i.dtype)
    assert torch.all(out[int(i.cu_seqlens[-1]):] == 7) and torch.all(lse[int(i.cu_seqlens[-1]):] == 7)
    return out, lse, args


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("lens,ctx,Hq,Hk,page", [
    ([1], [0], 1, 1, 16),                                   # one key
    ([1, 1, 1], [63, 64, 200], 8, 2, 64),                   # a tile's last key, the next one's first
    ([1] * 5, [0, 1, 500, 17, 1300], 12, 4, 16),            # ragged, cut items
    ([2, 0, 5], [40, 3, 333], 6, 2, 48),                    # a few tokens each, pages of 48
])
def test_decode(lib, dtype, D, lens, ctx, Hq, Hk, page):
    attn_case(lib, attn_inputs(D + len(lens), lens, ctx, Hq, Hk, D, page, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [48, 64, 128, 192, 256])
@pytest.mark.parametrize("lens,ctx,Hq,Hk,page", [
    ([70], [0], 2, 1, 32),                                  # a prompt's first chunk
    ([129, 1, 0, 40], [127, 300, 9, 0], 4, 4, 128),         # chunks next to decoding
    ([37, 90], [600, 2], 14, 2, 16),                        # seven heads per key head
    ([33], [5], 48, 2, 64),                                 # 24 heads per key head
])
def test_chunks(lib, dtype, D, lens, ctx, Hq, Hk, page):
    attn_case(lib, attn_inputs(D + sum(lens), lens, ctx, Hq, Hk, D, page, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [16, 32, 80, 112, 144, 208, 240])
def test_chunks_of_odd_head_sizes(lib, dtype, D):
    attn_case(lib, attn_inputs(D, [130, 1, 37], [5, 140, 260], 6, 2, D, 48, dtype))


@pytest.mark.parametrize("lens,ctx", [([1, 1, 1], [0, 100, 700]), ([50, 9, 260], [0, 31, 300])])
@pytest.mark.parametrize("kb,ks,window", [(1, 1, 5), (1, 1, 100), (4, 4, 0), (32, 16, 0), (32, 16, 3), (1, 1, 4000),
                                          (128, 128, 0)])
def test_windows_and_compressed_rows(lib, lens, ctx, kb, ks, window):
    """Rows that see nothing (tokens before the first compressed row) are 0 with lse -inf."""
    i = attn_inputs(kb + window, lens, ctx, 8, 2, 64, 32, key_block=kb, key_stride=ks)
    attn_case(lib, i, key_block=kb, key_stride=ks, window=window)


@pytest.mark.parametrize("stale", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,ctx,window,D", [([1, 1], [100, 1023], 0, 128), ([1, 2], [100, 300], 40, 64),
                                               ([90, 200], [11, 77], 0, 128), ([60, 33], [200, 700], 50, 192)])
def test_unseen_rows_may_hold_anything(lib, stale, dtype, lens, ctx, window, D):
    """Rows behind a sequence's end, before its window, and blocks that are not its own
    (their table entries are -1) do not reach the outputs."""
    if dtype == "fp16" and abs(stale) < 1e39 and not np.isinf(stale):
        stale = -65504.0
    attn_case(lib, attn_inputs(9, lens, ctx, 8, 2, D, 64, dtype), window=window, stale=stale)


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("rows", [1, 32, 33, 64, 96, 160, 224])
def test_warps_without_rows_clear_stale_values(lib, D, rows):
    """Items whose last row tile leaves one to three of its warps without rows: their lanes
    clear a part of the last key tile's values too, before the product reads any of them."""
    lens, ctx = [rows, 256 + rows, rows, 17], [3, 700, 1999, 90]
    attn_case(lib, attn_inputs(rows + D, lens, ctx, 2, 2, D, 32), stale=float("nan"), max_len=max(lens))


@pytest.mark.parametrize("Hq,Hk", [(128, 1), (16, 1), (17, 1), (64, 64), (15, 5), (36, 12)])
def test_head_layouts(lib, Hq, Hk):
    attn_case(lib, attn_inputs(Hq, [1, 3], [70, 200], Hq, Hk, 64, 16))


@pytest.mark.parametrize("D", [64, 128, 192])
@pytest.mark.parametrize("window", [0, 500])
def test_part_filled_items_between_full_ones(lib, D, window):
    """Items of at most 128 rows (half an item) with long and short contexts between full
    items: whatever runs ahead in them touches nothing that the others still use."""
    import torch
    lens, ctx = [13, 40, 9, 70, 3, 80, 1, 60, 2, 17], [2679, 12, 3000, 1, 1500, 5, 2000, 64, 2500, 0]
    i = attn_inputs(12, lens * 4, ctx * 4, 14, 2, D, 32)
    out, lse, args = attn_case(lib, i, window=window)
    for _ in range(5):
        o, l = lib.paged_attention(*args, max_len=80, window=window or None, return_lse=True)
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_max_len_unknown_and_padding(lib):
    i = attn_inputs(1, [3, 1, 1], [60, 400, 0], 8, 2, 128, 64, extra_tokens=9)
    a, la, _ = attn_case(lib, i, max_len=None)
    attn_case(lib, i, max_len=3)


@pytest.mark.parametrize("max_len", [2, 20])
def test_many_sequences(lib, max_len):
    """1200 sequences (several per thread of a CTA's plan), a third of them without tokens,
    as decoding (four rows per key head) and as chunks (20 tokens may come)."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 3, 1200)]
    if max_len > 2:
        lens[700] = 20
    attn_case(lib, attn_inputs(16, lens, [int(x) for x in rng.integers(0, 90, 1200)], 4, 2, 64, 16), max_len=max_len)


@pytest.mark.parametrize("lens,ctx", [([1, 2, 1], [20000, 30, 20300]), ([40, 1, 300], [6200, 30, 6100])])
def test_most_sequences(lib, lens, ctx):
    """As many sequences as a call may have, three of them with tokens: what those three give
    alone. The contexts are such that a CTA's part holds the end of one and the begin of the next."""
    import torch
    B, at = 2 ** 20, [0, 700001, 2 ** 20 - 1]
    i = attn_inputs(17, lens, ctx, 4, 1, 64, 128)
    out, lse, args = attn_case(lib, i)
    cu, sp = np.zeros(B + 1, np.int32), np.zeros(B, np.int32)
    tbl = np.full((B, i.block_table.shape[1]), -1, np.int32)
    for b, n, t, c in zip(at, lens, i.block_table, i.start_pos):
        cu[b + 1], tbl[b], sp[b] = n, t, c
    cu = np.cumsum(cu).astype(np.int32)
    o, l = lib.paged_attention(*args[:3], dev(tbl), dev(cu), dev(sp), max_len=max(lens), return_lse=True)
    assert lib.get_error() == 0
    assert torch.equal(o, out) and torch.equal(l, lse)


def test_strided_queries(lib):
    import torch
    i = attn_inputs(2, [40, 1], [100, 500], 8, 2, 128, 64)
    out, lse, args = attn_case(lib, i)
    qkv = torch.randn(41, 12, 128, device="cuda").to(torch.bfloat16)
    qkv[:, :8] = args[0]
    out2, lse2 = lib.paged_attention(qkv[:, :8], *args[1:], max_len=40, return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens,ctx", [([1], [3000]), ([1, 1, 1], [0, 5000, 40]), ([200, 1], [900, 4000])])
def test_long_context(lib, lens, ctx):
    attn_case(lib, attn_inputs(3, lens, ctx, 8, 2, 128, 64))


def test_large_scores(lib):
    """Scores far apart (weights under- and overflowing a fixed reference)."""
    attn_case(lib, attn_inputs(4, [1, 80], [700, 300], 4, 2, 128, 32), scale=4.0)


def test_growing_scores(lib):
    """The running maximum grows by much from tile to tile, and falls behind."""
    from workloads.synth import bf16_bits
    i = attn_inputs(5, [1, 70], [1500, 600], 4, 1, 64, 64)
    g = np.ones(i.k_cache.shape[:2], np.float32)
    for b in range(2):
        n = int(i.start_pos[b] + i.cu_seqlens[b + 1] - i.cu_seqlens[b])
        for j in range(n):
            g[i.block_table[b][j // 64], j % 64] = 0.2 + 6.0 * j / n if b == 0 else 6.0 * (n - j) / n
    i.k_cache = bf16_bits((to_f64(i.k_cache, "bf16") * g[..., None, None]).astype(np.float32))
    attn_case(lib, i)


def test_repeat_is_bit_identical(lib):
    import torch
    i = attn_inputs(6, [1] * 7 + [100], [10, 500, 2000, 3, 0, 77, 900, 60], 8, 2, 128, 64)
    out, lse, args = attn_case(lib, i)
    for _ in range(5):
        o, l = lib.paged_attention(*args, max_len=100, return_lse=True)
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_two_streams_at_once(lib):
    import torch
    i = attn_inputs(7, [1] * 6, [1000, 500, 2000, 3, 0, 77], 8, 2, 128, 64)
    j = attn_inputs(8, [130], [600], 8, 2, 128, 64)
    oi, li, ai = attn_case(lib, i)
    oj, lj, aj = attn_case(lib, j)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    res = []
    for _ in range(10):
        res.append((lib.paged_attention(*ai, max_len=1, return_lse=True, stream=s1),
                    lib.paged_attention(*aj, max_len=130, return_lse=True, stream=s2)))
    torch.cuda.synchronize()
    for (a, b) in res:
        assert torch.equal(a[0], oi) and torch.equal(a[1], li) and torch.equal(b[0], oj) and torch.equal(b[1], lj)
    assert lib.get_error() == 0


def test_bad_entries_are_reported(lib):
    import torch
    i = attn_inputs(9, [1, 1, 20], [100, 50, 30], 4, 2, 64, 16)
    out, lse, args = attn_case(lib, i)
    tbl = i.block_table.copy()
    tbl[0, 2] = i.k_cache.shape[0] + 9
    o, l = lib.paged_attention(*args[:3], dev(tbl), *args[4:], max_len=20, return_lse=True)
    assert lib.get_error() == 5 and lib.get_error() == 0
    assert torch.equal(o[1:], out[1:]) and torch.isfinite(o.float()).all()
    for cu, sp, ml in (([0, 1, 0, 22], [100, 50, 30], 22), ([0, 1, 2, 23], [100, 50, 30], 20),
                       ([0, 1, 2, 22], [100, -1, 30], 20), ([0, 1, 2, 22], [100, 50, 30], 19),
                       ([0, 1, 2, 22], [2 ** 31 - 1, 50, 30], 20), ([1, 1, 2, 22], [100, 50, 30], 20),
                       ([0, 1, 2, 22], [2 ** 31 - 1025, 50, 30], 20), ([0, 1, 2, 22], [100, 2 ** 31 - 2, 30], 20)):
        lib.paged_attention(*args[:4], dev(np.asarray(cu, np.int32)), dev(np.asarray(sp, np.int32)), max_len=ml)
        assert lib.get_error() == 5, (cu, sp, ml)
    torch.cuda.synchronize()


@pytest.mark.parametrize("raw", [False, True])
def test_default_stream_by_name(lib, raw):
    """The default stream given explicitly (its handle is 0) while another one is current: the
    call runs there, and what it allocates belongs to it."""
    import torch
    d = torch.device("cuda", torch.cuda.current_device())
    default = torch.cuda.default_stream()
    i = attn_inputs(33, [1, 30], [70, 200], 8, 2, 64, 16, rope=32)
    args = [b16(i.q, "bf16"), b16(i.k_cache, "bf16"), b16(i.v_cache, "bf16"), dev(i.block_table), dev(i.cu_seqlens),
            dev(i.start_pos)]
    w = b16(i.weight, "bf16")
    want = lib.paged_attention(*args, max_len=30)
    want_q, _ = lib.qk_norm_rope(args[0], None, w)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        with lib._on_stream(0, d, torch):
            assert torch.cuda.current_stream() == default
        s = 0 if raw else default
        assert torch.equal(lib.paged_attention(*args, max_len=30, stream=s), want)
        assert torch.equal(lib.qk_norm_rope(args[0], None, w, stream=s)[0], want_q)
    torch.cuda.synchronize()
    assert lib.get_error() == 0


@pytest.mark.parametrize("flag", [True, 1, np.True_, False, 0, np.False_, None])
def test_return_lse_is_a_truth_value(lib, flag):
    """The compiled binding (no stream given) and the Python one (a stream) take the same flags."""
    import torch
    i = attn_inputs(31, [1, 1], [70, 200], 8, 2, 64, 16)
    args = [b16(i.q, "bf16"), b16(i.k_cache, "bf16"), b16(i.v_cache, "bf16"), dev(i.block_table), dev(i.cu_seqlens),
            dev(i.start_pos)]
    for stream in (None, torch.cuda.current_stream()):
        r = lib.paged_attention(*args, max_len=1, return_lse=flag, stream=stream)
        assert type(r) is (tuple if flag else torch.Tensor)
    assert lib.get_error() == 0


def test_both_bindings_agree(lib, monkeypatch):
    """The compiled binding against the Python one: the same results, or the same refusals."""
    import torch
    i = attn_inputs(32, [2, 1], [70, 200], 8, 2, 64, 16, rope=32)
    q, k, v = (b16(a, "bf16") for a in (i.q, i.k, i.v))
    kc, vc, tbl, cu, sp = (b16(i.k_cache, "bf16"), b16(i.v_cache, "bf16"), dev(i.block_table), dev(i.cu_seqlens),
                           dev(i.start_pos))
    w, sin, cos = b16(i.weight, "bf16"), dev(i.sin), dev(i.cos)
    out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    odd = torch.empty(3 * 8 * 64 + 1, dtype=q.dtype, device="cuda")[1:].view(3, 8, 64)
    ws = torch.empty(lib.paged_attention_workspace(3, 8, 2, 64, 2), dtype=torch.uint8, device="cuda")

    def norm(*a, **kw):
        return lib.qk_norm_rope(*a, **kw)

    def append(*a, **kw):
        return lib.kv_append(*a[:2], kc.clone(), vc.clone(), *a[2:], **kw)

    def attn(*a, **kw):
        return lib.paged_attention(*a, **{"max_len": 2, **kw})

    A, N, P = (q, kc, vc, tbl, cu, sp), (q, k, w, w), (k, v, tbl, cu, sp)
    calls = [(norm, N, {}), (norm, N, dict(sin=sin, cos=cos, rope_pairs="halves", eps=0)), (norm, (q, None, w), {}),
             (norm, N, dict(sin=sin)), (norm, N, dict(sin=sin, cos=cos[:, :16])), (norm, N, dict(rope_pairs="x")),
             (norm, N, dict(eps=-1.0)), (norm, N, dict(eps=float("nan"))), (norm, N, dict(eps="1")),
             (norm, N, dict(eps=10 ** 400)), (norm, N, dict(eps=np.float32(1e-5))), (norm, (q, k, w), {}),
             (norm, (q, k, w, w[:32]), {}), (norm, (q, k[:2], w, w), {}), (norm, (q.float(), k, w, w), {}),
             (norm, (q, k.half(), w, w), {}), (norm, N, dict(q_out=odd)), (norm, N, dict(q_out=out[:, :, :32])),
             (norm, (q.cpu(), k, w, w), {}), (norm, (q, k.cpu(), w, w), {}), (norm, (None, k, w, w), {}),
             (norm, (q[:0], k[:0], w, w), {}), (norm, (q.transpose(1, 2), k, w, w), {}), (norm, (q[:, :, ::2], None, w), {}),
             (append, P, {}), (append, P, dict(norm_weight=w, sin=sin, cos=cos)), (append, P[:4], {}),
             (append, P, dict(norm_weight=w.float())), (append, P, dict(sin=sin.half(), cos=cos.half())),
             (append, (k, v[:, :1], tbl, cu, sp), {}), (append, (k, None, tbl, cu, sp), {}),
             (append, (k, v, tbl.long(), cu, sp), {}), (append, (k, v, tbl[:1], cu, sp), {}),
             (append, (k, v, tbl.t(), cu, sp), {}), (append, (k, v, tbl, cu[:0], sp), {}),
             (append, (k, v, tbl, cu, sp[:1]), {}), (append, P, dict(eps=float("inf"))), (append, P, dict(rope_pairs=None)),
             (attn, A, {}), (attn, A, dict(return_lse=True)), (attn, A, dict(lse=lse)), (attn, A, dict(out=out)),
             (attn, A, dict(out=out, lse=lse, workspace=ws)), (attn, A, dict(workspace=ws[:-1])),
             (attn, A, dict(workspace=ws.cpu())), (attn, A, dict(out=odd)), (attn, A, dict(out=out[:2])),
             (attn, A, dict(lse=lse.double())), (attn, A, dict(max_len=0)), (attn, A, dict(max_len=None)),
             (attn, A, dict(max_len=2.0)), (attn, A, dict(max_len=np.int64(2))), (attn, A, dict(max_len=True)),
             (attn, A, dict(max_len=2 ** 31)), (attn, A, dict(window=0)), (attn, A, dict(window=-1)),
             (attn, A, dict(window=7)), (attn, A, dict(window=2 ** 31)), (attn, A, dict(window=1.5)),
             (attn, A, dict(key_block=0)), (attn, A, dict(key_block=None)), (attn, A, dict(key_stride=-2)),
             (attn, A, dict(key_block=4, key_stride=4, return_lse=True)), (attn, A, dict(scale=0)), (attn, A, dict(scale=1)),
             (attn, A, dict(scale=np.float64(0.25))), (attn, A, dict(scale=float("nan"))), (attn, A, dict(scale=1e300)),
             (attn, A, dict(scale="1")), (attn, A[:5], {}), (attn, (q[:, :7], *A[1:]), {}), (attn, (q, kc.half(), *A[2:]), {}),
             (attn, (q, kc, vc[:1], *A[3:]), {}), (attn, (q, kc[:, :8], vc[:, :8], *A[3:]), {}), (attn, (q[:0], *A[1:]), {}),
             (attn, (q, kc, vc, tbl[:0], cu[:1], sp[:0]), {}), (attn, (q[:0], kc, vc, tbl[:0], cu[:1], sp[:0]), {})]

    def outcome(f, a, kw):
        try:
            r = f(*a, **kw)
        except Exception as e:  # noqa: BLE001  (whatever a user would see)
            return type(e), str(e)
        lib.get_error()
        r = r if isinstance(r, tuple) else (r,)
        return [None if t is None else (t.dtype, tuple(t.shape), t.stride(), bits(t.bfloat16()).tolist()) for t in r]

    from collections import Counter
    kinds = Counter()
    assert lib._torch_module() and lib._calls is not None
    for f, a, kw in calls:
        compiled = outcome(f, a, kw)
        with monkeypatch.context() as m:
            m.setattr(lib, "_calls", None)
            python = outcome(f, a, kw)
        assert compiled == python, (f.__name__, {n: x for n, x in kw.items()})
        kinds[isinstance(compiled, list)] += 1
    assert min(kinds.values()) > 20


def test_numbers_past_64_bits_are_refused(lib):
    """They would wrap to a small one (2^64 + 3 to a window of 3)."""
    i = attn_inputs(34, [1], [70], 8, 2, 64, 16)
    args = [b16(i.q, "bf16"), b16(i.k_cache, "bf16"), b16(i.v_cache, "bf16"), dev(i.block_table), dev(i.cu_seqlens),
            dev(i.start_pos)]
    for name in ("max_len", "window", "key_block", "key_stride"):
        for v in (2 ** 64 + 3, 2 ** 64, 2 ** 63, -2 ** 64 + 1):
            with pytest.raises((ValueError, lib.CmpError)):
                lib.paged_attention(*args, **{name: v})
    assert lib.get_error() == 0


def test_error_words_are_taken_once(lib):
    """Threads that ask for errors on streams of their own while another one's calls report
    them: each report is taken by exactly one of them (a token of one head of 16 channels is
    one warp's, which reports once), and none is lost."""
    import threading

    import torch
    i = make_paged_inputs(seed=35, lens=[1], ctx=[3], Hq=1, Hk=1, D=16, page=16)
    args = (b16(i.k, "bf16"), b16(i.v, "bf16"), b16(i.k_cache, "bf16"), b16(i.v_cache, "bf16"))
    good, bad, cu, sp = dev(i.block_table), dev(i.block_table * 0 - 1), dev(i.cu_seqlens), dev(i.start_pos)
    lib.kv_append(*args, good, cu, sp)
    torch.cuda.synchronize()
    assert lib.get_error() == 0
    stop, seen = threading.Event(), []

    def ask():
        s, n = torch.cuda.Stream(), 0
        while not stop.is_set():
            n += lib.get_error(s) == 5
        seen.append(n)

    askers = [threading.Thread(target=ask) for _ in range(3)]
    for t in askers:
        t.start()
    s = torch.cuda.Stream()
    mine, rounds = 0, 400
    for _ in range(rounds):
        lib.kv_append(*args, bad, cu, sp, stream=s)
        got = lib.get_error(s)
        assert got in (0, 5)
        mine += got == 5
        assert lib.get_error(s) == 0
    stop.set()
    for t in askers:
        t.join()
    assert mine + sum(seen) == rounds and lib.get_error() == 0


def long_call(seed, lens, ctx, Hq, Hk, D, dtype, blocks, page=512, ones=False):
    """Sequences over one cache of few blocks, each sequence's table repeating them in its own order."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float16 if dtype == "fp16" else torch.bfloat16
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    kc = (rand(blocks, page, Hk, D) * 0.5).to(dt)
    vc = torch.ones_like(kc) if ones else rand(blocks, page, Hk, D).to(dt)
    q = rand(sum(lens), Hq, D).to(dt)
    pages = max(-(-(n + c) // page) for n, c in zip(lens, ctx))
    tbl = torch.stack([torch.randperm(blocks, generator=g, device="cuda").repeat(-(-pages // blocks))[:pages]
                       for _ in lens]).int()
    cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")
    return q, kc, vc, tbl, cu, torch.tensor(ctx, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("keys", [2 ** 15, 2 ** 20])
def test_long_sums_keep_their_size(lib, D, keys):
    """Values of 1 come out as 1 however many keys a CTA sums (more items than CTAs). The sums of
    the weights, rounded to fp16 (h relative), lose at most 2^-12 in the accumulator, and the sum
    that they are divided by is off by (tiles of a part + 64) 2^-24; out is rounded once (h)."""
    args = long_call(D, [17] * 10, [keys - 17] * 10, 128, 16, D, "fp16", 2, ones=True)
    out, lse = lib.paged_attention(*args, max_len=17, return_lse=True)
    assert lib.get_error() == 0
    h = 2.0 ** -11
    err = float((out.double() - 1).abs().max())
    assert err <= (h + h + 2.0 ** -12 + 320 * 2.0 ** -24) * 1.001, err


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("heads", [2, 16])
def test_long_sums_of_decoding_keep_their_size(lib, D, heads):
    """The same of single tokens over 2^22 keys, 8 and 16 rows per item. A warp adds 2^16 times
    and rounds each sum, which errs to either side (at most 6 sqrt(2^16) 2^-24 but for one row in
    10^8), in the numerator and in the denominator; within 16 keys it may cut 16 times."""
    keys = 2 ** 22
    args = long_call(D, [1] * 20, [keys - 1] * 20, 16 * heads, 16, D, "fp16", 2, ones=True)
    out = lib.paged_attention(*args, max_len=1)
    assert lib.get_error() == 0
    h, u = 2.0 ** -11, 2.0 ** -24
    err = float((out.double() - 1).abs().max())
    assert err <= (h + h + 2 * 6 * 2 ** 8 * u + 32 * u) * 1.001, err


@pytest.mark.parametrize("D,G,dtype", [(64, 17, "bf16"), (128, 17, "fp16"), (128, 129, "bf16"), (192, 40, "fp16"),
                                       (192, 17, "bf16"), (256, 17, "fp16")])
@pytest.mark.parametrize("window", [0, 33000])
def test_pieces_of_several_parts(lib, D, G, dtype, window):
    """Contexts around the multiples of what is summed in one go (256 tiles of 128 or 64 keys),
    more items than CTAs: whole items in parts, cut ones in parts, and short ones between them."""
    import torch
    from tests.paged_helpers import HALF, TINY, U
    part = 256 * (128 if D <= 128 else 64)
    if G > 128:
        G, lens = 16, [9, 2, 16]
    else:
        lens = [1, 1, 1]
    ctx = [part - 1, part, part + 1, 2 * part - 2, 2 * part + 130, 40, 3 * part + 5, 7]
    ctx, lens = (ctx * 24)[:180], (lens * 60)[:180]
    args = long_call(D + G, lens, ctx, G, 1, D, dtype, 4)
    q, kc, vc, tbl, cu, sp = args
    out, lse = lib.paged_attention(*args, max_len=max(max(lens), 2), window=window or None, return_lse=True)
    again, lse2 = lib.paged_attention(*args, max_len=max(max(lens), 2), window=window or None, return_lse=True)
    assert lib.get_error() == 0
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    h, scale = HALF[dtype], D ** -0.5
    k64, v64 = kc.double().view(-1, D), vc.double().view(-1, D)
    worst = worst_lse = 0.0
    for b in [*range(8), 100, 179]:
        for t in (0, lens[b] - 1):
            row = int(cu[b]) + t
            n = ctx[b] + t + 1
            lo = max(0, n - window) if window else 0
            at = torch.arange(lo, n, device="cuda")
            at = tbl[b].long()[at // 512] * 512 + at % 512
            x = q[row].double() @ k64[at].t() * scale
            mag = (q[row].double().abs() @ k64[at].abs().t() * scale).amax(-1)
            want_lse = torch.logsumexp(x, -1)
            w = torch.exp(x - want_lse[:, None])
            want, vm = w @ v64[at], w @ v64[at].abs()
            dw = (2 * D + 8) * U * mag + 8 * U
            m = n - lo + 64
            lim = h * want.abs() + vm * (h + 2 * dw + 4 * m * U)[:, None] * (1 + h) + TINY[dtype] * (
                1 + v64[at].abs().sum(0))
            worst = max(worst, float(((out[row].double() - want).abs() / lim).max()))
            worst_lse = max(worst_lse, float(((lse[row].double() - want_lse).abs() /
                                              (dw + m * U + 4 * U * want_lse.abs())).max()))
    assert worst <= 1 and worst_lse <= 1, (worst, worst_lse)


@pytest.mark.parametrize("D,heads,tokens", [(128, (8, 2), 1), (192, (8, 4), 1), (256, (4, 1), 3)])
def test_waits_that_give_up_are_reported(lib, D, heads, tokens):
    """A decoding call whose key tiles never come: every warp gives up as one, the call ends,
    says so once, and the next call is right again."""
    import torch
    i = attn_inputs(D, [tokens] * 3, [100, 700, 3000], *heads, D, 64)
    out, lse, args = attn_case(lib, i)
    try:
        assert lib.debug_unreachable_barrier(1) == 0
        o, l = lib.paged_attention(*args, max_len=tokens, return_lse=True)
        torch.cuda.synchronize()
        assert lib.debug_unreachable_barrier(0) == 0                  # the knob was consumed
    finally:
        lib.debug_unreachable_barrier(0)
    assert lib.get_error() == 6 and lib.get_error() == 0
    assert torch.all(o == 0) and torch.all(torch.isneginf(l))
    again, lse2 = lib.paged_attention(*args, max_len=tokens, return_lse=True)
    assert lib.get_error() == 0 and torch.equal(again, out) and torch.equal(lse2, lse)


def test_captured_and_replayed(lib):
    """A decode step of all three operators in a graph, replayed after its inputs moved on."""
    import torch
    i = attn_inputs(10, [1, 1], [90, 300], 8, 2, 128, 64, rope=64)
    q, k, v = b16(i.q, "bf16"), b16(i.k, "bf16"), b16(i.v, "bf16")
    kc, vc, tbl, cu = b16(i.k_cache, "bf16"), b16(i.v_cache, "bf16"), dev(i.block_table), dev(i.cu_seqlens)
    sp, w, sin, cos = dev(i.start_pos), b16(i.weight, "bf16"), dev(i.sin), dev(i.cos)

    def step():
        qn, _ = lib.qk_norm_rope(q, None, w, sin=sin, cos=cos)
        lib.kv_append(k, v, kc, vc, tbl, cu, sp, norm_weight=w, sin=sin, cos=cos)
        return lib.paged_attention(qn, kc, vc, tbl, cu, sp, max_len=1, return_lse=True)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = step()
    for shift in (0, -1, -30):
        sp.copy_(dev(i.start_pos) + shift)
        g.replay()
        eager = step()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
    assert lib.get_error() == 0


# ---- together, and at the edges ------------------------------------------------


def test_nsa_step_together(lib):
    """One decode step over both caches of NSA: keys and values appended, the step's windows
    compressed by nsa_compress, attention over a window of raw rows and over the compressed
    rows, joined by lse: the softmax over both sets of keys."""
    import torch
    block, stride, win, Hq, Hk, D, page = 32, 16, 64, 8, 2, 128, 64
    ctx = [79, 200, 31, 127, 415]  # new lengths 80, 201, 32, 128, 416: four on a compression step
    B = len(ctx)
    i = attn_inputs(21, [1] * B, ctx, Hq, Hk, D, page, rope=64)
    q, k, v = b16(i.q, "bf16"), b16(i.k, "bf16"), b16(i.v, "bf16")
    kc, vc = b16(i.k_cache, "bf16"), b16(i.v_cache, "bf16")
    tbl, cu, sp = dev(i.block_table), dev(i.cu_seqlens), dev(i.start_pos)
    w, sin, cos = b16(i.weight, "bf16"), dev(i.sin), dev(i.cos)
    qn, _ = lib.qk_norm_rope(q, None, w, sin=sin, cos=cos)
    lib.kv_append(k, v, kc, vc, tbl, cu, sp, norm_weight=w, sin=sin, cos=cos)
    # the compressed rows' cache: sequence b owns block b of 32 rows; rows of earlier steps are there
    rows = 32
    g = torch.Generator(device="cuda").manual_seed(3)
    cmp_k = torch.randn(B, rows, Hk, D, generator=g, device="cuda").bfloat16()
    cmp_v = torch.randn(B, rows, Hk, D, generator=g, device="cuda").bfloat16()
    cw = torch.full((block, Hk), 1 / block, device="cuda").bfloat16()
    lens = [c + 1 for c in ctx]
    held = [(n - block) // stride + 1 for n in lens]
    slots = torch.tensor([b * rows + max(h - 1, 0) for b, h in enumerate(held)], dtype=torch.int32, device="cuda")
    act = torch.tensor(lens, dtype=torch.int64, device="cuda")
    for src, dst in ((kc, cmp_k), (vc, cmp_v)):
        before = dst.clone()
        lib.nsa_compress(src, cw, slots, act, dst.view(B * rows, Hk, D), compress_block_size=block,
                         compress_stride=stride, block_table=tbl, page_block_size=page)
        assert not torch.equal(before, dst)
    ctbl = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    raw = lib.paged_attention(qn, kc, vc, tbl, cu, sp, max_len=1, window=win, return_lse=True)
    com = lib.paged_attention(qn, cmp_k, cmp_v, ctbl, cu, sp, max_len=1, key_block=block, key_stride=stride,
                              return_lse=True)
    assert lib.get_error() == 0
    f = lambda t: to_f64(bits(t), "bf16")  # noqa: E731
    ref = [oracle.paged_attention(f(qn), f(a), f(b), t.cpu().numpy(), i.cu_seqlens, i.start_pos, D ** -0.5, **kw)
           for a, b, t, kw in ((kc, vc, tbl, dict(window=win)),
                               (cmp_k, cmp_v, ctbl, dict(key_block=block, key_stride=stride)))]
    for (out, lse), r in zip((raw, com), ref):
        assert_attention(bits(out), lse.cpu().numpy(), r, "bf16")
    from tests.paged_helpers import attention_limits
    total = np.logaddexp(ref[0].lse, ref[1].lse)
    want = sum(np.exp(r.lse - total)[..., None] * r.out for r in ref)
    got_total = torch.logaddexp(raw[1].double(), com[1].double())
    got = sum(torch.exp(x[1].double() - got_total)[..., None] * x[0].double() for x in (raw, com)).cpu().numpy()
    lim = [attention_limits(r, D, "bf16") for r in ref]
    # the weights are off by at most the sum of both lse errors, on the difference of the outs
    tol = np.maximum(lim[0][0], lim[1][0]) + (lim[0][1] + lim[1][1])[..., None] * 2 * (
        np.abs(ref[0].out) + np.abs(ref[1].out))
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("lens,ctx", [([1, 1, 1], [100, 300, 50]), ([40, 3, 200], [100, 300, 50])])
def test_nan_reaches_its_own_rows_only(lib, lens, ctx):
    """A NaN key that every token of sequence 1 sees: its head group's outs and lse there are
    NaN, all other rows bit for bit what they were."""
    import torch
    i = attn_inputs(13, lens, ctx, 8, 2, 128, 64)
    out, lse, args = attn_case(lib, i)
    kc = args[1].clone()
    kc[int(i.block_table[1][0]), 7, 1] = float("nan")
    o, l = lib.paged_attention(args[0], kc, *args[2:], max_len=max(lens), return_lse=True)
    assert lib.get_error() == 0
    t0, t1 = int(i.cu_seqlens[1]), int(i.cu_seqlens[2])
    hit = torch.zeros_like(l, dtype=torch.bool)
    hit[t0:t1, 4:] = True
    assert torch.isnan(l[hit]).all() and torch.isnan(o[hit]).all()
    assert torch.equal(l[~hit], lse[~hit]) and torch.equal(o[~hit], out[~hit])


def test_only_padding(lib):
    import torch
    i = attn_inputs(14, [0, 0], [30, 40], 8, 2, 64, 16, extra_tokens=5)
    attn_case(lib, i, max_len=5)
    attn_case(lib, i, max_len=1)
    append_case(lib, i)
    torch.cuda.synchronize()


def test_caches_past_2_31_elements(lib):
    """Blocks at the far end of caches of 4.6e9 elements each."""
    import torch
    blocks, page, Hk, D = 70000, 64, 8, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    i = attn_inputs(15, [1, 33], [130, 100], 16, Hk, D, page)
    n = i.k_cache.shape[0]
    kc, vc = (torch.empty((blocks, page, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc[blocks - n:], vc[blocks - n:] = b16(i.k_cache, "bf16"), b16(i.v_cache, "bf16")
    tbl = dev(np.where(i.block_table >= 0, i.block_table + blocks - n, -1).astype(np.int32))
    cu, sp = dev(i.cu_seqlens), dev(i.start_pos)
    small_k, small_v, small_tbl = b16(i.k_cache, "bf16"), b16(i.v_cache, "bf16"), dev(i.block_table)
    k, v, q = b16(i.k, "bf16"), b16(i.v, "bf16"), b16(i.q, "bf16")
    lib.kv_append(k, v, kc, vc, tbl, cu, sp)
    lib.kv_append(k, v, small_k, small_v, small_tbl, cu, sp)
    assert torch.equal(kc[blocks - n:], small_k) and torch.equal(vc[blocks - n:], small_v)
    for sel, ml in ((slice(0, 1), 1), (slice(0, 34), 33)):
        c = cu[:2] if ml == 1 else cu
        a = lib.paged_attention(q[sel], kc, vc, tbl[:len(c) - 1], c, sp[:len(c) - 1], max_len=ml, return_lse=True)
        b = lib.paged_attention(q[sel], small_k, small_v, small_tbl[:len(c) - 1], c, sp[:len(c) - 1], max_len=ml,
                                return_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert lib.get_error() == 0
