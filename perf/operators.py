"""The measured cases of the paged-cache operators: qk_norm_rope, kv_append and paged_attention.

``run`` computes a case either in its plain form (elementary torch operations in 32 bits, rounded
once at the end) or, with ``own``, through the package's entry points. ``exact`` is the definition
in 64 bits. Lengths follow from the case alone; tensors follow from the seed.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ---- cases ----------------------------------------------------------------------------------


def _attn(name, dtype, B, lens, ctx, mix, Hq, Hk, D, page, window=0, key_block=1, key_stride=1):
    """paged_attention: B sequences, chunk lengths in lens = "lo:hi", tokens before them in ctx = "lo:hi"."""
    return {"name": name, "op": "attention", "dtype": dtype, "B": B, "lens": lens, "ctx": ctx, "mix": mix, "Hq": Hq,
            "Hk": Hk, "D": D, "page": page, "window": window, "key_block": key_block, "key_stride": key_stride}


def _append(name, dtype, B, lens, ctx, mix, Hk, D, page, rope, pairs, norm):
    return {"name": name, "op": "append", "dtype": dtype, "B": B, "lens": lens, "ctx": ctx, "mix": mix, "Hk": Hk,
            "D": D, "page": page, "rope": rope, "pairs": pairs, "norm": norm}


def _norm(name, dtype, T, Hq, Hk, D, rope, pairs, packed):
    return {"name": name, "op": "qk_norm_rope", "dtype": dtype, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rope": rope,
            "pairs": pairs, "packed": packed}


def listed():
    return [
        # one request answering: one token over a short cache, latency alone
        _attn("attn_one_token", "bf16", 1, "1:1", "600:600", 0, 32, 8, 128, 64),
        # the decode step of the NSA cache (128 batches, 24 heads of 192, page 128), two query heads per key head
        _attn("attn_decode_nsa", "bf16", 128, "1:1", "200:2000", 1, 48, 24, 192, 128),
        # few requests whose lengths differ by four orders of magnitude, an odd head count and head size
        _attn("attn_decode_ragged", "fp16", 9, "1:1", "0:100000", 2, 20, 4, 80, 16),
        # decoding of a long context with drafts to verify: five tokens each, eight heads per key head
        _attn("attn_draft_verify", "bf16", 4, "5:5", "30000:60000", 3, 64, 8, 128, 64),
        # continuous batching: prompts being read in chunks next to requests that decode, ragged
        _attn("attn_mixed_batch", "bf16", 24, "1:700", "0:6000", 4, 28, 4, 128, 32, window=4096),
        # a chunk of a long prompt
        _attn("attn_prompt_chunk", "bf16", 1, "4096:4096", "12288:12288", 0, 32, 8, 128, 128),
        # prompt tokens over NSA's compressed rows (window 32, stride 16): the first 31 tokens see none
        _attn("attn_compressed_rows", "fp16", 2, "1500:2500", "0:9000", 5, 64, 4, 192, 64, key_block=32, key_stride=16),
        # one decode step's keys and values
        _append("append_decode", "bf16", 32, "1:1", "10:4000", 6, 8, 128, 64, 64, "interleaved", True),
        # a batch of prompts
        _append("append_prompts", "bf16", 6, "1000:8000", "0:3000", 7, 8, 128, 128, 128, "halves", True),
        # a ragged batch with an odd head size, half of each head rotated, keys that come normed
        _append("append_ragged", "fp16", 33, "0:301", "0:999", 8, 5, 80, 16, 32, "interleaved", False),
        # the queries and keys of one decode step, as parts of one projection's output
        _norm("norm_decode", "bf16", 32, 32, 8, 128, 64, "interleaved", True),
        # the queries and keys of prompts
        _norm("norm_prompts", "bf16", 16384, 32, 8, 128, 128, "halves", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "qk_norm_rope"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    D = rng.choice([64, 128, 128, 128, 192, 16 * rng.randint(2, 16)])
    mix = rng.randint(0, 10 ** 6)
    Hk = rng.choice([1, 2, 4, 8, rng.randint(1, 24)])
    if op == "qk_norm_rope":
        T = _log(rng, 1, 16000)
        Hq = Hk * rng.choice([1, 2, 4, 7, 8])
        while T * (Hq + Hk) * D > 16384 * 40 * 128:
            T = (T + 1) // 2
        c = _norm("", dtype, T, Hq, Hk, D, rng.choice([0, 32, 16 * rng.randint(1, D // 16), D]),
                  rng.choice(["interleaved", "halves"]), rng.random() < 0.5)
    elif op == "append":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(2, 16000 // B))
        c = _append("", dtype, B, "%d:%d" % (rng.choice([hi, hi // 2, 0]), hi), "0:%d" % _log(rng, 1, 3000), mix,
                    Hk if Hk * D <= 2048 else 8, D, rng.choice([16, 32, 64, 128]),
                    rng.choice([0, 32, 16 * rng.randint(1, D // 16), D]), rng.choice(["interleaved", "halves"]),
                    rng.random() < 0.5)
    else:
        G = rng.choice([1, 2, 4, 5, 7, 8, 16])
        kb, ks = rng.choice([(1, 1), (1, 1), (1, 1), (32, 16), (4, 4)])
        if rng.random() < 0.5:  # decode, possibly of a few tokens each
            B, hi = _log(rng, 1, 100), rng.choice([1, 1, 1, rng.randint(2, 8)])
            ctx = _log(rng, 30, max(31, 200000 // B))
        else:
            B, hi = _log(rng, 1, 12), _log(rng, 9, 2500)
            ctx = _log(rng, 30, 12000)
        while B * hi * G * Hk * (ctx + hi) > 1.2e9 or B * (ctx + hi) * Hk * D > 4e8:
            hi, ctx = max(1, hi * 3 // 4), max(1, ctx * 3 // 4)
        c = _attn("", dtype, B, "%d:%d" % (hi if hi == 1 else rng.choice([hi, hi // 2, 0]), hi),
                  "%d:%d" % (rng.choice([0, ctx // 2]), ctx), mix, G * Hk, Hk, D, rng.choice([16, 32, 64, 128]),
                  window=rng.choice([0, 0, _log(rng, 8, 4000)]), key_block=kb, key_stride=ks)
    del c["name"]
    return c


def _lengths(case):
    """(tokens, positions before them) of every sequence: spread over the case's ranges, half of them over the
    logarithm where the range is wide; both ends occur."""
    rng = random.Random(case["mix"])
    out = []
    for key in ("lens", "ctx"):
        lo, hi = (int(v) for v in case[key].split(":"))
        vals = []
        for i in range(case["B"]):
            if hi > 10 * max(lo, 1) and rng.random() < 0.5:
                vals.append(min(hi, max(lo, int(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 1)))))))
            else:
                vals.append(rng.randint(lo, hi))
        vals[-1] = hi
        if len(vals) > 1:
            vals[0] = lo
        out.append(vals)
    lens, ctx = out
    rng.shuffle(ctx)
    return lens, ctx


def _keys(case, p1):
    """Keys visible to a token with p1 = its position + 1."""
    kb, ks = case["key_block"], case["key_stride"]
    return (p1 - kb) // ks + 1 if p1 >= kb else 0


# ---- inputs ---------------------------------------------------------------------------------


def _rope_tables(positions, rope, device):
    """cos and sin per token, [T, rope] float32; both halves hold the same angles (computed in 64 bits)."""
    inv = 10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64, device=device) / rope)
    ang = positions.double()[:, None] * inv[None, :]
    ang = torch.cat([ang, ang], 1)
    return ang.cos().float(), ang.sin().float()


def _tables(lens, page, g):
    """Pages drawn from one shuffled pool; entries past a sequence's end are -1. (block_table, pages in the pool)"""
    n = [max(1, -(-v // page)) for v in lens]
    pool = sum(n) + 3
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(max(n), device=DEV)[None, :]
    cnt = torch.tensor(n, device=DEV)[:, None]
    first = torch.cumsum(cnt, 0) - cnt
    return torch.where(col < cnt, perm[(first + col).clamp(max=pool - 1)], -1).to(torch.int32), pool


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    D = case["D"]
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    s = dict(case)
    if case["op"] == "qk_norm_rope":
        T, Hq, Hk = case["T"], case["Hq"], case["Hk"]
        gain = torch.exp(0.5 * randn(Hq + 2 * Hk, D))
        if case["packed"]:  # queries, keys and values of one projection, side by side
            qkv = (randn(T, Hq + 2 * Hk, D) * gain).to(dt)
            s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        else:
            s["q"], s["k"] = (randn(T, Hq, D) * gain[:Hq]).to(dt), (randn(T, Hk, D) * gain[Hq:Hq + Hk]).to(dt)
        s["q_weight"], s["k_weight"] = (1 + 0.1 * randn(D)).to(dt), (1 + 0.1 * randn(D)).to(dt)
        s["cos"] = s["sin"] = None
        if case["rope"]:
            s["cos"], s["sin"] = _rope_tables(torch.randint(0, 100000, (T,), generator=g, device=DEV), case["rope"], DEV)
        return s
    lens, ctx = _lengths(case)
    B, T = case["B"], sum(lens)
    s["T"], s["max_len"] = T, max(lens)
    s["cu_seqlens"] = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device=DEV)
    s["start_pos"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    if case["op"] == "append":
        held = [n + c for n, c in zip(lens, ctx)]
    else:
        held = [_keys(case, n + c) for n, c in zip(lens, ctx)]
        s["max_keys"] = max(held)
    s["block_table"], pool = _tables(held, case["page"], g)
    shape = (pool, case["page"], case["Hk"], D)
    s["k_cache"] = torch.randn(shape, generator=g, device=DEV, dtype=dt)
    s["v_cache"] = torch.randn(shape, generator=g, device=DEV, dtype=dt)
    if case["op"] == "append":
        s["k"], s["v"] = randn(T, case["Hk"], D).to(dt), randn(T, case["Hk"], D).to(dt)
        s["norm_weight"] = (1 + 0.1 * randn(D)).to(dt) if case["norm"] else None
        s["cos"] = s["sin"] = None
        if case["rope"]:
            s["cos"], s["sin"] = _rope_tables(_token_rows(s)[1], case["rope"], DEV)
    else:
        s["q"] = randn(T, case["Hq"], D).to(dt)
    return s


# ---- plain form -----------------------------------------------------------------------------


def _token_rows(s):
    """(sequence, position) of every token."""
    t = torch.arange(s["T"], device=DEV)
    cu = s["cu_seqlens"].long()
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return b, s["start_pos"].long()[b] + t - cu[b]


def _norm_rope(x, weight, cos, sin, pairs):
    """x [T, H, D] float32: RMS norm over D (if weight), then the rotation of the last cos.shape[1] channels."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    if cos is None:
        return x
    R = cos.shape[1]
    head, tail = x[..., :x.shape[-1] - R], x[..., x.shape[-1] - R:]
    a, b = (tail[..., 0::2], tail[..., 1::2]) if pairs == "interleaved" else (tail[..., :R // 2], tail[..., R // 2:])
    c, n = cos[:, None, :], sin[:, None, :]
    ra = a * c[..., :R // 2] - b * n[..., :R // 2]
    rb = b * c[..., R // 2:] + a * n[..., R // 2:]
    tail = torch.stack([ra, rb], -1).flatten(-2) if pairs == "interleaved" else torch.cat([ra, rb], -1)
    return torch.cat([head, tail], -1)


def _plain_append(s):
    b, pos = _token_rows(s)
    page = s["page"]
    row = s["block_table"][b, pos // page].long() * page + pos % page
    k = _norm_rope(s["k"].float(), s["norm_weight"], s["cos"], s["sin"], s["pairs"])
    s["k_cache"].view(-1, *k.shape[1:])[row] = k.to(s["k_cache"].dtype)
    s["v_cache"].view(-1, *k.shape[1:])[row] = s["v"]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    B, L, N, page = s["B"], s["max_len"], s["max_keys"], s["page"]
    Hk, D, G = s["Hk"], s["D"], s["Hq"] // s["Hk"]
    b, pos = _token_rows(s)
    col = pos - s["start_pos"].long()[b]
    q = torch.zeros(B, L, Hk, G, D, device=DEV)
    q[b, col] = s["q"].float().view(-1, Hk, G, D)
    key = torch.arange(N, device=DEV)
    rows = s["block_table"].long()[:, key // page].clamp(min=0) * page + key % page
    k, v = s["k_cache"].view(-1, Hk, D)[rows].float(), s["v_cache"].view(-1, Hk, D)[rows].float()
    p1 = s["start_pos"].long()[:, None] + torch.arange(1, L + 1, device=DEV)[None, :]
    n = torch.where(p1 >= s["key_block"], (p1 - s["key_block"]) // s["key_stride"] + 1, 0)
    seen = key < n[:, :, None]
    if s["window"]:
        seen &= key >= n[:, :, None] - s["window"]
    qh = q.permute(0, 2, 3, 1, 4).reshape(B, Hk, G * L, D)
    x = torch.matmul(qh, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(D)).view(B, Hk, G, L, N)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True) if N else x.new_full((B, Hk, G, L, 1), -math.inf)
    m = torch.where(m == -math.inf, 0.0, m)
    x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hk, G * L, N), v.permute(0, 2, 1, 3)).view(B, Hk, G, L, D)
    o = torch.where(z > 0, o / z, 0.0)
    lse = (m + z.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4)[b, col].reshape(-1, Hk * G, D)
    return {"out": o.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2)[b, col].reshape(-1, Hk * G)}


def _plain(s):
    if s["op"] == "append":
        return _plain_append(s)
    if s["op"] == "attention":
        return _plain_attention(s)
    return {name: _norm_rope(s[name].float(), s[name + "_weight"], s["cos"], s["sin"], s["pairs"]).to(s[name].dtype)
            for name in ("q", "k")}


def run(state):
    if not own:
        return _plain(state)
    import streaming_kv_cache_varlen_b200 as cmp

    s = state
    if s["op"] == "append":
        cmp.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_seqlens"], s["start_pos"],
                      norm_weight=s["norm_weight"], sin=s["sin"], cos=s["cos"], rope_pairs=s["pairs"], eps=EPS)
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "attention":
        out, lse = cmp.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_seqlens"],
                                       s["start_pos"], max_len=s["max_len"], window=s["window"] or None,
                                       key_block=s["key_block"], key_stride=s["key_stride"], return_lse=True)
        return {"out": out, "lse": lse}
    q, k = cmp.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], sin=s["sin"], cos=s["cos"],
                            rope_pairs=s["pairs"], eps=EPS)
    return {"q": q, "k": k}


# ---- work -----------------------------------------------------------------------------------


def work(case):
    D, R = case["D"], case.get("rope", 0)
    if case["op"] == "qk_norm_rope":
        n = case["T"] * (case["Hq"] + case["Hk"]) * D
        return {"bytes": 4 * n + 8 * case["T"] * R + 4 * D, "flops": 4 * n}
    lens, ctx = _lengths(case)
    T, Hk = sum(lens), case["Hk"]
    if case["op"] == "append":
        return {"bytes": 8 * T * Hk * D + 8 * T * R + 8 * case["B"], "flops": 4 * T * Hk * D}
    pairs = rows = 0
    for n, c in zip(lens, ctx):
        seen = [_keys(case, c + i + 1) for i in range(n)]
        w = case["window"] or 1 << 60
        pairs += sum(min(v, w) for v in seen)
        rows += seen[-1] - max(0, seen[0] - w) if n else 0
    return {"bytes": 4 * rows * Hk * D + 4 * T * case["Hq"] * D + 4 * T * case["Hq"], "flops": 4 * pairs * case["Hq"] * D}


# ---- the definition in 64 bits ----------------------------------------------------------------


def _exact_rows(x, weight, cos, sin, pairs):
    x = x.double()
    if weight is not None:
        x = weight.double() * x / torch.sqrt(EPS + torch.sum(x ** 2, dim=-1, keepdim=True) / x.shape[-1])
    if cos is None:
        return x
    R, D = cos.shape[1], x.shape[-1]
    j = torch.arange(R // 2, device=x.device)
    ia, ib = (D - R + 2 * j, D - R + 2 * j + 1) if pairs == "interleaved" else (D - R + j, D - R // 2 + j)
    y = x.clone()
    cos, sin = cos.double(), sin.double()
    y[:, :, ia] = x[:, :, ia] * cos[:, None, j] - x[:, :, ib] * sin[:, None, j]
    y[:, :, ib] = x[:, :, ib] * cos[:, None, R // 2 + j] + x[:, :, ia] * sin[:, None, R // 2 + j]
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk_norm_rope":
        return {n: _exact_rows(s[n], s[n + "_weight"], s["cos"], s["sin"], case["pairs"]) for n in ("q", "k")}
    lens, ctx = _lengths(case)
    page, D, Hk = case["page"], case["D"], case["Hk"]
    table = s["block_table"].cpu()
    at = 0
    if case["op"] == "append":
        k = _exact_rows(s["k"], s["norm_weight"], s["cos"], s["sin"], case["pairs"])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for i, (n, c) in enumerate(zip(lens, ctx)):
            done = 0
            while done < n:  # one page at a time
                p = c + done
                m = min(n - done, page - p % page)
                blk = int(table[i, p // page])
                kc[blk, p % page:p % page + m] = k[at + done:at + done + m]
                vc[blk, p % page:p % page + m] = s["v"][at + done:at + done + m].double()
                done += m
            at += n
        return {"k_cache": kc, "v_cache": vc}
    if work(case)["flops"] > 2.5e12:
        return None
    G = case["Hq"] // Hk
    out = torch.zeros(sum(lens), case["Hq"], D, dtype=torch.float64, device=DEV)
    lse = torch.full((sum(lens), case["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for i, (n, c) in enumerate(zip(lens, ctx)):
        N = _keys(case, c + n) if n else 0
        if N:
            pages = table[i, :-(-N // page)].long().to(DEV)
            kk, vv = (s[x][pages].reshape(-1, Hk, D)[:N].double() for x in ("k_cache", "v_cache"))
            kb, ks, w = case["key_block"], case["key_stride"], case["window"] or 1 << 40
            for t0 in range(0, n, 1024):
                t1 = min(n, t0 + 1024)
                p1 = torch.arange(c + t0 + 1, c + t1 + 1, device=DEV)
                cnt = torch.clamp(torch.div(p1 - kb, ks, rounding_mode="floor") + 1, min=0)
                key = torch.arange(N, device=DEV)
                hide = (key[None] >= cnt[:, None]) | (key[None] < cnt[:, None] - w)
                for h in range(Hk):
                    qq = s["q"][at + t0:at + t1, h * G:(h + 1) * G].double()
                    x = torch.einsum("tgd,nd->gtn", qq, kk[:, h]) / math.sqrt(D)
                    x = x.masked_fill(hide[None], -math.inf)
                    z = torch.logsumexp(x, -1)
                    p = torch.exp(x - z.masked_fill(z == -math.inf, 0.0)[..., None])
                    out[at + t0:at + t1, h * G:(h + 1) * G] = torch.einsum("gtn,nd->tgd", p, vv[:, h])
                    lse[at + t0:at + t1, h * G:(h + 1) * G] = z.t()
        at += n
    return {"out": out, "lse": lse}
