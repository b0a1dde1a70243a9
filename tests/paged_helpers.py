"""Helpers for the GPU tests of the paged cache operators.

Tolerances, per element (u = 2^-24, h = eps / 2 of the dtype: one rounding, t the
smallest half step of the dtype, which subnormal results can be off by):

* norm and rotation: at most 16 u of relative error in the normed value (13
  additions under the square root count half, the mean's two roundings half, rsqrt
  4, two products), 2 u more for the rotation's product and fma, on the magnitude of
  the terms; then one rounding:  |y - ref| <= h |ref| + 20 u mag + t.
* attention: a score is a sum of D exact products with an fp32 accumulator (at
  worst 2 u per term, as truncating accumulators have) and three more roundings of a
  value up to score_mag:  ds = (2 D + 8) u score_mag. A weight is then off by a relative
  w = ds + 8 u (the exponential's 2^-22 and its argument), is rounded once for the
  product (h), and counts in numerator and denominator; both sums have at most n + 64
  terms (n keys, the joins of warps and pieces):
  |out - ref| <= h |ref| + weight_mag (h + 2 w + 4 (n + 64) u) + t (1 + sum |v|),
  the last term for weights below the dtype's normal range (relative to a sum of at
  least 1), and |lse - ref| <= w + (n + 64) u + 4 u |lse|.
"""

import numpy as np

from oracle.nsa import to_bits, to_f64

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}


def b16(a, dtype, device="cuda"):
    import torch
    dt = torch.float16 if dtype == "fp16" else torch.bfloat16
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(device).view(dt)


def dev(a, device="cuda"):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(device)


def bits(t):
    import torch
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def assert_normed(got_bits, ref, mag, dtype):
    g = to_f64(got_bits, dtype)
    lim = HALF[dtype] * np.abs(ref) * (1 + 1e-9) + 20 * U * mag * (1 + HALF[dtype]) + TINY[dtype]
    bad = ~(np.abs(g - ref) <= lim)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, worst {float((np.abs(g - ref) / lim).max()):.3g} x"


def attention_limits(res, D, dtype):
    h = HALF[dtype]
    w = (2 * D + 8) * U * res.score_mag + 8 * U
    n = (res.n + 64)[:, None].astype(np.float64)
    lim = h * np.abs(res.out) + res.weight_mag * (h + 2 * w + 4 * n * U)[..., None] * (1 + h) + TINY[dtype] * (
        1 + res.v_mag)
    lse = w + n * U + 4 * U * np.abs(np.where(np.isfinite(res.lse), res.lse, 0.0))
    return lim, lse


def assert_attention(got_bits, got_lse, res, dtype):
    """Rows of sequences against the oracle; rows that see no key exactly 0 and -inf."""
    r = res.rows
    g = to_f64(got_bits, dtype)[r]
    lim, lim_lse = attention_limits(res, got_bits.shape[-1], dtype)
    err = np.abs(g - res.out[r])
    bad = ~(err <= lim[r])
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outputs off, worst {np.nanmax(err / lim[r]):.3g} x the limit"
    empty = res.n == 0
    assert np.all(got_bits[r & empty] == 0)
    if got_lse is not None:
        assert np.all(np.isneginf(got_lse[r & empty]))
        f = r & ~empty
        d = np.abs(got_lse[f].astype(np.float64) - res.lse[f])
        assert np.all(d <= lim_lse[f]), f"lse off, worst {float((d / lim_lse[f]).max()):.3g} x the limit"


def round16(v, dtype):
    """float64 -> exact values of the dtype."""
    return to_f64(to_bits(v, dtype), dtype)
