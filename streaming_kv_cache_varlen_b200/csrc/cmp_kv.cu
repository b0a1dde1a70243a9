// Queries, keys and values on their way to the paged cache: qk_norm_rope (RMS
// norm of every head, then the position rotation) and kv_append (the same on a
// key, then keys and values stored at their sequence's next cache rows).
//
//   y_c = x_c * w_c / sqrt(mean_c x_c^2 + eps)                  (if normed)
//   of the last R channels, the pair (a, b) with table columns j and R/2 + j:
//   a' = a cos_j - b sin_j,   b' = b cos_{R/2+j} + a sin_{R/2+j}
//   interleaved pairs: channels (2j, 2j+1); halves: channels (j, R/2 + j)
// (the table convention of the Compressor's RoPE). All in fp32, one rounding to
// the output type at the end.
//
// HBM bound: each element is read once and written once. A head's D channels
// lie on LPH lanes of one warp, 8 consecutive channels (one 16-byte access) per
// lane, so the sum of squares is log2(LPH) shuffles; a halves pair is exchanged
// with the lane R/16 away, an interleaved pair stays inside the lane. A thread
// keeps its token's table values and weights in registers and runs over the
// token's heads, four heads' loads in flight at a time.
#include "cmp_internal.cuh"

#include <cuda_fp16.h>

namespace cmp {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;  // heads whose loads a thread has in flight

__device__ unsigned g_kv_err;  // error word of kv_append on this device

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float rope_at(const RopeTable& r, const void* t, int64_t i) {
  return r.f32 ? __ldg(static_cast<const float*>(t) + i)
               : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(t) + i) << 16);
}

// A lane's part of its token's rotation: y[e] = x[e] * c[e] + partner[e] * s[e]
// for the lane's 8 channels (the sign of the pair's first element folded into s).
struct LaneRope {
  float c[8], s[8];
  int partner;  // halves: lane within the head's group that holds the partners
  bool on;      // the lane's channels are rotated
};

// Channels c0 .. c0 + 7 of a head of D, table row `token`. R is a multiple of 16
// and D - R one of 16, so a lane's channels are rotated together or not at all.
__device__ __forceinline__ void load_rope(const RopeTable& r, int64_t token, int lane, int c0, int D, LaneRope& o) {
  const int R = r.dim;
  const int k = c0 - (D - R);  // first channel within the rotated part
  o.on = R > 0 && k >= 0 && c0 < D;
  o.partner = lane;
  if (!o.on) return;
  const int64_t row = token * R;
  if (r.halves) {
    const bool second = k >= R / 2;
    o.partner = second ? lane - R / 16 : lane + R / 16;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o.c[e] = rope_at(r, r.cos, row + k + e);
      const float s = rope_at(r, r.sin, row + k + e);
      o.s[e] = second ? s : -s;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o.c[2 * e] = rope_at(r, r.cos, row + k / 2 + e);
      o.s[2 * e] = -rope_at(r, r.sin, row + k / 2 + e);
      o.c[2 * e + 1] = rope_at(r, r.cos, row + R / 2 + k / 2 + e);
      o.s[2 * e + 1] = rope_at(r, r.sin, row + R / 2 + k / 2 + e);
    }
  }
}

// One head's 8 channels per lane: norm (with the weights wv, if normed) and
// rotation. Every lane of the warp takes part; lanes past D hold zeros.
template <bool BF16, int LPH>
__device__ __forceinline__ void norm_rope(float (&x)[8], bool normed, const uint4& wv, float inv_d, float eps,
                                          const RopeTable& r, const LaneRope& lr, int lane) {
  if (normed) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, LPH);
    const float sc = rsqrtf(fmaf(ss, inv_d, eps));
    float w[8];
    unpack8<BF16>(wv, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * sc * w[e];
  }
  if (r.dim == 0) return;
  float y[8];
  if (r.halves) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], lr.partner, LPH);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
  }
  if (lr.on) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(y[e], lr.s[e], x[e] * lr.c[e]);
  }
}

// Grid (tokens, head splits). The heads of a token (queries, then keys) go
// round the groups of LPH lanes of its gridDim.y CTAs.
template <bool BF16, int LPH>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const QkNormParams p) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % LPH;
  const int c0 = lane * 8;
  const bool live = c0 < p.D;
  const int groups = (kThreads / LPH) * gridDim.y;
  const int g = blockIdx.y * (kThreads / LPH) + threadIdx.x / LPH;
  const int heads = p.Hq + p.Hk;
  const uint16_t* qrow = p.q + t * p.q_stride + c0;
  const uint16_t* krow = p.k + t * p.k_stride + c0;
  LaneRope lr;
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  bool have = false;
  for (int h0 = 0; h0 < heads; h0 += groups * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * groups + g;
      v[u] = make_uint4(0, 0, 0, 0);
      if (live && h < heads)
        v[u] = *reinterpret_cast<const uint4*>(h < p.Hq ? qrow + (int64_t)h * p.D : krow + (int64_t)(h - p.Hq) * p.D);
    }
    if (!have) {  // after the first heads' loads are on their way
      have = true;
      load_rope(p.rope, t, lane, c0, p.D, lr);
      if (live) {
        wq = __ldg(reinterpret_cast<const uint4*>(p.q_weight + c0));
        if (p.Hk) wk = __ldg(reinterpret_cast<const uint4*>(p.k_weight + c0));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h0 + u * groups >= heads) break;  // uniform: no group has a head left
      const int h = h0 + u * groups + g;
      float x[8];
      unpack8<BF16>(v[u], x);
      norm_rope<BF16, LPH>(x, true, h < p.Hq ? wq : wk, p.inv_d, p.eps, p.rope, lr, lane);
      if (live && h < heads) {
        uint16_t* o = h < p.Hq ? p.q_out + t * p.qo_stride + (int64_t)h * p.D
                               : p.k_out + t * p.ko_stride + (int64_t)(h - p.Hq) * p.D;
        *reinterpret_cast<uint4*>(o + c0) = pack8<BF16>(x);
      }
    }
  }
}

// The sequence of token t, found by a whole warp: the largest b in [0, B) with
// cu[b] <= t, 32 probes at a time, so that a batch of up to 1024 sequences takes
// two dependent loads (a binary search takes ten). cu[0] <= t is assumed.
__device__ __forceinline__ int warp_find_seq(const int32_t* cu, int B, int t, int lane) {
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < n && __ldg(cu + i) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Grid (tokens + 1, head splits): CTA x < T stores token x (its keys, then its
// values, go round the groups), the CTA at x = T checks cu_seqlens as a whole.
template <bool BF16, int LPH>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendParams p) {
  if ((int64_t)blockIdx.x == p.T) {
    if (blockIdx.y == 0) {
      bool bad = threadIdx.x == 0 && __ldg(p.cu) != 0;
      for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int c = __ldg(p.cu + b), e = __ldg(p.cu + b + 1);
        bad = bad || e < c || e > p.T;
      }
      if (bad) atomicOr(&g_kv_err, kErrIndex);
    }
    return;
  }
  const int t = blockIdx.x;
  const int wl = threadIdx.x & 31;
  const int lane = threadIdx.x % LPH;
  const int c0 = lane * 8;
  const bool live = c0 < p.D;
  const int groups = (kThreads / LPH) * gridDim.y;
  const int g = blockIdx.y * (kThreads / LPH) + threadIdx.x / LPH;
  const int heads = 2 * p.Hk;
  const uint16_t* krow = p.k + (int64_t)t * p.k_stride + c0;
  const uint16_t* vrow = p.v + (int64_t)t * p.v_stride + c0;
  // the first heads and the table row do not depend on the sequence: load them
  // while it is looked up
  uint4 v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int h = u * groups + g;
    v[u] = make_uint4(0, 0, 0, 0);
    if (live && h < heads)
      v[u] = *reinterpret_cast<const uint4*>(h < p.Hk ? krow + (int64_t)h * p.D : vrow + (int64_t)(h - p.Hk) * p.D);
  }
  LaneRope lr;
  load_rope(p.rope, t, lane, c0, p.D, lr);
  uint4 wk = make_uint4(0, 0, 0, 0);
  const bool normed = p.norm_weight != nullptr;
  if (live && normed) wk = __ldg(reinterpret_cast<const uint4*>(p.norm_weight + c0));
  const int b = warp_find_seq(p.cu, p.B, t, wl);
  const int c = __ldg(p.cu + b), e = __ldg(p.cu + b + 1);
  if (t < c || t >= e) return;  // behind the last sequence: nothing to store
  const int64_t pos = (int64_t)(p.start_pos ? __ldg(p.start_pos + b) : 0) + (t - c);
  int64_t row = -1;
  if (pos >= t - c && pos < INT32_MAX) {
    const int64_t pg = pos / p.page;
    if (pg < p.table_stride) {
      const int blk = __ldg(p.table + (int64_t)b * p.table_stride + pg);
      if (blk >= 0 && blk < p.block_num) row = (int64_t)blk * p.page + pos % p.page;
    }
  }
  if (row < 0) {
    if (threadIdx.x == 0) atomicOr(&g_kv_err, kErrIndex);
    return;
  }
  uint16_t* kdst = p.k_cache + row * p.Hk * p.D + c0;
  uint16_t* vdst = p.v_cache + row * p.Hk * p.D + c0;
  for (int h0 = 0;;) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h0 + u * groups >= heads) break;
      const int h = h0 + u * groups + g;
      uint4 o = v[u];
      // the warp's first group decides whether any of its heads is a key
      if (h0 + u * groups + (g - (wl / LPH)) < p.Hk) {
        float x[8];
        unpack8<BF16>(v[u], x);
        norm_rope<BF16, LPH>(x, normed, wk, p.inv_d, p.eps, p.rope, lr, lane);
        if (h < p.Hk) o = pack8<BF16>(x);
      }
      if (live && h < heads)
        *reinterpret_cast<uint4*>(h < p.Hk ? kdst + (int64_t)h * p.D : vdst + (int64_t)(h - p.Hk) * p.D) = o;
    }
    h0 += groups * kUnroll;
    if (h0 >= heads) return;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * groups + g;
      if (live && h < heads)
        v[u] = *reinterpret_cast<const uint4*>(h < p.Hk ? krow + (int64_t)h * p.D : vrow + (int64_t)(h - p.Hk) * p.D);
    }
  }
}

// CTAs per token: enough that a small call covers the SMs, never more than its
// heads can feed.
int head_splits(int64_t T, int heads, int lph, int sms) {
  const int per_cta = kThreads / lph;
  const int most = (heads + per_cta - 1) / per_cta;
  int64_t want = (2 * (int64_t)sms + T - 1) / (T > 0 ? T : 1);
  return (int)(want < 1 ? 1 : want > most ? most : want);
}

template <bool BF16, int LPH>
cudaError_t run_norm(const QkNormParams& p, cudaStream_t s, int sms) {
  const dim3 grid((unsigned)p.T, (unsigned)head_splits(p.T, p.Hq + p.Hk, LPH, sms));
  qk_norm_rope_kernel<BF16, LPH><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <bool BF16, int LPH>
cudaError_t run_append(const KvAppendParams& p, cudaStream_t s, int sms) {
  const dim3 grid((unsigned)(p.T + 1), (unsigned)head_splits(p.T, 2 * p.Hk, LPH, sms));
  kv_append_kernel<BF16, LPH><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormParams& p, cudaStream_t s, int sms) {
  const int l = (p.D + 7) / 8;
  if (p.bf16) {
    if (l <= 2) return run_norm<true, 2>(p, s, sms);
    if (l <= 4) return run_norm<true, 4>(p, s, sms);
    if (l <= 8) return run_norm<true, 8>(p, s, sms);
    if (l <= 16) return run_norm<true, 16>(p, s, sms);
    return run_norm<true, 32>(p, s, sms);
  }
  if (l <= 2) return run_norm<false, 2>(p, s, sms);
  if (l <= 4) return run_norm<false, 4>(p, s, sms);
  if (l <= 8) return run_norm<false, 8>(p, s, sms);
  if (l <= 16) return run_norm<false, 16>(p, s, sms);
  return run_norm<false, 32>(p, s, sms);
}

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t s, int sms) {
  const int l = (p.D + 7) / 8;
  if (p.bf16) {
    if (l <= 2) return run_append<true, 2>(p, s, sms);
    if (l <= 4) return run_append<true, 4>(p, s, sms);
    if (l <= 8) return run_append<true, 8>(p, s, sms);
    if (l <= 16) return run_append<true, 16>(p, s, sms);
    return run_append<true, 32>(p, s, sms);
  }
  if (l <= 2) return run_append<false, 2>(p, s, sms);
  if (l <= 4) return run_append<false, 4>(p, s, sms);
  if (l <= 8) return run_append<false, 8>(p, s, sms);
  if (l <= 16) return run_append<false, 16>(p, s, sms);
  return run_append<false, 32>(p, s, sms);
}

// The error word of the current device's kv_append calls, read and cleared.
cudaError_t kv_take_error(unsigned* word) { return take_symbol_word(g_kv_err, word); }

}  // namespace cmp
