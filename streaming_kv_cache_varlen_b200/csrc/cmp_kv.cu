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
// with the lane R/16 away, an interleaved pair stays inside the lane. A warp takes
// a share of one token's heads, kUnroll heads per lane group with all their loads
// in flight, and keeps the token's table values (16-byte loads) and the weights in
// registers, two batches in turn; for kv_append it looks up its token's cache row meanwhile, so a CTA
// needs no barrier. 16384 tokens of 40 heads of 128, fully rotated, take 82 us (352 MB:
// 0.65 of the measured copy rate; one CTA per token with four-byte table loads took
// 112), the keys and values of 23000 tokens of 8 heads 47 us (214 MB, 0.69; 92).
#include "cmp_internal.cuh"

#include <cuda_fp16.h>

namespace cmp {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;  // heads a thread loads at once, while it computes as many others

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

// N (4 or 8) consecutive table values; i is a multiple of N.
template <int N>
__device__ __forceinline__ void rope_load(const RopeTable& r, const void* t, int64_t i, float (&f)[N]) {
  if (r.f32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(t) + i);
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const float4 v = __ldg(s + q);
      f[4 * q] = v.x;
      f[4 * q + 1] = v.y;
      f[4 * q + 2] = v.z;
      f[4 * q + 3] = v.w;
    }
  } else {
    const uint2* s = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(t) + i);
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const uint2 v = __ldg(s + q);
      f[4 * q] = __uint_as_float(v.x << 16);
      f[4 * q + 1] = __uint_as_float(v.x & 0xFFFF0000u);
      f[4 * q + 2] = __uint_as_float(v.y << 16);
      f[4 * q + 3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
  }
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
    rope_load<8>(r, r.cos, row + k, o.c);
    rope_load<8>(r, r.sin, row + k, o.s);
    if (!second) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o.s[e] = -o.s[e];
    }
  } else {
    float ca[4], cb[4], sa[4], sb[4];
    rope_load<4>(r, r.cos, row + k / 2, ca);
    rope_load<4>(r, r.cos, row + R / 2 + k / 2, cb);
    rope_load<4>(r, r.sin, row + k / 2, sa);
    rope_load<4>(r, r.sin, row + R / 2 + k / 2, sb);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o.c[2 * e] = ca[e];
      o.c[2 * e + 1] = cb[e];
      o.s[2 * e] = -sa[e];
      o.s[2 * e + 1] = sb[e];
    }
  }
}

// Sum over the LPH lanes of a head, in all of them.
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, LPH);
  return v;
}

// Mean squares (plus eps) between which no square of weight has left fp32's range.
// Beyond, a head of bf16 values is scaled by a power of two, which is exact and cancels.
// Above: some channel is 2^60 or more, so with 2^-70 the largest square lies in
// 2^-20 .. 2^116. Below (only with an eps below 1e-30): every channel is under 2^-46, so
// with 2^80 the squares lie in 2^-106 (bf16's smallest number) .. 2^68. Asking costs 3 %
// (16384 tokens of 40 heads of 128: 82.3 us, 79.9 without); asking once for two or four
// heads, which all have to be kept for it, takes 86 and 84.6.
constexpr float kMeanSquareMin = 1e-30f, kMeanSquareMax = 3.4028234e38f;
constexpr float kScaleDown = 0x1p-70f, kScaleUp = 0x1p80f;

// One head's 8 channels per lane: norm (with the weights wv, if normed) and
// rotation. Every lane of the warp takes part; lanes past D hold zeros.
template <bool BF16, int LPH>
__device__ __forceinline__ void norm_rope(float (&x)[8], bool normed, const uint4& wv, float inv_d, float eps,
                                          const RopeTable& r, const LaneRope& lr, int lane) {
  if (normed) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
    const float ms = fmaf(head_sum<LPH>(ss), inv_d, eps);
    float sc = rsqrtf(ms);
    // fp16's squares stay in range (2^-48 to 2^32)
    if (BF16 && __any_sync(0xffffffffu, !(ms >= kMeanSquareMin && ms <= kMeanSquareMax))) {
      const float f = ms > kMeanSquareMax ? kScaleDown : ms < kMeanSquareMin ? kScaleUp : 1.f;
      ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= f;
        ss = fmaf(x[e], x[e], ss);
      }
      sc = rsqrtf(fmaf(head_sum<LPH>(ss), inv_d, eps * f * f));
    }
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

// Grid (token quadruples, head splits): warp w of CTA (x, y) takes share y of the
// heads (queries, then keys) of token 4 x + w.
template <bool BF16, int LPH>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const QkNormParams p, int share) {
  constexpr int kGroups = 32 / LPH;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int lane = threadIdx.x % LPH, g = (threadIdx.x & 31) / LPH;
  const int c0 = lane * 8;
  const bool live = c0 < p.D;
  const int heads = min(p.Hq + p.Hk, ((int)blockIdx.y + 1) * share);
  const uint16_t* qrow = p.q + t * p.q_stride + c0;
  const uint16_t* krow = p.k + t * p.k_stride + c0;
  auto load = [&](uint4 (&v)[kUnroll], int h0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kGroups;
      v[u] = make_uint4(0, 0, 0, 0);
      if (live && h < heads)
        v[u] = *reinterpret_cast<const uint4*>(h < p.Hq ? qrow + (int64_t)h * p.D : krow + (int64_t)(h - p.Hq) * p.D);
    }
  };
  int h0 = blockIdx.y * share + g;
  uint4 va[kUnroll], vb[kUnroll];
  load(va, h0);
  LaneRope lr;
  load_rope(p.rope, t, lane, c0, p.D, lr);
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (live) {
    wq = __ldg(reinterpret_cast<const uint4*>(p.q_weight + c0));
    if (p.Hk) wk = __ldg(reinterpret_cast<const uint4*>(p.k_weight + c0));
  }
  uint16_t* qdst = p.q_out + t * p.qo_stride + c0;
  uint16_t* kdst = p.k_out + t * p.ko_stride + c0;
  auto store = [&](const uint4 (&v)[kUnroll], int h0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kGroups;
      if (h - g >= heads) break;  // uniform: no group of the warp has a head left
      float x[8];
      unpack8<BF16>(v[u], x);
      norm_rope<BF16, LPH>(x, true, h < p.Hq ? wq : wk, p.inv_d, p.eps, p.rope, lr, lane);
      if (live && h < heads)
        *reinterpret_cast<uint4*>(h < p.Hq ? qdst + (int64_t)h * p.D : kdst + (int64_t)(h - p.Hq) * p.D) =
            pack8<BF16>(x);
    }
  };
  constexpr int kStep = kGroups * kUnroll;
  for (;;) {  // two buffers, so that a store's loads were issued a round before
    if (h0 + kStep - g < heads) load(vb, h0 + kStep);
    store(va, h0);
    h0 += kStep;
    if (h0 - g >= heads) return;
    if (h0 + kStep - g < heads) load(va, h0 + kStep);
    store(vb, h0);
    h0 += kStep;
    if (h0 - g >= heads) return;
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

// Grid (token quadruples + 1, head splits): warp w of CTA (x, y) stores share y of
// the heads (keys, then values) of token 4 x + w; the last CTA of a row of the grid
// checks cu_seqlens as a whole.
template <bool BF16, int LPH>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendParams p, int share) {
  constexpr int kGroups = 32 / LPH;
  if (blockIdx.x == gridDim.x - 1) {
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
  if ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5) >= p.T) return;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int wl = threadIdx.x & 31;
  const int lane = wl % LPH, g = wl / LPH;
  const int c0 = lane * 8;
  const bool live = c0 < p.D;
  const int heads = min(2 * p.Hk, ((int)blockIdx.y + 1) * share);
  const uint16_t* krow = p.k + (int64_t)t * p.k_stride + c0;
  const uint16_t* vrow = p.v + (int64_t)t * p.v_stride + c0;
  // the first heads and the table row do not depend on the sequence: load them
  // while it is looked up
  int h0 = blockIdx.y * share + g;
  auto load = [&](uint4 (&v)[kUnroll], int h0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kGroups;
      v[u] = make_uint4(0, 0, 0, 0);
      if (live && h < heads)
        v[u] = *reinterpret_cast<const uint4*>(h < p.Hk ? krow + (int64_t)h * p.D : vrow + (int64_t)(h - p.Hk) * p.D);
    }
  };
  constexpr int kStep = kGroups * kUnroll;
  uint4 va[kUnroll], vb[kUnroll];
  load(va, h0);
  if (h0 + kStep - g < heads) load(vb, h0 + kStep);
  const bool normed = p.norm_weight != nullptr;
  LaneRope lr;
  lr.on = false;
  lr.partner = lane;
  uint4 wk = make_uint4(0, 0, 0, 0);
  if (h0 - g < p.Hk) {  // the share holds keys
    load_rope(p.rope, t, lane, c0, p.D, lr);
    if (live && normed) wk = __ldg(reinterpret_cast<const uint4*>(p.norm_weight + c0));
  }
  const int b = warp_find_seq(p.cu, p.B, t, wl);
  const int c = __ldg(p.cu + b), e = __ldg(p.cu + b + 1);
  if (t < c || t >= e) return;  // behind the last sequence: nothing to store
  const int64_t pos = (int64_t)(p.start_pos ? __ldg(p.start_pos + b) : 0) + (t - c);
  int64_t row = -1;
  if (pos >= t - c && pos < INT32_MAX) {
    const int pg = p.div_page.div((int)pos);
    if (pg < p.table_stride) {
      const int blk = __ldg(p.table + (int64_t)b * p.table_stride + pg);
      if (blk >= 0 && blk < p.block_num) row = (int64_t)blk * p.page + ((int)pos - pg * p.page);
    }
  }
  if (row < 0) {
    if (wl == 0) atomicOr(&g_kv_err, kErrIndex);
    return;
  }
  uint16_t* kdst = p.k_cache + row * p.Hk * p.D + c0;
  uint16_t* vdst = p.v_cache + row * p.Hk * p.D + c0;
  auto store = [&](const uint4 (&v)[kUnroll], int h0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kGroups;
      if (h - g >= heads) break;
      uint4 o = v[u];
      if (h - g < p.Hk) {  // the warp's first group decides whether any of its heads is a key
        float x[8];
        unpack8<BF16>(v[u], x);
        norm_rope<BF16, LPH>(x, normed, wk, p.inv_d, p.eps, p.rope, lr, lane);
        if (h < p.Hk) o = pack8<BF16>(x);
      }
      if (live && h < heads)
        *reinterpret_cast<uint4*>(h < p.Hk ? kdst + (int64_t)h * p.D : vdst + (int64_t)(h - p.Hk) * p.D) = o;
    }
  };
  for (;;) {
    store(va, h0);
    if (h0 + 2 * kStep - g < heads) load(va, h0 + 2 * kStep);
    h0 += kStep;
    if (h0 - g >= heads) return;
    store(vb, h0);
    if (h0 + 2 * kStep - g < heads) load(vb, h0 + 2 * kStep);
    h0 += kStep;
    if (h0 - g >= heads) return;
  }
}

// Heads per warp: a token's, fewer when the call is too small to give every SM a few
// warps that way (a decode step).
int head_share(int64_t T, int heads, int lph, int sms) {
  const int groups = 32 / lph;
  const int64_t wanted = (8 * (int64_t)sms + T - 1) / T;  // warps per token
  const int rounds = (heads + groups - 1) / groups;       // of the lane groups
  const int splits = (int)(wanted < rounds ? wanted : rounds);
  return (rounds + splits - 1) / splits * groups;
}

template <bool BF16, int LPH>
cudaError_t run_norm(const QkNormParams& p, cudaStream_t s, int sms) {
  const int heads = p.Hq + p.Hk, share = head_share(p.T, heads, LPH, sms);
  const dim3 grid((unsigned)((p.T + kWarps - 1) / kWarps), (unsigned)((heads + share - 1) / share));
  qk_norm_rope_kernel<BF16, LPH><<<grid, kThreads, 0, s>>>(p, share);
  return cudaGetLastError();
}

template <bool BF16, int LPH>
cudaError_t run_append(const KvAppendParams& p, cudaStream_t s, int sms) {
  const int heads = 2 * p.Hk, share = head_share(p.T, heads, LPH, sms);
  const dim3 grid((unsigned)((p.T + kWarps - 1) / kWarps + 1), (unsigned)((heads + share - 1) / share));
  kv_append_kernel<BF16, LPH><<<grid, kThreads, 0, s>>>(p, share);
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

// The error word of the current device's kv_append calls.
cudaError_t kv_error_word(unsigned** word) { return cudaGetSymbolAddress((void**)word, g_kv_err); }

}  // namespace cmp
