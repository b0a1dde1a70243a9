// Joins the pieces of the attention items that were cut between CTAs (see
// cmp_attn.cuh). Piece i of a row left its accumulator o_i, its reference
// maximum m_i (log2 units) and its sum l_i:
//   M = max m_i,  l = sum l_i 2^(m_i - M),  o = sum o_i 2^(m_i - M) / l.
// A CTA per (CTA c of the attention kernel, group of rows): it looks at the item
// that c began and did not end, if there is one. The pieces are added in a fixed
// order, so the result does not depend on timing.
//
// Decoding has few rows of many pieces: a CTA takes a row, each of its four warps
// every fourth piece, lanes over the channels (29 us with one warp per row, after a
// step whose longest sequence has 100000 keys; 8 us). Bound by latency: the note, the
// statistics (a lane per piece), the accumulators (eight pieces of a warp in flight)
// and the store follow one another, all but the last from L2.
//
// Chunks have 256 rows of few pieces: a CTA takes 64 channels of 32 rows, a lane per
// row, its warps every fourth group of four channels; the rows leave through shared
// memory.
#include "cmp_attn.cuh"

namespace cmp {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreads) attn_combine_kernel(const AttnParams p, int m_rows) {
  constexpr int V = DP / 32;  // channels per lane: 2, 4, 6 or 8, as DP / 64 float2
  __shared__ float2 part[kWarps][DP / 2];
  __shared__ float sums[kWarps];
  const int c = blockIdx.x, r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const int4 d0 = p.desc[2 * c];
  const int n = d0.x - c + 1, rows = d0.y, t0 = d0.z, row0 = d0.w;
  if (d0.x == 0 || r >= rows) return;
  const int h = p.desc[2 * c + 1].x;
  // piece 0 is CTA c's slot 1, piece i > 0 CTA c + i's slot 0
  auto base = [&](int i) { return ((int64_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * m_rows + r; };
  float mx = neg_inf();
  for (int i = lane; i < n; i += 32) mx = fmaxf(mx, p.part_ml[base(i) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ref = mx == neg_inf() ? 0.f : mx;
  float2 acc[V / 2];
#pragma unroll
  for (int v = 0; v < V / 2; ++v) acc[v] = make_float2(0.f, 0.f);
  float l = 0.f;
#pragma unroll 8
  for (int i = warp; i < n; i += kWarps) {
    const int64_t b = base(i);
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + b * 2);
    const float w = ex2(ml.x - ref);
    l = fmaf(ml.y, w, l);
#pragma unroll
    for (int v = 0; v < V / 2; ++v) {
      const float2 x = *reinterpret_cast<const float2*>(p.part + b * DP + v * 64 + lane * 2);
      acc[v].x = fmaf(x.x, w, acc[v].x);
      acc[v].y = fmaf(x.y, w, acc[v].y);
    }
  }
#pragma unroll
  for (int v = 0; v < V / 2; ++v) part[warp][v * 32 + lane] = acc[v];
  if (lane == 0) sums[warp] = l;
  __syncthreads();
  l = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t row = attn_out_row(p, t0, h, row0 + r);
  const int t = threadIdx.x;
  if (t < DP / 2 && t * 2 < p.D) {
    const float2 a = part[0][t], b = part[1][t], e = part[2][t], f = part[3][t];
    *reinterpret_cast<uint32_t*>(p.out + row * p.D + t * 2) =
        pack2<BF16>(((a.x + b.x) + (e.x + f.x)) * inv, ((a.y + b.y) + (e.y + f.y)) * inv);
  }
  if (t == 0 && p.lse) p.lse[row] = attn_lse(mx, l);
}

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreads) attn_combine_chunk_kernel(const AttnParams p, int m_rows) {
  constexpr int kPitch = 9;  // 16-byte chunks per row of 64 channels, one of padding against bank conflicts
  __shared__ uint4 tile[32][kPitch];
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const int4 d0 = p.desc[2 * c];
  const int n = d0.x - c + 1, rows = d0.y, t0 = d0.z, row0 = d0.w, r0 = blockIdx.y * 32;
  const int d0c = blockIdx.z * 16;  // first group of four channels
  if (d0.x == 0 || r0 >= rows) return;
  const int h = p.desc[2 * c + 1].x;
  const int r = min(r0 + lane, rows - 1);  // lanes behind the last row repeat it and write nothing
  auto slot = [&](int i) { return (int64_t)(c + i) * 2 + (i == 0 ? 1 : 0); };
  auto stat = [&](int i) { return *reinterpret_cast<const float2*>(p.part_ml + (slot(i) * m_rows + r) * 2); };
  float mx = neg_inf();
#pragma unroll 4
  for (int i = 0; i < n; ++i) mx = fmaxf(mx, stat(i).x);
  const float ref = mx == neg_inf() ? 0.f : mx;
  float l = 0.f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float2 ml = stat(i);
    l = fmaf(ml.y, ex2(ml.x - ref), l);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float4 acc[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float w = ex2(stat(i).x - ref);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c4 = d0c + q * kWarps + warp;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c4 * 4 < p.D) x = *reinterpret_cast<const float4*>(attn_chunk_part(p, DP, m_rows, slot(i), c4, r));
      acc[q].x = fmaf(x.x, w, acc[q].x);
      acc[q].y = fmaf(x.y, w, acc[q].y);
      acc[q].z = fmaf(x.z, w, acc[q].z);
      acc[q].w = fmaf(x.w, w, acc[q].w);
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int c4 = q * kWarps + warp;
    reinterpret_cast<uint2*>(tile[lane])[c4] = make_uint2(pack2<BF16>(acc[q].x * inv, acc[q].y * inv),
                                                          pack2<BF16>(acc[q].z * inv, acc[q].w * inv));
  }
  if (warp == 0 && d0c == 0 && r0 + lane < rows && p.lse) p.lse[attn_out_row(p, t0, h, row0 + r)] = attn_lse(mx, l);
  __syncthreads();
#pragma unroll
  for (int i = threadIdx.x; i < 32 * 8; i += kThreads) {
    const int x = i / 8, ch = i % 8, d = d0c * 4 + ch * 8;
    if (r0 + x < rows && d < p.D)
      *reinterpret_cast<uint4*>(p.out + attn_out_row(p, t0, h, row0 + r0 + x) * p.D + d) = tile[x][ch];
  }
}

template <bool BF16, int DP>
cudaError_t run(const AttnParams& p, int m, int ctas, cudaStream_t s) {
  if (m <= 16)
    return launch_chained(attn_combine_kernel<BF16, DP>, dim3((unsigned)ctas, (unsigned)m), dim3(kThreads), 0, s, 1, p,
                          m);
  return launch_chained(attn_combine_chunk_kernel<BF16, DP>, dim3((unsigned)ctas, (unsigned)(m / 32), DP / 64),
                        dim3(kThreads), 0,
                        s, 1, p, m);
}

}  // namespace

cudaError_t launch_attn_combine(const AttnParams& p, int m, int ctas, cudaStream_t s) {
  switch (attn_padded(p.D) / 64 * 2 + (p.bf16 ? 1 : 0)) {
    case 2: return run<false, 64>(p, m, ctas, s);
    case 3: return run<true, 64>(p, m, ctas, s);
    case 4: return run<false, 128>(p, m, ctas, s);
    case 5: return run<true, 128>(p, m, ctas, s);
    case 6: return run<false, 192>(p, m, ctas, s);
    case 7: return run<true, 192>(p, m, ctas, s);
    case 8: return run<false, 256>(p, m, ctas, s);
    default: return run<true, 256>(p, m, ctas, s);
  }
}

}  // namespace cmp
