// Joins the pieces of the attention items that were cut between CTAs (see
// cmp_attn.cuh). Piece i of a row left its accumulator o_i, its reference
// maximum m_i (log2 units) and its sum l_i:
//   M = max m_i,  l = sum l_i 2^(m_i - M),  o = sum o_i 2^(m_i - M) / l.
// A CTA per (CTA c of the attention kernel, group of rows): it looks at the item
// that c began and did not end, if there is one. W warps take a row, every W-th
// piece each, lanes over the channels, and their sums are added in warp order, so
// the result does not depend on timing. Bound by latency: the note, the statistics
// (a lane per piece), the accumulators (eight pieces of a warp in flight) and the
// store follow one another, all but the last from L2. Decoding has few rows of many
// pieces, so four warps share one (29 us with one, after a step whose longest
// sequence has 100000 keys); chunks have 256 rows of few pieces, a warp each (20 us
// more with four, in a batch of chunks).
#include "cmp_attn.cuh"

namespace cmp {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <bool BF16, int DP, int W>
__global__ void __launch_bounds__(kThreads) attn_combine_kernel(const AttnParams p, int m_rows) {
  constexpr int V = DP / 32;  // channels per lane: 2, 4, 6 or 8, as DP / 64 float2
  __shared__ float2 part[kWarps][DP / 2];
  __shared__ float sums[kWarps];
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const int4 d0 = p.desc[2 * c];
  if (d0.x == 0) return;
  const int n = d0.x - c + 1, rows = d0.y, t0 = d0.z, row0 = d0.w;
  const int h = p.desc[2 * c + 1].x;
  constexpr int kRowsPerCta = kWarps / W;
  for (int r = blockIdx.y * kRowsPerCta + (W == 1 ? warp : 0); r < rows; r += gridDim.y * kRowsPerCta) {
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
    for (int i = W == 1 ? 0 : warp; i < n; i += W) {
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
    const int64_t row = attn_out_row(p, t0, h, row0 + r);
    if (W == 1) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int v = 0; v < V / 2; ++v) {
        const int ch = v * 64 + lane * 2;
        if (ch < p.D)
          *reinterpret_cast<uint32_t*>(p.out + row * p.D + ch) = pack2<BF16>(acc[v].x * inv, acc[v].y * inv);
      }
      if (lane == 0 && p.lse) p.lse[row] = attn_lse(mx, l);
      continue;
    }
#pragma unroll
    for (int v = 0; v < V / 2; ++v) part[warp][v * 32 + lane] = acc[v];
    if (lane == 0) sums[warp] = l;
    __syncthreads();
    l = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int t = threadIdx.x;
    if (t < DP / 2 && t * 2 < p.D) {
      const float2 a = part[0][t], b = part[1][t], e = part[2][t], f = part[3][t];
      *reinterpret_cast<uint32_t*>(p.out + row * p.D + t * 2) =
          pack2<BF16>(((a.x + b.x) + (e.x + f.x)) * inv, ((a.y + b.y) + (e.y + f.y)) * inv);
    }
    if (t == 0 && p.lse) p.lse[row] = attn_lse(mx, l);
    __syncthreads();
  }
}

template <bool BF16, int DP>
cudaError_t run(const AttnParams& p, int m, int ctas, cudaStream_t s) {
  if (m <= 16)
    return launch_chained(attn_combine_kernel<BF16, DP, kWarps>, dim3((unsigned)ctas, (unsigned)m), dim3(kThreads), 0,
                          s, 1, p, m);
  return launch_chained(attn_combine_kernel<BF16, DP, 1>, dim3((unsigned)ctas, 32), dim3(kThreads), 0, s, 1, p, m);
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
