// Paged attention for few rows per key head (see cmp_attn.cuh for the operator
// and the division of the work): decoding, drafts to verify.
//
// HBM bound: every key and value is read once for all query heads of its group.
// One producer warp streams tiles of 64 keys and their values through a ring of
// shared-memory stages by TMA (each lane issues one box: 64 channels over a run
// of rows inside one page, and looks up that run's page). Four consumer warps take
// 16 keys of a tile each.
// The products are transposed, so that the keys fill the 16 rows of mma.sync and
// the few queries its 8 columns (8 rows per item; 16 are two column blocks):
//   S^T = K Q^T,  O^T += V^T P^T
// (with the queries as rows, an item of 8 rows or fewer spent twice the products and
// registers, and a warp has little else to overlap them with: 635 us for 128
// sequences of 24 key heads of 192, two query heads each, where this takes 419, 0.93
// of the measured copy rate). Softmax in registers, statistics per warp, so the
// warps never wait for one another inside an item; a row's reference is moved (and
// the accumulator rescaled) only when a score exceeds it by more than kLazy, so
// that a step needs no shuffle. At the end of an item the warps' accumulators are
// added in shared memory, in a fixed order.
#include "cmp_attn.cuh"

namespace cmp {
namespace {

constexpr int kKT = 64;                       // keys per tile
constexpr float kLazy = 8.f;                  // log2 of the largest weight

__device__ unsigned g_attn_err;

// DP: padded channels; NB: blocks of 8 rows per item
template <int DP, int NB>
struct DecodeCfg {
  static constexpr int kM = 8 * NB;
  static constexpr int kTileBytes = kKT * DP * 2;  // K or V
  static constexpr int kStageBytes = 2 * kTileBytes;
  // Eight consumer warps per SM where their registers and the stages allow: two CTAs
  // of four, or one of eight whose halves (groups) take every other tile. A stage
  // belongs to one group (an even number of stages): a group that runs ahead would
  // not know a stage's phase from the one two before by its parity.
  static constexpr int kCtasPerSm = DP <= 128 ? 2 : 1;
  static constexpr int kGroups = DP == 192 && NB == 1 ? 2 : 1;
  static constexpr int kWarps = 4 * kGroups;  // consumers; warp kWarps produces
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kStages = (kCtasPerSm == 2 ? 98304 : 196608) / kStageBytes;
  static_assert(kStages % kGroups == 0, "a stage belongs to one group");
  static constexpr int kPitch = DP + 4;            // floats per row of a merge buffer
  static constexpr int kMergeBytes = kGroups * kM * kPitch * 4;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + kMergeBytes;
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// An 8 x 8 matrix of 16-bit elements (two of a row per thread), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int kWarps>
__device__ __forceinline__ void bar_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

template <bool BF16, int DP, int NB>
__global__ void __launch_bounds__(DecodeCfg<DP, NB>::kThreads, DecodeCfg<DP, NB>::kCtasPerSm)
    attn_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const AttnParams p) {
  using C = DecodeCfg<DP, NB>;
  constexpr int KS = DP / 16;  // 16-channel steps
  constexpr int kM = C::kM, kGroups = C::kGroups, kWarps = C::kWarps, kThreads = C::kThreads;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = &sm100::smem_align1024<unsigned char>(smem_raw);
  float* merge = reinterpret_cast<float*>(ring + (size_t)C::kStages * C::kStageBytes);
  __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages];
  __shared__ float wm[kWarps][kM], wl[kWarps][kM];
  __shared__ AttnStart start;
  __shared__ int64_t warp_sum[kThreads / 32];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_trigger();
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < C::kStages; ++i) {
      sm100::mbar_init(&full[i], 1);
      sm100::mbar_init(&empty[i], 4);  // the warps of the group that takes the tile
    }
    sm100::fence_barrier_init();
  }
  attn_plan<kKT, kM, kThreads>(p, &start, warp_sum, &g_attn_err);
  AttnWalk<kKT, kM> walk(p);
  walk.begin(start.units, start.b, start.h, start.qt, start.off);
  const int64_t share = start.share;

  if (warp == kWarps) {  // ---- producer ----
    const int run_shift = p.run_shift;  // <= 6
    const int nruns = kKT >> run_shift;
    const int nblk = (p.D + 63) / 64;
    const int boxes = 2 * nblk * nruns;  // <= 32
    const uint32_t box_bytes = 128u << run_shift;
    // this lane's box: K or V, 64-channel block, run
    const bool has = lane < boxes;
    const int run = lane % nruns, blk = (lane / nruns) % nblk, which = lane / (nruns * nblk);
    const CUtensorMap* map = which ? &vmap : &kmap;
    const uint32_t dst_off = (uint32_t)(which * C::kTileBytes + blk * (kKT * 128) + (run << run_shift) * 128);
    const int no_row = (int)(p.block_num * p.page);  // past the cache: zeros land
    sm100::Armed armed;
    int st = 0, n = 0;
    uint32_t par = 0;
    bool alive = true;
    AttnPiece o;
    while (alive && !p.withhold && walk.next(o)) {
      if (o.hi <= o.lo) continue;
      const int32_t* trow = p.table + (int64_t)o.b * p.table_stride;
      for (int j = o.j0; j < o.j1; ++j, ++n) {
        const int key = j * kKT + (run << run_shift);
        const bool need = has && key < o.hi && key + (1 << run_shift) > o.lo;
        int row = no_row;
        if (need) {
          const int pg = p.div_page.div(key);
          const int e = pg < p.table_stride ? __ldg(trow + pg) : -1;
          if (e >= 0 && e < p.block_num) row = e * p.page + (key - pg * p.page);
          else atomicOr(&g_attn_err, kErrIndex);
        }
        const unsigned m = __ballot_sync(0xffffffffu, need);
        if (n >= C::kStages) alive = sm100::mbar_wait(&empty[st], par ^ 1u, &abort_flag);
        alive = __all_sync(0xffffffffu, alive);
        if (!alive) break;
        if (lane == 0) sm100::mbar_arrive_expect_tx(&full[st], (uint32_t)__popc(m) * box_bytes);
        armed.note(st, par);
        __syncwarp();
        if (need)
          sm100::tma_load_3d(ring + (size_t)st * C::kStageBytes + dst_off, map, &full[st], blk * 64, o.h, row);
        if (++st == C::kStages) {
          st = 0;
          par ^= 1u;
        }
      }
    }
    if (!sm100::drain_armed(full, C::kStages, armed) || !alive)
      if (lane == 0) atomicOr(&g_attn_err, kErrTimeout);
    return;
  }

  // ---- consumers ----
  const int g = lane >> 2, t4 = lane & 3;
  const int group = warp >> 2, quarter = warp & 3;
  // byte offsets in a 64-channel block of a tile (one 128-byte row per key, 16-byte
  // chunks XORed with key % 8) that this lane gives to ldmatrix, per 16-channel step:
  // K rows as they lie, V to be transposed
  uint32_t koff[4], voff[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int kk = quarter * 16 + (lane & 15), vk = quarter * 16 + (lane & 7) + ((lane >> 4) << 3);
    koff[k] = (uint32_t)(kk * 128 + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4));
    voff[k] = (uint32_t)(vk * 128 + (((2 * k + ((lane >> 3) & 1)) ^ (lane & 7)) << 4));
  }
  int st = 0, n = 0;  // ring stage and number of the next tile
  uint32_t par = 0;
  AttnPiece o;
  bool begun = false;
  bool ok = true;  // no wait of this warp has given up; the same in all its lanes
  if (start.units == 0 && tid == 0) attn_write_desc(p, blockIdx.x, 0, nullptr);
  while (walk.next(o)) {
    // Q^T fragments (row 8 nb + g, channels 2 t4, + 1 and + 8, + 9 of a step), zeros
    // past the item's rows; visible keys of rows 8 nb + 2 t4 and + 1
    uint32_t qf[KS][NB][2];
    int lo[NB][2], hi[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int r = 8 * b + g;
      const bool there = r < o.rows;
      const int rr = o.row0 + (there ? r : 0);
      const int tok = p.div_g.div(rr);
      const uint16_t* src = p.q + (int64_t)(o.s.t0 + tok) * p.q_stride + (int64_t)(o.h * p.G + rr - tok * p.G) * p.D;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int c = k * 16 + 2 * t4;
        const bool in = there && k * 16 < p.D;
        qf[k][b][0] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + c)) : 0u;
        qf[k][b][1] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + c + 8)) : 0u;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        lo[b][i] = hi[b][i] = 0;
        if (8 * b + 2 * t4 + i < o.rows) attn_row_range(p, o.s, o.row0 + 8 * b + 2 * t4 + i, lo[b][i], hi[b][i]);
      }
    }
    int lo_all, hi_all;  // keys that every row of the item sees
    {
      int x;
      attn_row_range(p, o.s, o.row0, x, hi_all);
      attn_row_range(p, o.s, o.row0 + o.rows - 1, lo_all, x);
    }
    float acc[KS][NB][4];  // O^T: channels 16 s + g (+ 8), rows 8 nb + 2 t4 (+ 1)
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[s][b][e] = 0.f;
    float ref[NB][2], l[NB][2];  // of rows 8 nb + 2 t4 (+ 1); l: this thread's keys only
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      ref[b][0] = ref[b][1] = neg_inf();
      l[b][0] = l[b][1] = 0.f;
    }

    if (o.hi > o.lo) {
      for (int j = o.j0; j < o.j1; ++j, ++n) {
        if ((n & (kGroups - 1)) == group) {
          ok = __all_sync(0xffffffffu, ok && sm100::mbar_wait(&full[st], par, &abort_flag));
          unsigned char* kt = ring + (size_t)st * C::kStageBytes;
          unsigned char* vt = kt + C::kTileBytes;
          const int key0 = j * kKT + quarter * 16;  // this warp's keys
          if (ok && key0 < o.hi && key0 + 16 > o.lo) {
            if (key0 < o.lo || key0 + 16 > o.hi) {
              // values behind the sequence's end (or before the window) may hold
              // anything, a NaN times a weight of 0 included: make them zeros
              for (int i = lane; i < 16 * (DP / 8); i += 32) {
                const int k = i & 15, ch = i >> 4;
                if (key0 + k < o.lo || key0 + k >= o.hi)
                  *reinterpret_cast<uint4*>(vt + (ch >> 3) * (kKT * 128) + (quarter * 16 + k) * 128 + ((ch & 7) << 4)) =
                      make_uint4(0, 0, 0, 0);
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the stage's next TMA write comes after
              __syncwarp();
            }
            // S^T = K Q^T in two chains
            float sa[NB][4], sb[NB][4];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int e = 0; e < 4; ++e) sa[b][e] = sb[b][e] = 0.f;
            const uint32_t ka = sm100::smem_u32(kt), va = sm100::smem_u32(vt);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint32_t a[4];
              ldsm4(ka + (k >> 2) * (kKT * 128) + koff[k & 3], a);
#pragma unroll
              for (int b = 0; b < NB; ++b) mma16816<BF16>(k & 1 ? sb[b] : sa[b], a, qf[k][b][0], qf[k][b][1]);
            }
            // keys g (e < 2) and g + 8, row e & 1
            float x[NB][4];
            bool grow = false;
            const bool edge = key0 < lo_all || key0 + 16 > hi_all;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                x[b][e] = (sa[b][e] + sb[b][e]) * p.scale_log2;
                const int key = key0 + g + (e >> 1) * 8;
                if (edge && (key < lo[b][e & 1] || key >= hi[b][e & 1])) x[b][e] = neg_inf();
                grow |= x[b][e] > ref[b][e & 1] + kLazy;
              }
            if (__any_sync(0xffffffffu, grow)) {  // also a row's first visible key
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  float mx = fmaxf(x[b][i], x[b][i + 2]);
#pragma unroll
                  for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                  const float nref = mx > ref[b][i] + kLazy ? mx : ref[b][i];
                  const float corr = nref == neg_inf() ? 1.f : ex2(ref[b][i] - nref);
                  ref[b][i] = nref;
                  l[b][i] *= corr;
#pragma unroll
                  for (int s = 0; s < KS; ++s) {
                    acc[s][b][i] *= corr;
                    acc[s][b][i + 2] *= corr;
                  }
                }
            }
            uint32_t pf[NB][2];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float r = ref[b][e & 1];
                x[b][e] = ex2(x[b][e] - (r == neg_inf() ? 0.f : r));
              }
              l[b][0] += x[b][0] + x[b][2];
              l[b][1] += x[b][1] + x[b][3];
              pf[b][0] = transpose8(pack2<BF16>(x[b][0], x[b][1]));
              pf[b][1] = transpose8(pack2<BF16>(x[b][2], x[b][3]));
            }
            // O^T += V^T P^T, added outside the product: the tensor core cuts its fp32 sums
            // off, always towards zero, which over 2^22 keys lost 0.7 % of a row (the
            // additions cost nothing at 8 rows per item, at most 1 % at 16)
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              uint32_t a[4];
              ldsm4t(va + (s >> 2) * (kKT * 128) + voff[s & 3], a);
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                float t[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816<BF16>(t, a, pf[b][0], pf[b][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[s][b][e] += t[e];
              }
            }
          }
          __syncwarp();
          if (lane == 0) sm100::mbar_arrive(&empty[st]);
        }
        if (++st == C::kStages) {
          st = 0;
          par ^= 1u;
        }
      }
    }
    // ---- end of the piece: add the warps' accumulators, a buffer per group ----
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[b][i] += __shfl_xor_sync(0xffffffffu, l[b][i], d);
        if (g == 0) {
          wm[warp][8 * b + 2 * t4 + i] = ref[b][i];
          wl[warp][8 * b + 2 * t4 + i] = l[b][i];
        }
      }
    bar_consumers<kWarps>();
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * b + 2 * t4 + i;
        float m = wm[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = fmaxf(m, wm[w][r]);
        const float f = ex2(ref[b][i] - (m == neg_inf() ? 0.f : m));
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          acc[s][b][i] *= f;
          acc[s][b][i + 2] *= f;
        }
      }
    float* mg = merge + group * (kM * C::kPitch);
    for (int w = 0; w < 4; ++w) {  // in warp order: the same sum every time
      if (quarter == w) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float* d = mg + (8 * b + 2 * t4 + (e & 1)) * C::kPitch + 16 * s + g + (e >> 1) * 8;
              *d = w ? *d + acc[s][b][e] : acc[s][b][e];
            }
      }
      bar_consumers<kWarps>();
    }
    const bool whole = o.whole();
    const int slot = o.j0 > o.T0 ? 0 : 1;
    const int64_t pbase = ((int64_t)blockIdx.x * 2 + slot) * kM;
    constexpr int kLanesPerRow = DP / 8;  // 8 columns per thread
    for (int i = tid; i < kM * kLanesPerRow; i += kWarps * 32) {
      const int r = i / kLanesPerRow, c = (i % kLanesPerRow) * 8;
      if (r >= o.rows) break;
      float m = wm[0][r], lsum = 0.f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, wm[w][r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) lsum = fmaf(wl[w][r], ex2(wm[w][r] - (m == neg_inf() ? 0.f : m)), lsum);
      float v[8];
      const float* src = merge + r * C::kPitch + c;
#pragma unroll
      for (int q = 0; q < 8; q += 4) {
        const float4 a = *reinterpret_cast<const float4*>(src + q);
        float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (kGroups == 2) b = *reinterpret_cast<const float4*>(src + kM * C::kPitch + q);
        v[q] = a.x + b.x;
        v[q + 1] = a.y + b.y;
        v[q + 2] = a.z + b.z;
        v[q + 3] = a.w + b.w;
      }
      if (whole) {
        const int64_t row = attn_out_row(p, o.s.t0, o.h, o.row0 + r);
        const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
        if (c < p.D) {
          uint4 u;
          u.x = pack2<BF16>(v[0] * inv, v[1] * inv);
          u.y = pack2<BF16>(v[2] * inv, v[3] * inv);
          u.z = pack2<BF16>(v[4] * inv, v[5] * inv);
          u.w = pack2<BF16>(v[6] * inv, v[7] * inv);
          *reinterpret_cast<uint4*>(p.out + row * p.D + c) = u;
        }
        if (c == 0 && p.lse) p.lse[row] = attn_lse(m, lsum);
      } else {
        float* dst = p.part + (pbase + r) * DP + c;
        *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
        if (c == 0) *reinterpret_cast<float2*>(p.part_ml + (pbase + r) * 2) = make_float2(m, lsum);
      }
    }
    if (tid == 0 && o.j0 == o.T0 && !whole) {
      attn_write_desc(p, blockIdx.x, attn_last_cta(blockIdx.x, share, o), &o);
      begun = true;
    }
    bar_consumers<kWarps>();  // wm, wl and merge are free again
  }
  if (!ok && lane == 0) atomicOr(&g_attn_err, kErrTimeout);
  if (tid == 0 && !begun && start.units > 0) attn_write_desc(p, blockIdx.x, 0, nullptr);
}

int g_conf[2][4][2][64];

template <bool BF16, int DP, int NB>
cudaError_t run(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s, int ctas) {
  using C = DecodeCfg<DP, NB>;
  auto* kernel = attn_decode_kernel<BF16, DP, NB>;
  const cudaError_t e = smem_attr_once(kernel, C::kSmem, g_conf[BF16][DP / 64 - 1][NB - 1]);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, C::kThreads, C::kSmem, s>>>(k, v, p);
  return cudaGetLastError();
}

template <bool BF16, int DP>
cudaError_t run(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s, int ctas, int m) {
  return m == 8 ? run<BF16, DP, 1>(p, k, v, s, ctas) : run<BF16, DP, 2>(p, k, v, s, ctas);
}

}  // namespace

int attn_decode_rows(int64_t rows) { return rows <= 8 ? 8 : 16; }

int attn_decode_ctas(int D, int sms) { return (attn_padded(D) <= 128 ? 2 : 1) * sms; }

cudaError_t launch_attn_decode(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s,
                               int ctas, int m) {
  switch (attn_padded(p.D) / 64 * 2 + (p.bf16 ? 1 : 0)) {
    case 2: return run<false, 64>(p, k, v, s, ctas, m);
    case 3: return run<true, 64>(p, k, v, s, ctas, m);
    case 4: return run<false, 128>(p, k, v, s, ctas, m);
    case 5: return run<true, 128>(p, k, v, s, ctas, m);
    case 6: return run<false, 192>(p, k, v, s, ctas, m);
    case 7: return run<true, 192>(p, k, v, s, ctas, m);
    case 8: return run<false, 256>(p, k, v, s, ctas, m);
    default: return run<true, 256>(p, k, v, s, ctas, m);
  }
}

cudaError_t attn_decode_error_word(unsigned** word) { return cudaGetSymbolAddress((void**)word, g_attn_err); }

// Promotion to 128 bytes: a head's row is 3 lines at 192 channels, and its neighbours
// are read much later (with 256 bytes the step above took 465 us). A row that is no
// multiple of 128 bytes shares lines with its neighbours: of 80 channels, 664 MB are
// fetched for 444; other promotions were not measured there.
bool attn_cache_map(CUtensorMap* m, const void* cache, const AttnParams& p) {
  sm100::EncodeTiledFn f = sm100::encode_fn();
  if (!f) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.Hk, (cuuint64_t)p.block_num * p.page};
  const cuuint64_t strides[2] = {(cuuint64_t)p.D * 2, (cuuint64_t)p.Hk * p.D * 2};
  const cuuint32_t box[3] = {64, 1, 1u << p.run_shift};
  const cuuint32_t estr[3] = {1, 1, 1};
  return f(m, p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
           const_cast<void*>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace cmp
