// Paged attention for few rows per key head (see cmp_attn.cuh for the operator
// and the division of the work): decoding, drafts to verify.
//
// HBM bound: every key and value is read once for all query heads of its group.
// One producer warp streams tiles of 64 keys and their values through a ring of
// shared-memory stages by TMA (each lane issues one box: 64 channels over a run
// of rows inside one page, and looks up that run's page). Four consumer warps take
// 16 keys of every tile each: S = Q K^T on 16 x 16 x D with mma.sync, an online
// softmax in registers (running maximum and sum per warp, so the warps never wait
// for one another inside an item), and O += P V from the same registers. The
// rows of a tile are few (16 at most), so the tensor work is a few percent of the
// stream's time at any rate; what counts is that the stream never pauses. At the
// end of an item the four warps' accumulators are added in shared memory.
#include "cmp_attn.cuh"

namespace cmp {
namespace {

constexpr int kM = kAttnDecodeRows;
constexpr int kKT = 64;                      // keys per tile
constexpr int kWarps = 4;                    // consumer warps; warp kWarps produces
constexpr int kThreads = (kWarps + 1) * 32;

__device__ unsigned g_attn_err;

template <int DP>
struct DecodeCfg {
  static constexpr int kTileBytes = kKT * DP * 2;        // K or V
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kCtasPerSm = DP <= 128 ? 2 : 1;
  static constexpr int kStages = DP <= 64 ? 6 : DP <= 128 ? 3 : DP <= 192 ? 4 : 3;
  static constexpr int kPitch = DP + 8;                   // floats per row of the merge buffer
  static constexpr int kMergeBytes = kM * kPitch * 4;
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

__device__ __forceinline__ void bar_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

// Byte offset of (key, 16-byte chunk) in a tile that TMA wrote with the 128-byte
// swizzle: blocks of 64 channels, one 128-byte row per key.
__device__ __forceinline__ uint32_t tile_at(int key, int chunk) {
  return (uint32_t)((chunk >> 3) * (kKT * 128) + key * 128 + (((chunk & 7) ^ (key & 7)) << 4));
}

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreads, DecodeCfg<DP>::kCtasPerSm)
    attn_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const AttnParams p) {
  using C = DecodeCfg<DP>;
  constexpr int KS = DP / 16;  // K steps of Q K^T
  constexpr int NT = DP / 8;   // 8-column blocks of the accumulator
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
      sm100::mbar_init(&empty[i], kWarps);
    }
    sm100::fence_barrier_init();
  }
  attn_plan<kKT, kThreads>(p, kM, &start, warp_sum, &g_attn_err);
  AttnWalk<kKT> walk(p, kM);
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
    int n = 0;
    bool alive = true;
    AttnPiece o;
    while (alive && walk.next(o)) {
      if (o.hi <= o.lo) continue;
      const int32_t* trow = p.table + (int64_t)o.b * p.table_stride;
      for (int j = o.j0; j < o.j1; ++j, ++n) {
        const int st = n % C::kStages;
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
        if (n >= C::kStages) alive = sm100::mbar_wait(&empty[st], (uint32_t)(n / C::kStages - 1) & 1u, &abort_flag);
        alive = __all_sync(0xffffffffu, alive);
        if (!alive) break;
        if (lane == 0) sm100::mbar_arrive_expect_tx(&full[st], (uint32_t)__popc(m) * box_bytes);
        armed.note(st, (uint32_t)(n / C::kStages) & 1u);
        __syncwarp();
        if (need)
          sm100::tma_load_3d(ring + (size_t)st * C::kStageBytes + dst_off, map, &full[st], blk * 64, o.h, row);
      }
    }
    if (!sm100::drain_armed(full, C::kStages, armed) || !alive)
      if (lane == 0) atomicOr(&g_attn_err, kErrTimeout);
    return;
  }

  // ---- consumers ----
  const int g = lane >> 2, t4 = lane & 3;  // row (and row + 8) and column pair of a fragment
  int n = 0;
  AttnPiece o;
  bool begun = false;
  if (start.units == 0 && tid == 0) attn_write_desc(p, blockIdx.x, 0, nullptr);
  while (walk.next(o)) {
    // Q fragments: rows g and g + 8; rows past the item are zeros
    uint32_t qf[KS][4];
    int lo[2], hi[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      const bool ok = r < o.rows;
      lo[i] = hi[i] = 0;
      if (ok) attn_row_range(p, o.s, o.row0 + r, lo[i], hi[i]);
      const int rr = o.row0 + r;
      const int tok = p.div_g.div(rr);
      const uint16_t* src = p.q + (int64_t)(o.s.t0 + tok) * p.q_stride + (int64_t)(o.h * p.G + rr - tok * p.G) * p.D;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int c = k * 16 + 2 * t4;
        const bool in = ok && k * 16 < p.D;
        qf[k][i] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + c)) : 0u;
        qf[k][i + 2] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + c + 8)) : 0u;
      }
    }
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    float mrow[2] = {neg_inf(), neg_inf()}, lrow[2] = {0.f, 0.f};

    if (o.hi > o.lo) {
      for (int j = o.j0; j < o.j1; ++j, ++n) {
        const int st = n % C::kStages;
        const bool ok = sm100::mbar_wait(&full[st], (uint32_t)(n / C::kStages) & 1u, &abort_flag);
        unsigned char* kt = ring + (size_t)st * C::kStageBytes;
        unsigned char* vt = kt + C::kTileBytes;
        const int key0 = j * kKT + warp * 16;  // this warp's keys
        if (ok && key0 < o.hi && key0 + 16 > o.lo) {
          if (key0 < o.lo || key0 + 16 > o.hi) {
            // values behind the sequence's end (or before the window) may hold
            // anything, a NaN times a weight of 0 included: make them zeros
            for (int i = lane; i < 16 * (DP / 8); i += 32) {
              const int k = i & 15;
              if (key0 + k < o.lo || key0 + k >= o.hi)
                *reinterpret_cast<uint4*>(vt + tile_at(warp * 16 + k, i >> 4)) = make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the stage's next TMA write comes after
            __syncwarp();
          }
          // S = Q K^T: 16 rows x 16 keys
          float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
          const uint32_t kb = sm100::smem_u32(kt);
          const int krow = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            if (k * 16 < p.D) {
              uint32_t b[4];
              ldsm4(kb + tile_at(krow, k * 2 + ((lane >> 3) & 1)), b);
              mma16816<BF16>(s0, qf[k], b[0], b[1]);
              mma16816<BF16>(s1, qf[k], b[2], b[3]);
            }
          }
          // online softmax; row i of this thread: s*[2i], s*[2i + 1]
          uint32_t pf[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x[4] = {s0[2 * i], s0[2 * i + 1], s1[2 * i], s1[2 * i + 1]};
            const int c = key0 + 2 * t4;
            const int kk[4] = {c, c + 1, c + 8, c + 9};
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = kk[e] >= lo[i] && kk[e] < hi[i] ? x[e] * p.scale_log2 : neg_inf();
            float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx = fmaxf(mx, mrow[i]);
            const float ref = mx == neg_inf() ? 0.f : mx;
            const float corr = ex2(mrow[i] - ref);
            mrow[i] = mx;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e] = ex2(x[e] - ref);
              sum += x[e];
            }
            lrow[i] = fmaf(lrow[i], corr, sum);
            pf[i] = pack2<BF16>(x[0], x[1]);
            pf[i + 2] = pack2<BF16>(x[2], x[3]);
            if (__any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll
              for (int c2 = 0; c2 < NT; ++c2) {
                acc[c2][2 * i] *= corr;
                acc[c2][2 * i + 1] *= corr;
              }
            }
          }
          // O += P V
          const uint32_t vb = sm100::smem_u32(vt);
          const int vrow = warp * 16 + (lane & 15);
#pragma unroll
          for (int c = 0; c < NT; c += 2) {
            if (c * 8 < p.D) {
              uint32_t b[4];
              ldsm4t(vb + tile_at(vrow, c + (lane >> 4)), b);
              mma16816<BF16>(acc[c], pf, b[0], b[1]);
              mma16816<BF16>(acc[c + 1], pf, b[2], b[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&empty[st]);
      }
    }
    // ---- end of the piece: add the four warps' accumulators ----
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lrow[i] += __shfl_xor_sync(0xffffffffu, lrow[i], 1);
      lrow[i] += __shfl_xor_sync(0xffffffffu, lrow[i], 2);
      if (t4 == 0) {
        wm[warp][g + 8 * i] = mrow[i];
        wl[warp][g + 8 * i] = lrow[i];
      }
    }
    bar_consumers();
    float mall[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      float m = wm[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, wm[w][r]);
      mall[i] = m;
      const float f = ex2(mrow[i] - (m == neg_inf() ? 0.f : m));
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        acc[c][2 * i] *= f;
        acc[c][2 * i + 1] *= f;
      }
    }
    for (int w = 0; w < kWarps; ++w) {  // in warp order: the same sum every time
      if (warp == w) {
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float2* d = reinterpret_cast<float2*>(merge + (g + 8 * i) * C::kPitch + c * 8 + 2 * t4);
            float2 v = make_float2(acc[c][2 * i], acc[c][2 * i + 1]);
            if (w) {
              const float2 old = *d;
              v.x += old.x;
              v.y += old.y;
            }
            *d = v;
          }
      }
      bar_consumers();
    }
    const bool whole = o.whole();
    const int slot = o.j0 > o.T0 ? 0 : 1;
    const int64_t pbase = ((int64_t)blockIdx.x * 2 + slot) * kM;
    constexpr int kLanesPerRow = DP / 8;  // 8 columns per thread
    for (int i = tid; i < kM * kLanesPerRow; i += kWarps * 32) {
      const int r = i / kLanesPerRow, c = (i % kLanesPerRow) * 8;
      if (r >= o.rows) break;
      float m = wm[0][r], l = 0.f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, wm[w][r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) l = fmaf(wl[w][r], ex2(wm[w][r] - (m == neg_inf() ? 0.f : m)), l);
      const float* src = merge + r * C::kPitch + c;
      const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
      if (whole) {
        const int64_t row = attn_out_row(p, o.s.t0, o.h, o.row0 + r);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (c < p.D) {
          uint4 v;
          v.x = pack2<BF16>(a.x * inv, a.y * inv);
          v.y = pack2<BF16>(a.z * inv, a.w * inv);
          v.z = pack2<BF16>(b.x * inv, b.y * inv);
          v.w = pack2<BF16>(b.z * inv, b.w * inv);
          *reinterpret_cast<uint4*>(p.out + row * p.D + c) = v;
        }
        if (c == 0 && p.lse) p.lse[row] = attn_lse(m, l);
      } else {
        float* dst = p.part + (pbase + r) * DP + c;
        *reinterpret_cast<float4*>(dst) = a;
        *reinterpret_cast<float4*>(dst + 4) = b;
        if (c == 0) *reinterpret_cast<float2*>(p.part_ml + (pbase + r) * 2) = make_float2(m, l);
      }
    }
    if (tid == 0) {
      if (o.j0 == o.T0 && !whole) {
        attn_write_desc(p, blockIdx.x, attn_last_cta(blockIdx.x, share, o), &o);
        begun = true;
      }
    }
    bar_consumers();  // wm, wl and merge are free again
  }
  if (tid == 0 && !begun && start.units > 0) attn_write_desc(p, blockIdx.x, 0, nullptr);
}

int g_conf[2][4][64];

template <bool BF16, int DP>
cudaError_t run(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s, int ctas) {
  auto* kernel = attn_decode_kernel<BF16, DP>;
  const cudaError_t e = smem_attr_once(kernel, DecodeCfg<DP>::kSmem, g_conf[BF16][DP / 64 - 1]);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, kThreads, DecodeCfg<DP>::kSmem, s>>>(k, v, p);
  return cudaGetLastError();
}

}  // namespace

int attn_decode_ctas(const AttnParams& p, int sms) { return (attn_padded(p.D) <= 128 ? 2 : 1) * sms; }

cudaError_t launch_attn_decode(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s,
                               int ctas) {
  switch (attn_padded(p.D) / 64 * 2 + (p.bf16 ? 1 : 0)) {
    case 2: return run<false, 64>(p, k, v, s, ctas);
    case 3: return run<true, 64>(p, k, v, s, ctas);
    case 4: return run<false, 128>(p, k, v, s, ctas);
    case 5: return run<true, 128>(p, k, v, s, ctas);
    case 6: return run<false, 192>(p, k, v, s, ctas);
    case 7: return run<true, 192>(p, k, v, s, ctas);
    case 8: return run<false, 256>(p, k, v, s, ctas);
    default: return run<true, 256>(p, k, v, s, ctas);
  }
}

cudaError_t attn_decode_take_error(unsigned* word) { return take_symbol_word(g_attn_err, word); }

bool attn_cache_map(CUtensorMap* m, const void* cache, const AttnParams& p) {
  sm100::EncodeTiledFn f = sm100::encode_fn();
  if (!f) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.Hk, (cuuint64_t)p.block_num * p.page};
  const cuuint64_t strides[2] = {(cuuint64_t)p.D * 2, (cuuint64_t)p.Hk * p.D * 2};
  const cuuint32_t box[3] = {64, 1, 1u << p.run_shift};
  const cuuint32_t estr[3] = {1, 1, 1};
  return f(m, p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
           const_cast<void*>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace cmp
