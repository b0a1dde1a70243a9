// Paged attention for many rows per key head (see cmp_attn.cuh for the operator
// and the division of the work): chunks of prompts, batches that mix them with
// decoding.
//
// Both products run on tcgen05, M = 128 rows of one key head's group at a time:
//   S = Q K^T   Q and K in shared memory, S in TMEM (fp32, KT columns)
//   O += P V    P (16-bit) in TMEM over the columns of S, V in shared memory as it
//               lies in the cache (keys x channels: an MN-major B operand), O in TMEM
// An item is two row tiles that share every K and V tile: while one tile's rows
// are in the softmax, the tensor core works for the other. Warps 0-3 and 4-7 are
// the two tiles' softmax warps, one row per thread (no shuffles); warp 8 issues the
// products, warp 9 the TMA boxes. The order of a step is PV_0(j), QK_0(j+1), PV_1(j),
// QK_1(j+1): products of one thread run in order, so S_w(j+1) may take the columns of
// P_w(j) without a wait. The accumulator is rescaled by its own softmax warp, and
// only when a row's maximum has grown by more than 2^kLazy since its reference was
// set: the weights are then at most 2^kLazy, exact in either type's range, and the
// common factor cancels in out and lse.
#include "cmp_attn.cuh"

namespace cmp {
namespace {

constexpr int kRows = 128;                // rows per MMA tile
constexpr int kThreads = 12 * 32;
// Registers per thread after the roles split: 8 softmax warps hold a row of S each
// (128 values), the other 4 give theirs up. 8 * 208 + 4 * 88 = 12 * 168, the launch's.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr float kLazy = 8.f;              // log2 of the largest weight

__device__ unsigned g_attn_err;

template <int DP>
struct ChunkCfg {
  static constexpr int kTiles = DP <= 192 ? 2 : 1;    // row tiles per item: 2 * DP + 2 * KT <= 512 TMEM columns
  static constexpr int kKT = DP <= 128 ? 128 : 64;    // keys per tile
  static constexpr int kQBytes = kRows * DP * 2;
  static constexpr int kTileBytes = kKT * DP * 2;     // K or V
  static constexpr int kStages = DP <= 64 ? 8 : 5;
  static constexpr size_t kSmem = 1024 + (size_t)kTiles * kQBytes + (size_t)kStages * kTileBytes;
  static constexpr int kM = kRows * kTiles;
};

// Named by the pair of softmax warps' barriers and the ring's.
template <int DP>
struct ChunkBars {
  uint64_t full[ChunkCfg<DP>::kStages], empty[ChunkCfg<DP>::kStages];
  uint64_t q_ready[2], s_full[2], p_ready[2], o_full[2], last;
};

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

template <bool BF16, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_chunk_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const AttnParams p) {
  using C = ChunkCfg<DP>;
  constexpr int KT = C::kKT;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* qs = &sm100::smem_align1024<unsigned char>(smem_raw);
  unsigned char* ring = qs + (size_t)C::kTiles * C::kQBytes;
  __shared__ __align__(8) ChunkBars<DP> bars;
  __shared__ AttnStart start;
  __shared__ int64_t warp_sum[kThreads / 32];
  __shared__ int abort_flag;
  __shared__ uint32_t tmem_slot;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_trigger();
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < C::kStages; ++i) {
      sm100::mbar_init(&bars.full[i], 1);
      sm100::mbar_init(&bars.empty[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      sm100::mbar_init(&bars.q_ready[w], 4);
      sm100::mbar_init(&bars.s_full[w], 1);
      sm100::mbar_init(&bars.p_ready[w], 4);
      sm100::mbar_init(&bars.o_full[w], 1);
    }
    sm100::mbar_init(&bars.last, 1);
    sm100::fence_barrier_init();
  }
  if (warp == 8) sm100::tmem_alloc(&tmem_slot, 512);
  sm100::tc_fence_before();
  attn_plan<KT, kThreads>(p, C::kM, &start, warp_sum, &g_attn_err);  // ends with __syncthreads
  sm100::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  AttnWalk<KT> walk(p, C::kM);
  walk.begin(start.units, start.b, start.h, start.qt, start.off);
  AttnPiece o;

  if (warp >= 8) {
    sm100::regs_dec<kOtherRegs>();
    if (warp == 9) {  // ---- producer: K and V tiles in turn ----
      const int run_shift = p.run_shift;
      const int nruns = KT >> run_shift;
      const int nblk = (p.D + 63) / 64;
      const uint32_t box_bytes = 128u << run_shift;
      const bool has = lane < nblk * nruns;  // at most 16 boxes
      const int run = lane % nruns, blk = lane / nruns;
      const uint32_t dst_off = (uint32_t)(blk * (KT * 128) + (run << run_shift) * 128);
      const int no_row = (int)(p.block_num * p.page);  // past the cache: zeros land
      sm100::Armed armed;
      int n = 0;
      bool alive = true;
      while (alive && walk.next(o)) {
        if (o.hi <= o.lo) continue;
        const int32_t* trow = p.table + (int64_t)o.b * p.table_stride;
        for (int j = o.j0; alive && j < o.j1; ++j) {
          const int key = j * KT + (run << run_shift);
          const bool need = has && key < o.hi && key + (1 << run_shift) > o.lo;
          int row = no_row;
          if (need) {
            const int pg = key / p.page;
            const int e = pg < p.table_stride ? __ldg(trow + pg) : -1;
            if (e >= 0 && e < p.block_num) row = e * p.page + key % p.page;
            else atomicOr(&g_attn_err, kErrIndex);
          }
          const unsigned m = __ballot_sync(0xffffffffu, need);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const int st = n % C::kStages;
            if (n >= C::kStages)
              alive = sm100::mbar_wait(&bars.empty[st], (uint32_t)(n / C::kStages - 1) & 1u, &abort_flag);
            alive = __all_sync(0xffffffffu, alive);
            if (!alive) break;
            if (lane == 0) sm100::mbar_arrive_expect_tx(&bars.full[st], (uint32_t)__popc(m) * box_bytes);
            armed.note(st, (uint32_t)(n / C::kStages) & 1u);
            __syncwarp();
            if (need)
              sm100::tma_load_3d(ring + (size_t)st * C::kTileBytes + dst_off, kv ? &vmap : &kmap, &bars.full[st],
                                 blk * 64, o.h, row);
          }
        }
      }
      if (!sm100::drain_armed(bars.full, C::kStages, armed) || !alive)
        if (lane == 0) atomicOr(&g_attn_err, kErrTimeout);
    } else if (warp == 8) {  // ---- products ----
      if (lane == 0) {
        constexpr uint32_t idesc_qk = sm100::idesc_16bit_f32(kRows, KT, BF16, false);
        const uint32_t idesc_pv = sm100::idesc_16bit_f32(kRows, p.D, BF16, true);
        const int ks = p.D / 16;
        const uint32_t ring_a = sm100::smem_u32(ring), q_a = sm100::smem_u32(qs);
        uint32_t nq[2] = {0, 0}, np[2] = {0, 0};  // Q tiles and P tiles taken so far, of each row tile
        int n = 0;                                // ring position of the item's first tile
        bool ok = true;
        auto take = [&](uint64_t* bar, uint32_t& count) {
          ok = ok && sm100::mbar_wait(bar, count++ & 1u, &abort_flag);
          sm100::tc_fence_after();
        };
        auto stage = [&](int i) {  // wait for ring position i
          ok = ok && sm100::mbar_wait(&bars.full[i % C::kStages], (uint32_t)(i / C::kStages) & 1u, &abort_flag);
          sm100::tc_fence_after();
          return ring_a + (uint32_t)(i % C::kStages) * C::kTileBytes;
        };
        auto qk = [&](int w, uint32_t ka) {
          const uint32_t qa = q_a + w * C::kQBytes;
          for (int k = 0; k < ks; ++k)
            sm100::mma_bf16(tmem + w * KT, sm100::sw128_kmajor_desc(qa + (k >> 2) * (kRows * 128) + (k & 3) * 32),
                            sm100::sw128_kmajor_desc(ka + (k >> 2) * (KT * 128) + (k & 3) * 32), idesc_qk, k > 0);
          sm100::mma_commit(&bars.s_full[w]);
        };
        auto pv = [&](int w, uint32_t va, bool first) {
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            sm100::mma_ts(tmem + C::kTiles * KT + w * DP, tmem + w * KT + k * 8,
                          sm100::sw128_mnmajor_desc(va + k * 2048, KT * 128), idesc_pv, !first || k > 0);
        };
        while (ok && walk.next(o)) {
          if (o.hi <= o.lo) continue;
          const int act = o.rows > kRows ? 2 : 1;
          const int cnt = o.j1 - o.j0;
          uint32_t ka = stage(n);
          for (int w = 0; w < act; ++w) {
            take(&bars.q_ready[w], nq[w]);
            if (ok) qk(w, ka);
          }
          if (ok) sm100::mma_commit(&bars.empty[n % C::kStages]);
          for (int i = 0; ok && i < cnt; ++i, n += 2) {
            const bool more = i + 1 < cnt;
            const uint32_t va = stage(n + 1);
            for (int w = 0; w < act; ++w) {
              take(&bars.p_ready[w], np[w]);
              if (!ok) break;
              pv(w, va, i == 0);
              if (more) {
                if (w == 0) ka = stage(n + 2);
                if (ok) qk(w, ka);
              } else {
                sm100::mma_commit(&bars.o_full[w]);
              }
            }
            if (!ok) break;
            sm100::mma_commit(&bars.empty[(n + 1) % C::kStages]);
            if (more) sm100::mma_commit(&bars.empty[(n + 2) % C::kStages]);
          }
        }
        // no product is in flight when the columns are freed
        sm100::mma_commit(&bars.last);
        if (!sm100::mbar_wait_bounded(&bars.last, 0, 20000000ull) || !ok) atomicOr(&g_attn_err, kErrTimeout);
      }
    }
  } else if (warp < 4 * C::kTiles) {  // ---- softmax: one row per thread ----
    sm100::regs_inc<kSoftmaxRegs>();
    const int w = warp >> 2, r = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_t = lanes + w * KT, o_t = lanes + C::kTiles * KT + w * DP;
    unsigned char* qw = qs + (size_t)w * C::kQBytes;
    uint32_t ns = 0, no = 0;  // S tiles and accumulators taken
    int n = 0;
    bool begun = false, ok = true;
    while (ok && walk.next(o)) {
      const int row = w * kRows + r;  // of the item
      const bool mine = row < o.rows;
      const bool whole = o.whole();
      if (tid == 0 && !whole && o.j0 == o.T0) {
        attn_write_desc(p, blockIdx.x, attn_last_cta(blockIdx.x, start.share, o), &o);
        begun = true;
      }
      if (o.hi <= o.lo) {
        if (mine) {
          const int64_t orow = attn_out_row(p, o.s.t0, o.h, o.row0 + row);
          for (int c = 0; c < p.D; c += 8)
            *reinterpret_cast<uint4*>(p.out + orow * p.D + c) = make_uint4(0, 0, 0, 0);
          if (p.lse) p.lse[orow] = neg_inf();
        }
        continue;
      }
      const int cnt = o.j1 - o.j0;
      if (o.rows <= w * kRows) {  // this row tile has no rows
        n += 2 * cnt;
        continue;
      }
      // Q to shared memory (K-major, 128-byte swizzle), zeros behind the item's rows
#pragma unroll 8
      for (int i = r; i < kRows * (DP / 8); i += kRows) {
        const int qr = i / (DP / 8), c = i % (DP / 8);
        const int ir = o.row0 + w * kRows + qr;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (w * kRows + qr < o.rows && c * 8 < p.D)
          v = __ldg(reinterpret_cast<const uint4*>(p.q + (int64_t)(o.s.t0 + ir / p.G) * p.q_stride +
                                                   (int64_t)(o.h * p.G + ir % p.G) * p.D + c * 8));
        *reinterpret_cast<uint4*>(qw + (c >> 3) * (kRows * 128) + qr * 128 + (((c & 7) ^ (qr & 7)) << 4)) = v;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&bars.q_ready[w]);

      int lo = 0, hi = 0;
      if (mine) attn_row_range(p, o.s, o.row0 + row, lo, hi);
      const bool warp_rows = w * kRows + (warp & 3) * 32 < o.rows;
      float ref = neg_inf(), l = 0.f;  // reference (log2 units) and sum of the row's weights
      for (int i = 0; i < cnt; ++i, n += 2) {
        const int key0 = (o.j0 + i) * KT;
        if (key0 < o.lo || key0 + KT > o.hi) {
          // values behind the sequence's end (or before the window) may hold
          // anything, a NaN times a weight of 0 included: make them zeros
          const int st = (n + 1) % C::kStages;
          ok = sm100::mbar_wait(&bars.full[st], (uint32_t)((n + 1) / C::kStages) & 1u, &abort_flag) && ok;
          unsigned char* vt = ring + (size_t)st * C::kTileBytes;
          for (int e = r; ok && e < KT * (DP / 8); e += kRows) {
            const int k = e / (DP / 8), c = e % (DP / 8);
            if (key0 + k < o.lo || key0 + k >= o.hi)
              *reinterpret_cast<uint4*>(vt + (c >> 3) * (KT * 128) + k * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        ok = sm100::mbar_wait(&bars.s_full[w], ns++ & 1u, &abort_flag) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        sm100::tc_fence_after();
        if (warp_rows) {
          uint32_t x[KT / 32][32];
#pragma unroll
          for (int c = 0; c < KT / 32; ++c) sm100::tmem_ld32(s_t + c * 32, x[c]);
#pragma unroll
          for (int c = 0; c < KT / 32; ++c) sm100::tmem_ld_wait(x[c]);
          const int clo = lo - key0, chi = hi - key0;  // the row's visible columns
          if (__any_sync(0xffffffffu, clo > 0 || chi < KT)) {
#pragma unroll
            for (int c = 0; c < KT; ++c)
              if (c < clo || c >= chi) x[c / 32][c % 32] = 0xff800000u;
          }
          float mx = neg_inf();
#pragma unroll
          for (int c = 0; c < KT; c += 2)
            mx = max3(mx, __uint_as_float(x[c / 32][c % 32]), __uint_as_float(x[c / 32][c % 32 + 1]));
          mx *= p.scale_log2;
          const bool grow = mx > ref + kLazy;  // also the first visible key's tile
          if (__any_sync(0xffffffffu, grow)) {
            const float nref = grow ? mx : ref;
            const float corr = grow ? ex2(ref - nref) : 1.f;
            l *= corr;
            ref = nref;
            if (i > 0) {
#pragma unroll
              for (int c = 0; c < DP; c += 32) {
                uint32_t a[32];
                sm100::tmem_ld32(o_t + c, a);
                sm100::tmem_ld_wait(a);
#pragma unroll
                for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * corr);
                sm100::tmem_st32(o_t + c, a);
              }
            }
          }
          const float base = ref == neg_inf() ? 0.f : -ref;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < KT / 32; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float a = ex2(fmaf(__uint_as_float(x[c][e]), p.scale_log2, base));
              const float b = ex2(fmaf(__uint_as_float(x[c][e + 1]), p.scale_log2, base));
              sum[e % 4] += a;
              sum[e % 4 + 1] += b;
              pk[e / 2] = pack2<BF16>(a, b);
            }
            sm100::tmem_st16(s_t + c * 16, pk);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          sm100::tmem_st_wait();
        }
        sm100::tc_fence_before();
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&bars.p_ready[w]);
      }
      if (!ok) break;
      // ---- end of the piece ----
      ok = sm100::mbar_wait(&bars.o_full[w], no++ & 1u, &abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      sm100::tc_fence_after();
      if (warp_rows) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t orow = mine ? attn_out_row(p, o.s.t0, o.h, o.row0 + row) : 0;
        const int64_t prow = ((int64_t)blockIdx.x * 2 + (o.j0 > o.T0 ? 0 : 1)) * C::kM + row;
#pragma unroll
        for (int c = 0; c < DP; c += 32) {
          uint32_t a[32];
          sm100::tmem_ld32(o_t + c, a);
          sm100::tmem_ld_wait(a);
          if (!mine) continue;
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              if (c + e >= p.D) break;
              uint32_t v[4];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                v[u] = pack2<BF16>(__uint_as_float(a[e + 2 * u]) * inv, __uint_as_float(a[e + 2 * u + 1]) * inv);
              *reinterpret_cast<uint4*>(p.out + orow * p.D + c + e) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              if (c + e >= p.D) break;
              *reinterpret_cast<uint4*>(p.part + prow * DP + c + e) = make_uint4(a[e], a[e + 1], a[e + 2], a[e + 3]);
            }
          }
        }
        if (mine) {
          if (!whole) *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(ref, l);
          else if (p.lse) p.lse[orow] = attn_lse(ref, l);
        }
      }
      sm100::tc_fence_before();
    }
    if (tid == 0 && !begun) attn_write_desc(p, blockIdx.x, 0, nullptr);
  } else {
    sm100::regs_dec<kOtherRegs>();
  }
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == 8) sm100::tmem_dealloc(tmem, 512);
}

int g_conf[2][4][64];

template <bool BF16, int DP>
cudaError_t run(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s, int ctas) {
  auto* kernel = attn_chunk_kernel<BF16, DP>;
  const cudaError_t e = smem_attr_once(kernel, ChunkCfg<DP>::kSmem, g_conf[BF16][DP / 64 - 1]);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, kThreads, ChunkCfg<DP>::kSmem, s>>>(k, v, p);
  return cudaGetLastError();
}

}  // namespace

int attn_chunk_rows(int D) { return attn_padded(D) <= 192 ? 2 * kRows : kRows; }
int attn_chunk_key_tile(int D) { return attn_padded(D) <= 128 ? 128 : 64; }

cudaError_t launch_attn_chunk(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s,
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

cudaError_t attn_chunk_take_error(unsigned* word) { return take_symbol_word(g_attn_err, word); }

}  // namespace cmp
