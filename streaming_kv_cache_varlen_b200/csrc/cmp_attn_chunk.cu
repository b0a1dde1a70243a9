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
// products, warp 9 the TMA boxes, warp 10 walks the CTA's part and leaves its pieces
// in shared memory a few ahead. The order of a step is PV_0(j), QK_0(j+1), PV_1(j),
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
// (128 values), the other 4 give theirs up. 8 * 216 + 4 * 72 = 12 * 168, the launch's.
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr int kPieces = 4;                // pieces the scheduler runs ahead
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
  uint64_t piece_full[kPieces], piece_empty[kPieces];
};

// A piece as the roles read it.
struct ChunkPiece {
  AttnPiece o;
  int last_cta;    // of its item (a piece that begins an item and does not end it)
  int tok0, rem0;  // row0 = tok0 * G + rem0
  bool valid;      // false: the CTA's part ends here
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
  __shared__ ChunkPiece pieces[kPieces];
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
    for (int i = 0; i < kPieces; ++i) {
      sm100::mbar_init(&bars.piece_full[i], 1);
      sm100::mbar_init(&bars.piece_empty[i], 4 * C::kTiles + 2);  // softmax warps, products, producer
    }
    sm100::mbar_init(&bars.last, 1);
    sm100::fence_barrier_init();
  }
  if (warp == 8) sm100::tmem_alloc(&tmem_slot, 512);
  sm100::tc_fence_before();
  attn_plan<KT, kThreads>(p, C::kM, &start, warp_sum, &g_attn_err);  // ends with __syncthreads
  sm100::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // Piece i of this CTA, when the scheduler has written it (its .valid is false
  // behind the last one, or if the wait gave up); one arrival frees the slot.
  auto piece = [&](int i) -> const ChunkPiece* {
    const int s = i % kPieces;
    return sm100::mbar_wait(&bars.piece_full[s], (uint32_t)(i / kPieces) & 1u, &abort_flag) ? &pieces[s] : nullptr;
  };
  auto piece_done = [&](int i) { sm100::mbar_arrive(&bars.piece_empty[i % kPieces]); };

  if (warp >= 8) {
    sm100::regs_dec<kOtherRegs>();
    if (warp == 10) {  // ---- scheduler: the pieces of this CTA's part, a few ahead ----
      if (lane == 0) {
        AttnWalk<KT> walk(p, C::kM);
        walk.begin(start.units, start.b, start.h, start.qt, start.off);
        const int64_t share = start.share;
        for (int i = 0;; ++i) {
          const int s = i % kPieces;
          if (i >= kPieces &&
              !sm100::mbar_wait(&bars.piece_empty[s], (uint32_t)(i / kPieces - 1) & 1u, &abort_flag))
            break;
          ChunkPiece& c = pieces[s];
          AttnPiece o;
          const bool valid = walk.next(o);
          if (valid) {
            c.o = o;
            c.last_cta = attn_last_cta(blockIdx.x, share, o);
            c.tok0 = o.row0 / p.G;
            c.rem0 = o.row0 - c.tok0 * p.G;
          }
          c.valid = valid;
          sm100::mbar_arrive(&bars.piece_full[s]);
          if (!valid) break;
        }
      }
    }
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
      for (int pi = 0; alive; ++pi) {
        const ChunkPiece* c = piece(pi);
        alive = __all_sync(0xffffffffu, c != nullptr);
        if (!alive || !c->valid) break;
        const AttnPiece o = c->o;
        __syncwarp();
        if (lane == 0) piece_done(pi);
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
        uint32_t nq = 0, np = 0;  // parities of the next Q and P tile, bit w: row tile w
        int n = 0;                                // ring position of the item's first tile
        bool ok = true;
        auto take = [&](uint64_t* bar, uint32_t& parities, int w) {
          ok = ok && sm100::mbar_wait(bar + w, (parities >> w) & 1u, &abort_flag);
          parities ^= 1u << w;
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
        for (int pi = 0; ok; ++pi) {
          const ChunkPiece* c = piece(pi);
          ok = c != nullptr;
          if (!ok || !c->valid) break;
          const bool keys = c->o.hi > c->o.lo;
          const int act = c->o.rows > kRows ? 2 : 1;
          const int cnt = c->o.j1 - c->o.j0;
          piece_done(pi);
          if (!keys) continue;
          uint32_t ka = stage(n);
          for (int w = 0; w < act; ++w) {
            take(bars.q_ready, nq, w);
            if (ok) qk(w, ka);
          }
          if (ok) sm100::mma_commit(&bars.empty[n % C::kStages]);
          for (int i = 0; ok && i < cnt; ++i, n += 2) {
            const bool more = i + 1 < cnt;
            const uint32_t va = stage(n + 1);
            for (int w = 0; w < act; ++w) {
              take(bars.p_ready, np, w);
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
    // Q rows of a piece, the warp's 32: loaded to registers while the piece before
    // it ends, then stored K-major with the 128-byte swizzle (zeros behind the rows)
    constexpr int kCols = DP / 8;  // 16-byte chunks per row
    uint4 qreg[kCols];
    const int wrow = w * kRows + (warp & 3) * 32;  // first row of the warp within an item
    auto active = [&](const ChunkPiece* c) { return c->valid && c->o.hi > c->o.lo && c->o.rows > w * kRows; };
    auto load_q = [&](const ChunkPiece* c) {
      const uint16_t* base = p.q + (int64_t)(c->o.s.t0 + c->tok0) * p.q_stride + (int64_t)c->o.h * p.G * p.D;
      const int rows = active(c) ? c->o.rows : 0, rem0 = c->rem0;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int e = i * 32 + lane, qr = wrow + e / kCols, ch = e % kCols;
        const int tok = attn_div_g(p, rem0 + qr), head = rem0 + qr - tok * p.G;
        qreg[i] = make_uint4(0, 0, 0, 0);
        if (qr < rows && ch * 8 < p.D)
          qreg[i] = __ldg(reinterpret_cast<const uint4*>(base + (int64_t)tok * p.q_stride + head * p.D + ch * 8));
      }
    };
    const ChunkPiece* c = piece(0);
    ok = __all_sync(0xffffffffu, c != nullptr);
    if (ok) load_q(c);
    for (int pi = 0; ok && c->valid; ++pi) {
      const int row = w * kRows + r;  // of the item
      const bool mine = row < c->o.rows;
      if (tid == 0 && !c->o.whole() && c->o.j0 == c->o.T0) {
        attn_write_desc(p, blockIdx.x, c->last_cta, &c->o);
        begun = true;
      }
      const int tok = attn_div_g(p, c->rem0 + row);
      const int64_t orow =
          (int64_t)(c->o.s.t0 + c->tok0 + tok) * p.Hq + c->o.h * p.G + c->rem0 + row - tok * p.G;  // of out and lse
      if (c->o.hi <= c->o.lo && mine) {
        for (int e = 0; e < p.D; e += 8)
          *reinterpret_cast<uint4*>(p.out + orow * p.D + e) = make_uint4(0, 0, 0, 0);
        if (p.lse) p.lse[orow] = neg_inf();
      }
      const int cnt = c->o.hi > c->o.lo ? c->o.j1 - c->o.j0 : 0;
      const bool act = active(c);
      const bool warp_rows = wrow < c->o.rows;
      float ref = neg_inf(), l = 0.f;  // reference (log2 units) and sum of the row's weights
      if (act) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          const int e = i * 32 + lane, qr = (warp & 3) * 32 + e / kCols, ch = e % kCols;
          *reinterpret_cast<uint4*>(qw + (ch >> 3) * (kRows * 128) + qr * 128 + (((ch & 7) ^ (qr & 7)) << 4)) = qreg[i];
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&bars.q_ready[w]);
        int lo = 0, hi = 0;
        if (mine) {
          hi = attn_keys(p, c->o.s.start + c->tok0 + tok + 1);
          lo = p.window ? max(0, hi - p.window) : 0;
        }
        for (int i = 0; i < cnt; ++i, n += 2) {
          const int key0 = (c->o.j0 + i) * KT;
          if (key0 < c->o.lo || key0 + KT > c->o.hi) {
            // values behind the sequence's end (or before the window) may hold
            // anything, a NaN times a weight of 0 included: make them zeros
            const int st = (n + 1) % C::kStages, klo = c->o.lo, khi = c->o.hi;
            ok = sm100::mbar_wait(&bars.full[st], (uint32_t)((n + 1) / C::kStages) & 1u, &abort_flag) && ok;
            unsigned char* vt = ring + (size_t)st * C::kTileBytes;
            for (int e = r; ok && e < KT * kCols; e += kRows) {
              const int k = e / kCols, ch = e % kCols;
              if (key0 + k < klo || key0 + k >= khi)
                *reinterpret_cast<uint4*>(vt + (ch >> 3) * (KT * 128) + k * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          ok = sm100::mbar_wait(&bars.s_full[w], ns++ & 1u, &abort_flag) && ok;
          ok = __all_sync(0xffffffffu, ok);
            sm100::tc_fence_after();
          if (warp_rows) {
            uint32_t x[KT / 32][32];
#pragma unroll
            for (int b = 0; b < KT / 32; ++b) sm100::tmem_ld32(s_t + b * 32, x[b]);
#pragma unroll
            for (int b = 0; b < KT / 32; ++b) sm100::tmem_ld_wait(x[b]);
            const int clo = lo - key0, chi = hi - key0;  // the row's visible columns
            if (__any_sync(0xffffffffu, clo > 0 || chi < KT)) {
#pragma unroll
              for (int e = 0; e < KT; ++e)
                if (e < clo || e >= chi) x[e / 32][e % 32] = 0xff800000u;
            }
            float mx = neg_inf();
#pragma unroll
            for (int e = 0; e < KT; e += 2)
              mx = max3(mx, __uint_as_float(x[e / 32][e % 32]), __uint_as_float(x[e / 32][e % 32 + 1]));
            mx *= p.scale_log2;
            const bool grow = mx > ref + kLazy;  // also the first visible key's tile
            if (__any_sync(0xffffffffu, grow)) {
              const float nref = grow ? mx : ref;
              const float corr = grow ? ex2(ref - nref) : 1.f;
              l *= corr;
              ref = nref;
              if (i > 0) {
#pragma unroll
                for (int d = 0; d < DP; d += 32) {
                  uint32_t a[32];
                  sm100::tmem_ld32(o_t + d, a);
                  sm100::tmem_ld_wait(a);
#pragma unroll
                  for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * corr);
                  sm100::tmem_st32(o_t + d, a);
                }
              }
            }
            const float base = ref == neg_inf() ? 0.f : -ref;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < KT / 32; ++b) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float u = ex2(fmaf(__uint_as_float(x[b][e]), p.scale_log2, base));
                const float v = ex2(fmaf(__uint_as_float(x[b][e + 1]), p.scale_log2, base));
                sum[e % 4] += u;
                sum[e % 4 + 1] += v;
                pk[e / 2] = pack2<BF16>(u, v);
              }
              sm100::tmem_st16(s_t + b * 16, pk);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            sm100::tmem_st_wait();
          }
          sm100::tc_fence_before();
          __syncwarp();
          if (lane == 0) sm100::mbar_arrive(&bars.p_ready[w]);
        }
      } else {
        n += 2 * cnt;  // no rows of this tile
      }
      if (!ok) break;
      // ---- end of the piece; the next one's Q is loaded meanwhile ----
      const ChunkPiece* next = piece(pi + 1);
      ok = __all_sync(0xffffffffu, next != nullptr);
      if (!ok) break;
      load_q(next);
      if (act) {
        ok = sm100::mbar_wait(&bars.o_full[w], no++ & 1u, &abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        sm100::tc_fence_after();
        if (warp_rows) {
          const bool whole = c->o.whole();
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int64_t prow = ((int64_t)blockIdx.x * 2 + (c->o.j0 > c->o.T0 ? 0 : 1)) * C::kM + row;
          unsigned char* orow_s = qw + r * 128;  // whole rows pass through the warp's part of the Q tile
#pragma unroll
          for (int d = 0; d < DP; d += 32) {
            uint32_t a[32];
            sm100::tmem_ld32(o_t + d, a);
            sm100::tmem_ld_wait(a);
            if (whole) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  v[u] = pack2<BF16>(__uint_as_float(a[e + 2 * u]) * inv, __uint_as_float(a[e + 2 * u + 1]) * inv);
                const int ch = (d + e) / 8;
                *reinterpret_cast<uint4*>(orow_s + (ch >> 3) * (kRows * 128) + (((ch & 7) ^ (r & 7)) << 4)) =
                    make_uint4(v[0], v[1], v[2], v[3]);
              }
            } else if (mine) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                if (d + e >= p.D) break;
                *reinterpret_cast<uint4*>(p.part + prow * DP + d + e) = make_uint4(a[e], a[e + 1], a[e + 2], a[e + 3]);
              }
            }
          }
          if (whole) {
            __syncwarp();
            const int rows = c->o.rows, rem0 = c->rem0;
            uint16_t* base = p.out + ((int64_t)(c->o.s.t0 + c->tok0) * p.Hq + (int64_t)c->o.h * p.G) * p.D;
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
              const int e = i * 32 + lane, qr = (warp & 3) * 32 + e / kCols, ch = e % kCols;
              const int ir = w * kRows + qr;
              const int t = attn_div_g(p, rem0 + ir), head = rem0 + ir - t * p.G;
              const uint4 v =
                  *reinterpret_cast<const uint4*>(qw + (ch >> 3) * (kRows * 128) + qr * 128 + (((ch & 7) ^ (qr & 7)) << 4));
              if (ir < rows && ch * 8 < p.D)
                *reinterpret_cast<uint4*>(base + ((int64_t)t * p.Hq + head) * p.D + ch * 8) = v;
            }
          }
          if (mine) {
            if (!whole) *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(ref, l);
            else if (p.lse) p.lse[orow] = attn_lse(ref, l);
          }
        }
        sm100::tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) piece_done(pi);
      c = next;
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
