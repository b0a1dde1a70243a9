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
// common factor cancels in out and lse. P is handed over in halves, so that its
// product starts while the second half's exponentials run.
//
// Bound by the chain scores - softmax - weights - products of a row tile, of which two
// run in turn: 128 keys of a pair of tiles take 3400 clocks, of which the tensor core
// works 2050 and the special function unit 2050 (16 exponentials a clock). 4096 tokens
// of 32 heads of 128 over 16384 positions (962 GFLOP) take 726 us, 0.81 of the measured
// matrix product burst (842 to 847 us back to back, where power limits the clock).
// The running reference and sum of a softmax in one pass: Milakov and Gimelshein, Online
// normalizer calculation for softmax (2018). Measured and not kept: 2^x by polynomial for
// 1/8 to 3/8 of the weights (as fast or slower: its 15 instructions a pair take the issue slots that the
// special function unit leaves), half a row per thread on 16 softmax warps (800 us: a
// second pass over TMEM, as 64 scores and the rest do not fit 104 registers), tiles of
// 64 keys with two score buffers (800 to 950 us: the fixed cost of a step, 500 clocks,
// comes twice as often), one issuing warp per row tile (870 us: the tiles fall into
// step and wait for the special function unit together).
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
  static constexpr int kStages = DP <= 64 ? 8 : 4;     // a fifth of 32 KB made no case faster
  static constexpr size_t kSmem = 1024 + (size_t)kTiles * kQBytes + (size_t)kStages * kTileBytes;
  static constexpr int kM = kRows * kTiles;
};

// Barriers: of the ring, of a row tile's Q, S, P and O, of the pieces.
template <int DP>
struct ChunkBars {
  uint64_t full[ChunkCfg<DP>::kStages], empty[ChunkCfg<DP>::kStages];
  uint64_t q_ready[2], s_full[2], p_half[2], p_ready[2], o_full[2], last;
  uint64_t piece_full[kPieces], piece_empty[kPieces];
};

// Key tiles that are summed in the accumulator before they leave it. The tensor core cuts
// sums off instead of rounding them, up to 2^-23 of the accumulator for each 16 keys, always
// towards zero: a row of 2^20 keys lost 0.7 % in one go. The parts of a longer piece are
// added in fp32 (rounded) in the piece's slot of the workspace, at 2^-12 each at most.
constexpr int kPartTiles = 256;

// Kinds of parts: the first of the piece, the part after which the item's rows are complete
// (no other CTA has a piece of it), part of a piece that begins the item.
constexpr uint32_t kPartFirst = 1, kPartEnd = 2, kPartBegins = 4;

// A part of a piece (most have one) as the roles read it.
struct ChunkPiece {
  AttnPiece o;         // [j0, j1): the part's tiles
  int last_cta;        // of its item (a piece that begins an item and does not end it; else 0)
  int tok0, rem0;      // row0 = tok0 * G + rem0
  uint32_t kind;       // kPart...
  bool valid;          // false: the CTA's share of the work ends here
};

// The largest of three; NaN if one of them is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Adds what this thread left of its row in the workspace to the accumulator in TMEM and to
// the row's reference and sum; part: its first four channels there, `stride` floats apart
// from the next four. A call, as its registers in line made the usual pieces' stores slower
// (4000 tokens over compressed rows 129 us instead of 124.5).
__device__ __noinline__ float2 add_part(uint32_t o_t, const float* part, int stride, const float* ml_at, int D, bool mine,
                                        float ref, float l) {
  float w_old = 0.f, w_new = 1.f;
  if (mine) {
    const float2 ml = *reinterpret_cast<const float2*>(ml_at);
    const float m = fmaxf(ml.x, ref), at = m == neg_inf() ? 0.f : m;
    w_old = ex2(ml.x - at);
    w_new = ex2(ref - at);
    l = fmaf(ml.y, w_old, l * w_new);
    ref = m;
  }
#pragma unroll 1
  for (int d = 0; d < D; d += 16) {
    uint32_t a[16];
    sm100::tmem_ld16(o_t + d, a);
    sm100::tmem_ld_wait16(a);
    if (mine) {
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 x = *reinterpret_cast<const float4*>(part + (int64_t)((d + e) / 4) * stride);
        a[e] = __float_as_uint(fmaf(x.x, w_old, __uint_as_float(a[e]) * w_new));
        a[e + 1] = __float_as_uint(fmaf(x.y, w_old, __uint_as_float(a[e + 1]) * w_new));
        a[e + 2] = __float_as_uint(fmaf(x.z, w_old, __uint_as_float(a[e + 2]) * w_new));
        a[e + 3] = __float_as_uint(fmaf(x.w, w_old, __uint_as_float(a[e + 3]) * w_new));
      }
    }
    __syncwarp();
    sm100::tmem_st16(o_t + d, a);
  }
  sm100::tmem_st_wait();
  return make_float2(ref, l);
}

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
  const int tid = threadIdx.x, warp = sm100::uniform(tid >> 5), lane = tid & 31;

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
      sm100::mbar_init(&bars.p_half[w], 4);
      sm100::mbar_init(&bars.p_ready[w], 4);
      sm100::mbar_init(&bars.o_full[w], 1);
    }
    sm100::mbar_init(&bars.last, 1);
    for (int i = 0; i < kPieces; ++i) {
      sm100::mbar_init(&bars.piece_full[i], 1);
      sm100::mbar_init(&bars.piece_empty[i], 4 * C::kTiles + 2);  // softmax warps, products, producer
    }
    sm100::fence_barrier_init();
  }
  if (warp == 8) sm100::tmem_alloc(&tmem_slot, 512);
  sm100::tc_fence_before();
  attn_plan<KT, C::kM, kThreads>(p, &start, warp_sum, &g_attn_err);  // ends with __syncthreads
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
        AttnWalk<KT, C::kM> walk(p);
        walk.begin(start.units, start.b, start.h, start.qt, start.off);
        const int64_t share = start.share;
        AttnPiece o;
        int j = 0, j1 = 0;  // tiles of the piece that no part has yet
        for (int i = 0;; ++i) {
          const int s = i % kPieces;
          if (i >= kPieces &&
              !sm100::mbar_wait(&bars.piece_empty[s], (uint32_t)(i / kPieces - 1) & 1u, &abort_flag))
            break;
          ChunkPiece& c = pieces[s];
          bool valid = true;
          const bool first = j == j1;
          if (first) {
            valid = walk.next(o);
            j = o.j0;
            j1 = o.j1;
          }
          if (valid) {
            c.o = o;
            c.o.j0 = j;
            j = min(j + kPartTiles, j1);
            c.o.j1 = j;
            c.kind = (first ? kPartFirst : 0) | (o.whole() && j == j1 ? kPartEnd : 0) | (o.j0 == o.T0 ? kPartBegins : 0);
            c.last_cta = 0;
            if (o.j0 == o.T0 && !o.whole()) c.last_cta = attn_last_cta(blockIdx.x, share, o);
            c.tok0 = p.div_g.div(o.row0);
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
            const int pg = p.div_page.div(key);
            const int e = pg < p.table_stride ? __ldg(trow + pg) : -1;
            if (e >= 0 && e < p.block_num) row = e * p.page + (key - pg * p.page);
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
      // the whole warp keeps the loop (its values stay uniform), one lane issues
      constexpr uint32_t idesc_qk = sm100::idesc_16bit_f32(kRows, KT, BF16, false);
      const uint32_t idesc_pv = sm100::idesc_16bit_f32(kRows, p.D, BF16, true);
      const int ks = p.D / 16;
      const bool leader = sm100::elect_one();
      const uint32_t q_lo = sm100::sw128_lo(sm100::smem_u32(qs), 16), k_lo = sm100::sw128_lo(sm100::smem_u32(ring), 16),
                     v_lo = sm100::sw128_lo(sm100::smem_u32(ring), KT * 128);
      uint32_t nq = 0, nh = 0, np = 0;  // parities of the next Q tile and halves of P, bit w: row tile w
      int st = 0;                // ring stage of the next K or V tile
      uint32_t par = 0;          // and its parity
      bool ok = true;
      auto take = [&](uint64_t* bar, uint32_t& parities, int w) {
        ok = __all_sync(0xffffffffu, ok && sm100::mbar_wait(bar + w, (parities >> w) & 1u, &abort_flag));
        parities ^= 1u << w;
        sm100::tc_fence_after();
      };
      auto stage = [&]() {  // wait for the next tile; its stage
        ok = __all_sync(0xffffffffu, ok && sm100::mbar_wait(&bars.full[st], par, &abort_flag));
        sm100::tc_fence_after();
        const int s = st;
        if (++st == C::kStages) {
          st = 0;
          par ^= 1u;
        }
        return s;
      };
      auto commit = [&](uint64_t* bar) {
        if (leader) sm100::mma_commit(bar);
      };
      auto qk = [&](int w, int s) {
        const uint32_t a = q_lo + (uint32_t)w * (C::kQBytes >> 4), b = k_lo + (uint32_t)s * (C::kTileBytes >> 4);
        if (leader) {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            if (k < ks)
              sm100::mma_ss(tmem + w * KT, a + (((k >> 2) * (kRows * 128) + (k & 3) * 32) >> 4), sm100::kSw128Hi,
                            b + (((k >> 2) * (KT * 128) + (k & 3) * 32) >> 4), sm100::kSw128Hi, idesc_qk, k > 0);
          sm100::mma_commit(&bars.s_full[w]);
        }
        __syncwarp();
      };
      auto pv_half = [&](int w, int s, bool first, int k0) {
        const uint32_t b = v_lo + (uint32_t)s * (C::kTileBytes >> 4) + k0 * (2048 >> 4);
        if (leader) {
#pragma unroll
          for (int k = 0; k < KT / 32; ++k)
            sm100::mma_ts(tmem + C::kTiles * KT + w * DP, tmem + w * KT + (k0 + k) * 8, b + k * (2048 >> 4),
                          sm100::kSw128Hi, idesc_pv, !first || k0 + k > 0);
        }
        __syncwarp();
      };
      auto pv = [&](int w, int s, bool first) {
        take(bars.p_half, nh, w);
        if (ok) pv_half(w, s, first, 0);
        take(bars.p_ready, np, w);
        if (ok) pv_half(w, s, first, KT / 32);
      };
      for (int pi = 0; ok; ++pi) {
        const ChunkPiece* c = piece(pi);
        ok = __all_sync(0xffffffffu, c != nullptr);
        if (!ok || !c->valid) break;
        const bool keys = c->o.hi > c->o.lo;
        const int act = c->o.rows > kRows ? 2 : 1;
        const int cnt = c->o.j1 - c->o.j0;
        __syncwarp();
        if (leader) piece_done(pi);
        if (!keys) continue;
        int kst = stage();
        for (int w = 0; w < act; ++w) {
          take(bars.q_ready, nq, w);
          if (ok) qk(w, kst);
        }
        if (ok) commit(&bars.empty[kst]);
        for (int i = 0; ok && i < cnt; ++i) {
          const bool more = i + 1 < cnt;
          const int vst = stage();
          pv(0, vst, i == 0);
          if (!ok) break;
          if (more) {
            kst = stage();
            if (ok) qk(0, kst);
          } else {
            commit(&bars.o_full[0]);
          }
          if (act == 2) {
            pv(1, vst, i == 0);
            if (!ok) break;
            if (more) qk(1, kst);
            else commit(&bars.o_full[1]);
          }
          commit(&bars.empty[vst]);
          if (more) commit(&bars.empty[kst]);
        }
      }
      // no product is in flight when the columns are freed
      commit(&bars.last);
      if ((!sm100::mbar_wait_bounded(&bars.last, 0, 20000000ull) || !ok) && leader) atomicOr(&g_attn_err, kErrTimeout);
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
    // (an access of the warp is 4 rows x 128 bytes: row 4 j + lane / 8, 64-channel block b)
    constexpr int kCols = DP / 8, kBlk = DP / 64;  // 16-byte chunks and blocks per row
    uint4 qreg[8 * kBlk];
    const int lrow = lane >> 3, lch = lane & 7;
    const int wrow = w * kRows + (warp & 3) * 32;  // first row of the warp within an item
    auto active = [&](const ChunkPiece* c) { return c->valid && c->o.hi > c->o.lo && c->o.rows > w * kRows; };
    // lrow as a value the compiler knows nothing of: what follows from it is computed
    // where it is used, not kept in registers across the tiles
    auto fresh = [&]() {
      int v = lrow;
      asm volatile("" : "+r"(v));
      return v;
    };
    auto load_q = [&](const ChunkPiece* c, bool there) {  // not there: zeros (and no register stays live)
      const uint16_t* base = p.q + (int64_t)(c->o.s.t0 + c->tok0) * p.q_stride + (int64_t)c->o.h * p.G * p.D + lch * 8;
      const int rows = there && active(c) ? c->o.rows : 0, rem0 = c->rem0, row = fresh();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int x = wrow + 4 * j + row;
        const int tok = p.div_g.div(rem0 + x), head = rem0 + x - tok * p.G;
        const uint16_t* src = base + (int64_t)tok * p.q_stride + head * p.D;
#pragma unroll
        for (int b = 0; b < kBlk; ++b) {
          qreg[j * kBlk + b] = make_uint4(0, 0, 0, 0);
          if (x < rows && b * 64 + lch * 8 < p.D) qreg[j * kBlk + b] = __ldg(reinterpret_cast<const uint4*>(src + b * 64));
        }
      }
    };
    // the lane's chunk of row 4 j + lrow of the warp's 32, block b, in the Q tile
    auto q_at = [&](int row, int j, int b) {  // row = lrow; (4 j + lrow) & 7 = lrow + 4 (j & 1)
      return reinterpret_cast<uint4*>(qw + ((warp & 3) * 32 + row) * 128 + j * 512 + b * (kRows * 128) +
                                      ((lch ^ (row + 4 * (j & 1))) << 4));
    };
    const ChunkPiece* c = &pieces[0];
    ok = __all_sync(0xffffffffu, piece(0) != nullptr);
    load_q(c, ok);
    for (int pi = 0; ok && c->valid; ++pi) {
      const int row = w * kRows + r;  // of the item
      const bool mine = row < c->o.rows;
      const uint32_t kind = c->kind;
      if (tid == 0 && (kind & kPartFirst) && c->last_cta) {
        attn_write_desc(p, blockIdx.x, c->last_cta, &c->o);
        begun = true;
      }
      auto out_row = [&]() {  // of out and lse
        const int tok = p.div_g.div(c->rem0 + row);
        return (int64_t)(c->o.s.t0 + c->tok0 + tok) * p.Hq + c->o.h * p.G + c->rem0 + row - tok * p.G;
      };
      if (c->o.hi <= c->o.lo && mine) {
        const int64_t orow = out_row();
        for (int e = 0; e < p.D; e += 8)
          *reinterpret_cast<uint4*>(p.out + orow * p.D + e) = make_uint4(0, 0, 0, 0);
        if (p.lse) p.lse[orow] = neg_inf();
      }
      const int cnt = c->o.hi > c->o.lo ? c->o.j1 - c->o.j0 : 0;
      const bool act = active(c);
      const bool warp_rows = wrow < c->o.rows;
      float ref = neg_inf(), l = 0.f;  // reference (log2 units) and sum of the row's weights
      if (act) {
        const int qrow = fresh();
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int b = 0; b < kBlk; ++b) *q_at(qrow, j, b) = qreg[j * kBlk + b];
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&bars.q_ready[w]);
        int lo = 0, hi = INT32_MAX;  // of a row that is not there: nothing to mask
        if (mine) {
          hi = attn_keys(p, c->o.s.start + c->tok0 + p.div_g.div(c->rem0 + row) + 1);
          lo = p.window ? max(0, hi - p.window) : 0;
        }
        for (int i = 0; i < cnt; ++i, n += 2) {
          const int key0 = (c->o.j0 + i) * KT;
          ok = sm100::mbar_wait(&bars.s_full[w], ns++ & 1u, &abort_flag) && ok;
          ok = __all_sync(0xffffffffu, ok);
          if (key0 < c->o.lo || key0 + KT > c->o.hi) {
            // values behind the sequence's end (or before the window) may hold
            // anything, a NaN times a weight of 0 included: make them zeros. Only now:
            // these scores say that the ring has come to this tile. A row tile without
            // rows lets its warps run pieces ahead, and the parity of a stage cannot tell
            // its phase from the one two rounds before.
            const int st = (n + 1) % C::kStages, klo = c->o.lo, khi = c->o.hi;
            ok = __all_sync(0xffffffffu, ok && sm100::mbar_wait(&bars.full[st], (uint32_t)((n + 1) / C::kStages) & 1u, &abort_flag));
            unsigned char* vt = ring + (size_t)st * C::kTileBytes;
            for (int e = r; ok && e < KT * kCols; e += kRows) {
              const int k = e / kCols, ch = e % kCols;
              if (key0 + k < klo || key0 + k >= khi)
                *reinterpret_cast<uint4*>(vt + (ch >> 3) * (KT * 128) + k * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            // lane 0 arrives for the warp; a warp without rows does so with nothing else between
            __syncwarp();
          }
          if (!ok) break;
          sm100::tc_fence_after();
          if (warp_rows) {
            uint32_t x[KT / 32][32];
#pragma unroll
            for (int b = 0; b < KT / 32; ++b) sm100::tmem_ld32(s_t + b * 32, x[b]);
#pragma unroll
            for (int b = 0; b < KT / 32; ++b) sm100::tmem_ld_wait(x[b]);
            const int clo = lo - key0, chi = hi - key0;  // the row's visible columns
            const bool edge = __any_sync(0xffffffffu, clo > 0 || chi < KT);
            if (edge) {
#pragma unroll
              for (int e = 0; e < KT; ++e)
                if (e < clo || e >= chi) x[e / 32][e % 32] = 0xff800000u;
            }
            float mx4[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
            for (int e = 0; e < KT; e += 2)
              mx4[e / 2 % 4] =
                  max3(mx4[e / 2 % 4], __uint_as_float(x[e / 32][e % 32]), __uint_as_float(x[e / 32][e % 32 + 1]));
            const float mx = p.scale_log2 * max3(max3(mx4[0], mx4[1], mx4[2]), mx4[3], mx4[3]);
            const bool grow = mx > ref + kLazy;  // also the first visible key's tile; not a NaN
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
            const uint64_t scale2 = sm100::f2_pack(p.scale_log2, p.scale_log2), base2 = sm100::f2_pack(base, base);
            uint64_t sum2[2] = {0, 0};
#pragma unroll
            for (int b = 0; b < KT / 32; ++b) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float u0, u1;
                sm100::f2_unpack(sm100::f2_fma(sm100::f2_pack(__uint_as_float(x[b][2 * e]), __uint_as_float(x[b][2 * e + 1])),
                                               scale2, base2),
                                 u0, u1);
                u0 = ex2(u0);
                u1 = ex2(u1);
                sum2[e & 1] = sm100::f2_add(sum2[e & 1], sm100::f2_pack(u0, u1));
                pk[e] = pack2<BF16>(u0, u1);
              }
              sm100::tmem_st16(s_t + b * 16, pk);
              if (b == KT / 64 - 1) {  // the first half's product may start
                sm100::tmem_st_wait();
                sm100::tc_fence_before();
                __syncwarp();
                if (lane == 0) sm100::mbar_arrive(&bars.p_half[w]);
              }
            }
            float s0, s1, s2, s3;
            sm100::f2_unpack(sum2[0], s0, s1);
            sm100::f2_unpack(sum2[1], s2, s3);
            l += (s0 + s1) + (s2 + s3);
            sm100::tmem_st_wait();
          } else if (lane == 0) {
            sm100::mbar_arrive(&bars.p_half[w]);
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
      const ChunkPiece* next = &pieces[(pi + 1) % kPieces];
      ok = __all_sync(0xffffffffu, piece(pi + 1) != nullptr);
      load_q(next, ok);
      if (!ok) break;
      if (act) {
        ok = sm100::mbar_wait(&bars.o_full[w], no++ & 1u, &abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        sm100::tc_fence_after();
        if (warp_rows) {
          const bool finish = kind & kPartEnd;
          // slot 1 is also where the parts of a whole item are added: the piece that a CTA
          // begins and does not end is its last one
          const int64_t slot = (int64_t)blockIdx.x * 2 + ((kind & kPartBegins) ? 1 : 0);
          if (!(kind & kPartFirst)) {
            const float2 ml = add_part(o_t, attn_chunk_part(p, DP, C::kM, slot, 0, row), C::kM * 4,
                                       p.part_ml + (slot * C::kM + row) * 2, p.D, mine, ref, l);
            ref = ml.x;
            l = ml.y;
          }
          const float inv = l == 0.f ? 0.f : 1.f / l;
          unsigned char* orow_s = qw + r * 128;  // whole rows pass through the warp's part of the Q tile
#pragma unroll
          for (int d = 0; d < DP; d += 32) {
            uint32_t a[32];
            sm100::tmem_ld32(o_t + d, a);
            sm100::tmem_ld_wait(a);
            if (finish) {
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
                *reinterpret_cast<uint4*>(attn_chunk_part(p, DP, C::kM, slot, (d + e) / 4, row)) =
                    make_uint4(a[e], a[e + 1], a[e + 2], a[e + 3]);
              }
            }
          }
          if (finish) {
            __syncwarp();
            const int rows = c->o.rows, rem0 = c->rem0, qrow = fresh();
            uint16_t* base =
                p.out + ((int64_t)(c->o.s.t0 + c->tok0) * p.Hq + (int64_t)c->o.h * p.G) * p.D + lch * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int x = wrow + 4 * j + qrow;
              const int t = p.div_g.div(rem0 + x), head = rem0 + x - t * p.G;
              uint16_t* dst = base + ((int64_t)t * p.Hq + head) * p.D;
#pragma unroll
              for (int b = 0; b < kBlk; ++b) {
                const uint4 v = *q_at(qrow, j, b);
                if (x < rows && b * 64 + lch * 8 < p.D) *reinterpret_cast<uint4*>(dst + b * 64) = v;
              }
            }
          }
          if (mine) {
            if (!finish) *reinterpret_cast<float2*>(p.part_ml + (slot * C::kM + row) * 2) = make_float2(ref, l);
            else if (p.lse) p.lse[out_row()] = attn_lse(ref, l);
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

cudaError_t attn_chunk_error_word(unsigned** word) { return cudaGetSymbolAddress((void**)word, g_attn_err); }

}  // namespace cmp
