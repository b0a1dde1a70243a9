// Attention of a chunk of new tokens over a paged cache: what its kernels share
// (the call's parameters, the division of the work, the joining of split rows).
//
// A token at position p sees the first n(p) keys of its sequence,
//   n(p) = 0 if p + 1 < key_block, else (p + 1 - key_block) / key_stride + 1,
// (key j stands for positions j*key_stride .. j*key_stride + key_block - 1), of
// those the last `window` if there is a window. The query heads of one key head
// are rows of the same tile: row r of a (sequence, key head) is token r / G, query
// head r % G of the group of G = Hq / Hk.
//
// Work: an item is a tile of M rows of one (sequence, key head); its units are
// kItemCost for loading its queries and storing its rows, then the tiles of KT keys
// that any of its rows sees (an item without keys has one empty tile, so that its
// rows are written). All units of a call form a line,
// sequence by sequence, head by head, row tile by row tile, and CTA c takes the
// c-th of equal parts of it, whatever the lengths are. An item that a part's end
// cuts is finished in pieces: each piece leaves its fp32 accumulator and its
// softmax statistics in the workspace (a CTA leaves at most two: slot 0 for an
// item begun by an earlier CTA, slot 1 for one that it begins and does not end),
// and attn_combine_kernel joins them in the order of the keys.
//
// Roundings to 16 bits: the weights, before their product with V (the tensor core
// takes both factors in one 16-bit type; fp32 weights would cost a second product,
// half as much again in chunks, for an error below out's own rounding), and out. Each
// weight is off by at most half a step, to either side; their sum l stays fp32.
#pragma once

#include "cmp_internal.cuh"
#include "cmp_sm100.cuh"

#include <cuda_fp16.h>

namespace cmp {

struct AttnParams {
  const uint16_t* q;         // token t at q + t * q_stride, its [Hq, D] dense
  const int32_t* table;      // [B, table_stride]
  const int32_t* cu;         // [B + 1]
  const int32_t* start_pos;  // [B] or null
  uint16_t* out;             // [T, Hq, D]
  float* lse;                // [T, Hq] or null
  float* part;               // workspace: accumulators of cut items, ctas x 2 slots of M x DP (decoding:
                             // row by row; chunks: see attn_chunk_part)
  float* part_ml;            // [ctas][2][M][2]: running maximum (log2 units), sum
  int4* desc;                // [ctas][2]: the item a CTA begins and does not end
  int64_t q_stride, table_stride, block_num;
  int B, T, Hq, Hk, G, D, page, bf16;
  FastDiv div_g, div_stride, div_page;  // by G, key_stride, page
  int key_block, key_stride, window;    // window 0: none
  int max_len;
  int withhold;       // testing: no tile is loaded, every wait for one runs out (decoding)
  int run_shift;      // keys per TMA box: 1 << run_shift, a divisor of the page
  float scale_log2;   // scale * log2(e)
};

struct AttnSeq {
  int t0, len, start;  // first row of q, tokens, position of the first one
  bool bad;
};

// Positions a sequence may have: the keys of the last tile, and of the run behind
// it, still have 32-bit numbers.
constexpr int64_t kMaxPositions = INT32_MAX - 1024;

// Sequences of a call. A CTA passes those without tokens in its part one after another (0.2 us
// each: 206 ms for 2^20 between two that have some), while its other warps wait for the next
// piece of work, for at most two seconds.
constexpr int64_t kMaxSequences = 1 << 20;

// Sequence b, with length 0 if its entries are not usable (bad is set then).
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int b) {
  AttnSeq s;
  const int c = __ldg(p.cu + b), e = __ldg(p.cu + b + 1);
  s.start = p.start_pos ? __ldg(p.start_pos + b) : 0;
  s.t0 = c;
  s.len = e - c;
  s.bad = c < 0 || e < c || e > p.T || s.start < 0 || (b == 0 && c != 0) ||
          (int64_t)s.start + (e - c) > kMaxPositions || s.len > p.max_len;
  if (s.bad) s.len = 0;
  return s;
}

__device__ __forceinline__ int attn_keys(const AttnParams& p, int p1) {  // p1 = position + 1
  if (p.key_stride == 1) return max(p1 - p.key_block + 1, 0);
  return p1 < p.key_block ? 0 : p.div_stride.div(p1 - p.key_block) + 1;
}

// Keys [lo, hi) that any of the rows [row0, row0 + rows) sees; hi <= lo: none.
__device__ __forceinline__ void attn_range(const AttnParams& p, const AttnSeq& s, int row0, int rows, int& lo,
                                           int& hi) {
  hi = attn_keys(p, s.start + p.div_g.div(row0 + rows - 1) + 1);
  lo = p.window ? max(0, attn_keys(p, s.start + p.div_g.div(row0) + 1) - p.window) : 0;
}

// The visible keys [lo, hi) of one row.
__device__ __forceinline__ void attn_row_range(const AttnParams& p, const AttnSeq& s, int row, int& lo, int& hi) {
  hi = attn_keys(p, s.start + p.div_g.div(row) + 1);
  lo = p.window ? max(0, hi - p.window) : 0;
}

// One piece of an item: tiles [j0, j1) of its [T0, T1).
struct AttnPiece {
  AttnSeq s;
  int b, h;        // sequence, key head
  int row0, rows;  // rows of the (sequence, key head)
  int lo, hi;      // keys any row sees (hi <= lo: none)
  int T0, T1, j0, j1;
  __device__ __forceinline__ bool whole() const { return j0 == T0 && j1 == T1; }
};

// Tiles [T0, T1) of keys [lo, hi); one empty tile without keys.
template <int KT>
__device__ __forceinline__ void attn_tiles(int lo, int hi, int& T0, int& T1) {
  T0 = hi > lo ? lo / KT : 0;
  T1 = hi > lo ? (hi + KT - 1) / KT : 1;
}

// What an item costs beside its tiles, in tiles. Measured on items of one to three
// tiles of the chunk kernel: 6 us each beside 1.5 to 2 us per tile. Without it a batch
// that mixes short and long contexts waits for the CTAs whose parts are all short
// items: 16 tokens of 16 heads each over compressed rows took 322 us, with it 155 us
// (with a cost of 1 or 5 tiles 3 to 5 % more).
constexpr int kItemCost = 3;

// Row tiles of one key head of a sequence.
template <int M>
__device__ __forceinline__ int attn_row_tiles(const AttnParams& p, const AttnSeq& s) {
  return (int)(((uint32_t)s.len * (uint32_t)p.G + (M - 1)) / M);  // T * Hq <= INT32_MAX
}

// n / d, in 32 bits where they suffice (a 64-bit division takes half a microsecond).
__device__ __forceinline__ int64_t attn_div64(int64_t n, int64_t d) {
  if (((n | d) >> 32) == 0) return (int64_t)((uint32_t)n / (uint32_t)d);
  return n / d;
}

// A CTA's way along its part of the line. M rows per item.
template <int KT, int M>
struct AttnWalk {
  const AttnParams& p;
  int64_t left;  // units still to do
  int b, h, qt, off;
  int nq;
  AttnSeq s;
  __device__ __forceinline__ AttnWalk(const AttnParams& p_) : p(p_) {}
  __device__ __forceinline__ void open() {
    s = attn_seq(p, b);
    nq = attn_row_tiles<M>(p, s);
  }
  __device__ __forceinline__ void begin(int64_t units, int b_, int h_, int qt_, int off_) {
    left = units;
    b = b_;
    h = h_;
    qt = qt_;
    off = off_;
    if (left > 0) open();
  }
  __device__ __forceinline__ bool next(AttnPiece& o) {
    while (left > 0) {
      while (qt >= nq) {
        qt = 0;
        if (++h >= p.Hk) {
          h = 0;
          if (++b >= p.B) return false;
          open();
        }
        if (nq == 0) h = p.Hk - 1;
      }
      o.s = s;
      o.b = b;
      o.h = h;
      o.row0 = qt * M;
      o.rows = min(M, s.len * p.G - o.row0);
      attn_range(p, s, o.row0, o.rows, o.lo, o.hi);
      attn_tiles<KT>(o.lo, o.hi, o.T0, o.T1);
      const int n = o.T1 - o.T0 + kItemCost;
      const int take = (int)min(left, (int64_t)(n - off));
      o.j0 = o.T0 + max(off - kItemCost, 0);
      o.j1 = o.T0 + max(off + take - kItemCost, 0);
      left -= take;
      off += take;
      if (off >= n) {
        off = 0;
        ++qt;
      }
      if (o.j1 > o.j0) return true;  // else the part ends before the item's first tile: the next CTA begins it
    }
    return false;
  }
};

// Where a CTA's part begins, found by all NT threads of the CTA together.
struct AttnStart {
  int64_t share, units;  // units per CTA; this CTA's units
  int b, h, qt, off;
};

// Units of row tile qt of one key head of sequence s.
template <int KT, int M>
__device__ __forceinline__ int attn_tile_units(const AttnParams& p, const AttnSeq& s, int qt) {
  int lo, hi, T0, T1;
  const int r = qt * M;
  attn_range(p, s, r, min(M, s.len * p.G - r), lo, hi);
  attn_tiles<KT>(lo, hi, T0, T1);
  return T1 - T0 + kItemCost;
}

// Units of one key head of each lane's sequence, by the whole warp: sequences of
// few row tiles by their own lane, the others by all lanes one after another.
template <int KT, int M>
__device__ __forceinline__ int64_t attn_head_units(const AttnParams& p, const AttnSeq& s, int lane) {
  const int nq = attn_row_tiles<M>(p, s);
  int64_t n = 0;
  if (nq <= 4)
    for (int qt = 0; qt < nq; ++qt) n += attn_tile_units<KT, M>(p, s, qt);
  for (unsigned big = __ballot_sync(0xffffffffu, nq > 4); big; big &= big - 1) {
    const int src = __ffs(big) - 1;
    AttnSeq t;
    t.len = __shfl_sync(0xffffffffu, s.len, src);
    t.start = __shfl_sync(0xffffffffu, s.start, src);
    const int tq = __shfl_sync(0xffffffffu, nq, src);
    int64_t part = 0;
    for (int qt = lane; qt < tq; qt += 32) part += attn_tile_units<KT, M>(p, t, qt);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == src) n = part;
  }
  return n;
}

// Every thread sums its run of consecutive sequences, the block scans the sums,
// and the warp whose run holds the part's first unit walks to it. *err gets
// kErrIndex from CTA 0 if a sequence is not usable. Ends with __syncthreads.
template <int KT, int M, int NT>
__device__ __forceinline__ void attn_plan(const AttnParams& p, AttnStart* st, int64_t* warp_sum, unsigned* err) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + NT - 1) / NT;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int64_t sum = 0;
  bool bad = false;
  for (int i = 0; i < per; ++i) {  // lanes of a warp together
    AttnSeq s;
    s.t0 = s.len = s.start = 0;
    s.bad = false;
    if (b0 + i < b1) s = attn_seq(p, b0 + i);
    bad |= s.bad;
    sum += attn_head_units<KT, M>(p, s, lane) * p.Hk;
  }
  if (bad && blockIdx.x == 0) atomicOr(err, kErrIndex);
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) warp_sum[warp] = inc;
  if (tid == 0) st->units = 0;
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < (NT + 31) / 32; ++w) {
    if (w < warp) base += warp_sum[w];
    total += warp_sum[w];
  }
  base += inc - sum;
  const int64_t share = attn_div64(total + gridDim.x - 1, gridDim.x);
  int64_t u = (int64_t)blockIdx.x * share;
  // the warp whose run holds unit u walks to it, 32 row tiles at a time
  const unsigned owner = __ballot_sync(0xffffffffu, u < total && u >= base && u < base + sum);
  if (owner) {
    const int src = __ffs(owner) - 1;
    const int sb0 = __shfl_sync(0xffffffffu, b0, src), sb1 = __shfl_sync(0xffffffffu, b1, src);
    int64_t v = u - __shfl_sync(0xffffffffu, base, src);
    for (int b = sb0; b < sb1; ++b) {
      const AttnSeq s = attn_seq(p, b);
      const int nq = attn_row_tiles<M>(p, s);
      int64_t hu = 0;
      for (int qt = lane; qt < nq; qt += 32) hu += attn_tile_units<KT, M>(p, s, qt);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) hu += __shfl_xor_sync(0xffffffffu, hu, o);
      if (v >= hu * p.Hk) {
        v -= hu * p.Hk;
        continue;
      }
      const int h = (int)attn_div64(v, hu);
      v -= h * hu;
      for (int qt0 = 0;; qt0 += 32) {
        const int n = qt0 + lane < nq ? attn_tile_units<KT, M>(p, s, qt0 + lane) : 0;
        int64_t c = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t t = __shfl_up_sync(0xffffffffu, c, o);
          if (lane >= o) c += t;
        }
        const unsigned past = __ballot_sync(0xffffffffu, v < c);
        if (past) {
          if (lane == __ffs(past) - 1) {
            st->share = share;
            st->units = min(share, total - u);
            st->b = b;
            st->h = h;
            st->qt = qt0 + lane;
            st->off = (int)(v - (c - n));
          }
          break;
        }
        v -= __shfl_sync(0xffffffffu, c, 31);
      }
      break;
    }
  }
  __syncthreads();
}

// Four channels (group c4) of a row of a slot of the chunk kernel: the rows of one
// group lie side by side, so that the threads of a warp, a row each, write (and the
// combine kernel reads) 512 contiguous bytes. Row by row, a piece of 256 rows of 192
// channels took 8 us to leave.
__device__ __forceinline__ float* attn_chunk_part(const AttnParams& p, int dp, int m, int64_t slot, int c4, int row) {
  return p.part + ((slot * (dp / 4) + c4) * m + row) * 4;
}

// The CTA's note on the item that it begins and leaves to later CTAs: the last
// of them (0: there is none; CTA 0 is never one), the rows and where they go.
__device__ __forceinline__ void attn_write_desc(const AttnParams& p, int cta, int last_cta, const AttnPiece* o) {
  p.desc[2 * cta] = o ? make_int4(last_cta, o->rows, o->s.t0, o->row0) : make_int4(0, 0, 0, 0);
  if (o) p.desc[2 * cta + 1] = make_int4(o->h, 0, 0, 0);
}

// The last CTA of the item of a piece that its CTA does not end: `rest` tiles
// follow, the next CTAs do `share` each.
__device__ __forceinline__ int attn_last_cta(int cta, int64_t share, const AttnPiece& o) {
  return cta + (int)attn_div64(o.T1 - o.j1 + share - 1, share);
}

// Row r of a piece's item -> the row of out / lse ([T * Hq]).
__device__ __forceinline__ int64_t attn_out_row(const AttnParams& p, int t0, int h, int r) {
  const int t = p.div_g.div(r);
  return (int64_t)(t0 + t) * p.Hq + h * p.G + (r - t * p.G);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }

// log of sum exp from the running maximum (log2 units) and the sum.
__device__ __forceinline__ float attn_lse(float m, float l) {
  return l == 0.f ? neg_inf() : fmaf(m, 0.69314718055994531f, logf(l));  // a NaN stays one
}

// Accumulator columns of a head of D channels: a multiple of 64.
inline int attn_padded(int D) { return (D + 63) / 64 * 64; }

// Host: the cache as a 3-D tensor (d, key head, row) with boxes of 64 channels of
// one head over 1 << run_shift rows, landing 128-byte swizzled.
bool attn_cache_map(CUtensorMap* m, const void* cache, const AttnParams& p);

// Decoding: items of 8 or 16 rows (`m`).
constexpr int kAttnDecodeRows = 16;  // the most rows per key head and sequence it runs with
int attn_decode_rows(int64_t rows);
int attn_decode_ctas(int D, int sms);
cudaError_t launch_attn_decode(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s,
                               int ctas, int m);
cudaError_t attn_decode_error_word(unsigned** word);
// Chunks: 128-row MMA tiles, one CTA per SM.
int attn_chunk_rows(int D);      // rows per item
int attn_chunk_key_tile(int D);  // keys per tile
cudaError_t launch_attn_chunk(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s,
                              int ctas);
cudaError_t attn_chunk_error_word(unsigned** word);
cudaError_t launch_attn_combine(const AttnParams& p, int m, int ctas, cudaStream_t s);

}  // namespace cmp
