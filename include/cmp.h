/*
 * cmp.h — C ABI of the B200 streaming KV-cache Compressor.
 *
 * One call compresses every ratio-token window that the call completes into
 * one bf16 row of D channels (DeepSeek-V4 C4A / C4Li / C128A attention):
 *
 *   1. dual projection   kv = x·Wkvᵀ,  score = x·Wgateᵀ + ape[p mod ratio]
 *      ("compressor torch_extension API", 计算公式 1-2; "CANN PyPTO 算子实战:
 *      Compressor", 主要计算过程);
 *   2. per-window pooling: a per-channel softmax over the window's rows weights
 *      a sum of its kv rows; for ratio 4 (coff 2) a window pairs columns [0, D)
 *      of the previous window's 4 rows with columns [D, 2D) of its own 4 rows,
 *      and the first window of a sequence has no previous rows
 *      ("compressor torch_extension API", 计算公式 2-5; "NPU DeepSeek-V4 Ascend C
 *      融合算子优化", Compressor 计算公式; "CANN PyPTO 算子实战", 压缩窗口与状态更新);
 *   3. RMSNorm (eps 1e-6) with norm_weight, interleaved RoPE on the last
 *      rope_head_dim channels, and, if rotate, a product with the D×D hadamard
 *      matrix ("CANN PyPTO 算子实战", 压缩窗口与状态更新, kernel 派发逻辑).
 *
 * Streaming: kv_state / score_state keep, in fp32, the projected rows of
 * windows a later call still has to pool. They are paged: position p of
 * sequence b lives in slot (table[b][p / block_size], p % block_size) of its
 * pool, with kv_block_table for kv_state and state_block_table for
 * score_state ("CANN PyPTO 算子实战", 参数说明; "Triton-Ascend Compressor",
 * state_block_table example). A call reads slots of positions before
 * start_pos[b] and writes slots of positions from start_pos[b] on, so the
 * slots it reads and the slots it writes are disjoint and an identical call
 * repeated gives identical results.
 *
 * Conventions for every entry point below:
 *  - bf16 tensors are passed as cmp_bf16 (their 16-bit patterns);
 *  - all tensors are dense, row-major and contiguous;
 *  - "device" pointers are CUDA device memory of the current device, owned by
 *    the caller (the library never frees or keeps them past the call);
 *  - "host" pointers are ordinary host memory;
 *  - entry points returning int return a cmp_status.
 */
#ifndef CMP_H_
#define CMP_H_

#include <stdbool.h>
#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define CMP_API __attribute__((visibility("default")))
#else
#define CMP_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t cmp_bf16;

typedef enum cmp_status {
  CMP_OK = 0,
  CMP_ERR_NULLPTR = 1,      /* a required pointer is NULL */
  CMP_ERR_INVALID = 2,      /* a size or argument outside the supported range */
  CMP_ERR_UNSUPPORTED = 3,  /* a ratio the library does not implement */
  CMP_ERR_CUDA = 4,         /* a CUDA runtime call or kernel launch failed */
  CMP_ERR_DEVICE_INDEX = 5, /* a kernel met a bad index (see cmp_get_error) */
  CMP_ERR_TIMEOUT = 6       /* a kernel gave up waiting on its own pipeline */
} cmp_status;

/* Shape scalars of one call; the pages' operator reads them from tensor shapes.
 *   B            sequences (requests) in the call, >= 0
 *   T            total tokens = rows of x = cu_seqlens[B], >= 0
 *   H            hidden size: a multiple of 512 in [512, 16384]
 *   D            compressed row width: 128 or 512
 *   block_num    pool rows of kv_state and of score_state, >= 1
 *   block_size   positions per pool row, in [1, 1024]
 *   table_stride columns of kv_block_table and state_block_table, >= 1
 * ("compressor torch_extension API", 约束说明: D in {128, 512}; H a multiple of
 * 512; block_size 1..1024. H down to 512 is accepted for small tests.) */
typedef struct cmp_dims {
  int32_t B;
  int32_t T;
  int32_t H;
  int32_t D;
  int32_t block_num;
  int32_t block_size;
  int32_t table_stride;
} cmp_dims;

/* Rows of out, sin and cos: min(T, T / ratio + B)
 * ("CANN PyPTO 算子实战", 返回值说明: out is [min(T, T//ratio + B), D]).
 * Returns -1 if ratio < 1, B < 0 or T < 0. Host only. */
CMP_API int64_t cmp_out_rows(int64_t B, int64_t T, int32_t ratio);

/* Host-side output-row layout, for callers that build sin/cos per row.
 * Window w of sequence b completes when the token at position (w+1)*ratio - 1
 * arrives ("CANN PyPTO 算子实战", 数值精度与验证要点: (start_pos + i + 1) % ratio == 0).
 * Sequence b reserves cap_b = min(L_b, L_b / ratio + 1) consecutive rows after
 * those of sequences 0..b-1; its k-th completed window goes to the k-th of
 * them. For every row n < n_out: row_seq[n] = b and row_window[n] = w if the
 * row holds window w of sequence b, else row_seq[n] = row_window[n] = -1.
 * cu_seqlens [B+1], start_pos [B] (NULL: all 0), row_seq / row_window
 * [n_out]: host memory. n_out must equal cmp_out_rows(B, cu_seqlens[B], ratio).
 * Errors: CMP_ERR_NULLPTR, CMP_ERR_INVALID (cu_seqlens not rising from 0,
 * start_pos < 0, n_out mismatch, positions past INT32_MAX). */
CMP_API int cmp_out_row_layout(const int32_t* cu_seqlens, const int32_t* start_pos, int32_t B,
                       int32_t ratio, int64_t n_out, int32_t* row_seq, int32_t* row_window);

/* The Compressor ("CANN PyPTO 算子实战", 函数原型 and 参数说明, plus cu_seqlens
 * for packed variable-length input from "compressor torch_extension API").
 *
 *  x                  device bf16 [T, H]; sequence b owns rows
 *                     cu_seqlens[b] .. cu_seqlens[b+1]-1, at absolute positions
 *                     start_pos[b], start_pos[b]+1, ...
 *  kv_state           device fp32 [block_num, block_size, coff*D], updated in place
 *  score_state        device fp32 [block_num, block_size, coff*D], updated in place
 *                     (holds x·Wgateᵀ + ape, as the pooling reads it)
 *  kv_block_table     device int32 [B, table_stride]: pool row of kv_state per block
 *  state_block_table  device int32 [B, table_stride]: pool row of score_state per block
 *                     Entries a call does not need are never read (may be -1).
 *  sin, cos           device bf16 [n_out, rope_head_dim]: RoPE tables of output
 *                     row n; element 2j of a pair uses column j, element 2j+1
 *                     column rope_head_dim/2 + j
 *  wkv, wgate         device bf16 [coff*D, H]
 *  ape                device fp32 [ratio, coff*D]: added to the score of the
 *                     token at position p from row p mod ratio
 *  norm_weight        device bf16 [D]
 *  hadamard           device bf16 [D, D] (out = out @ hadamard); NULL iff !rotate
 *  start_pos          device int32 [B]; NULL means every sequence starts at 0
 *  cu_seqlens         device int32 [B+1], rising from 0 to T
 *  ratio              tokens per window: 1, 2, 4, 8, 16, 32, 64 or 128;
 *                     coff = 2 for ratio 4, else 1 (ratio 1: every token is
 *                     its own window, so only projection and normalisation
 *                     remain, as the Triton-Ascend Compressor article notes)
 *  rope_head_dim      64 (the only value the pages support)
 *  rotate             apply the hadamard product
 *  out                device bf16 [n_out, D], n_out = cmp_out_rows(B, T, ratio);
 *                     every row is written (rows with no window: 0)
 *  stream             cudaStream_t to run on (NULL: the legacy default stream)
 *  dims               host pointer to the shape scalars
 *
 * State update: for sequence b with e = start_pos[b] + L_b, the rows of
 * positions p in [start_pos[b], e) with p >= (e/ratio - coff + 1)*ratio are
 * written to both states — exactly the rows a later call can still read. No
 * other state byte changes.
 *
 * Asynchronous on stream; no host synchronisation. The first call on a
 * (device, stream) pair allocates a workspace that later calls reuse (it grows
 * if a later call needs more); see cmp_workspace_size / cmp_release_workspaces.
 * Results are bitwise reproducible run to run (no floating-point atomics).
 * Requirements the library does not check: the pool rows used by different
 * sequences are disjoint, and the tables map the blocks a call needs (the Python
 * binding's debug_check_tables checks both on the host, for tests and debugging).
 *
 * Returns CMP_OK, CMP_ERR_NULLPTR, CMP_ERR_INVALID, CMP_ERR_UNSUPPORTED or
 * CMP_ERR_CUDA, all decided on the host before anything is launched, except
 * CMP_ERR_CUDA for a failed launch. B == 0 or T == 0 is a successful no-op.
 * Faults found inside kernels (a needed table entry outside [0, block_num) or
 * a block index past table_stride; cu_seqlens not rising from 0 to T;
 * start_pos < 0; positions past INT32_MAX) never trap: the access is skipped,
 * an error word on the device is set, and cmp_get_error reports it. */
CMP_API int cmp_compressor(const cmp_bf16* x, float* kv_state, float* score_state,
                   const int32_t* kv_block_table, const int32_t* state_block_table,
                   const cmp_bf16* sin, const cmp_bf16* cos, const cmp_bf16* wkv,
                   const cmp_bf16* wgate, const float* ape, const cmp_bf16* norm_weight,
                   const cmp_bf16* hadamard, const int32_t* start_pos, const int32_t* cu_seqlens,
                   int32_t ratio, int32_t rope_head_dim, bool rotate, cmp_bf16* out,
                   void* stream, const cmp_dims* dims);

/* No counterpart on the pages: an entry point for callers that must not
 * allocate device memory at call time (for example a serving engine that
 * reserves all device memory at start-up, or a caller running with the GPU
 * nearly full, where a cudaMalloc could fail or synchronise the device).
 *
 * Same arguments and results as cmp_compressor, for decode-sized calls:
 * T <= 64 tokens, and the call's scratch (error word, per-sequence metadata,
 * fp32 projection rows: about 12*B + 8*T*coff*D bytes) must fit a fixed
 * 1 MiB array in device memory that the library image carries; larger calls
 * return CMP_ERR_INVALID before launching anything. It never calls cudaMalloc,
 * cudaFree or any allocating routine.
 *
 * The first call on each device (with that device current) looks up the
 * array's device address once (cudaGetSymbolAddress); make that first call
 * before any stream capture. All calls on a device share the array, so calls
 * that overlap on the GPU race and must be ordered by the caller (one stream,
 * or events). The array keeps the last call's contents. Its error word starts
 * at zero when the library is loaded, kernels only set bits in it, and
 * cmp_get_error reads and clears it: device-side errors (a bad needed table
 * entry, cu_seqlens or start_pos) are reported by cmp_get_error(stream) on the
 * same device, once the calls' stream is synchronised (pass that stream).
 * After a device reset (cudaDeviceReset), call cmp_release_workspaces before
 * the next call: the array may move when the library image is loaded again,
 * and that call makes the next one look its address up afresh. */
CMP_API int cmp_compressor_noalloc(const cmp_bf16* x, float* kv_state, float* score_state,
                                   const int32_t* kv_block_table, const int32_t* state_block_table,
                                   const cmp_bf16* sin, const cmp_bf16* cos, const cmp_bf16* wkv,
                                   const cmp_bf16* wgate, const float* ape, const cmp_bf16* norm_weight,
                                   const cmp_bf16* hadamard, const int32_t* start_pos,
                                   const int32_t* cu_seqlens, int32_t ratio, int32_t rope_head_dim,
                                   bool rotate, cmp_bf16* out, void* stream, const cmp_dims* dims);

/* Synchronises stream, then returns and clears the error word the kernels of
 * the current device set: CMP_OK, CMP_ERR_DEVICE_INDEX or CMP_ERR_TIMEOUT
 * (CMP_ERR_CUDA if the synchronisation itself fails). Covers the calls made on
 * `stream` and, on the current device, every cmp_compressor_noalloc,
 * cmp_kv_append and cmp_paged_attention call that has finished. */
CMP_API int cmp_get_error(void* stream);

/* Bytes of device workspace a call with these shapes uses (the two-phase
 * "query the workspace, then run" pattern of the aclnn API on "NsaCompressWithCache").
 * Returns 0 for invalid dims. Host only. */
CMP_API size_t cmp_workspace_size(const cmp_dims* dims, int32_t ratio);

/* Frees every workspace the library holds (synchronises the devices first) and
 * forgets the cached device addresses of cmp_compressor_noalloc's array.
 * Returns CMP_OK or CMP_ERR_CUDA. */
CMP_API int cmp_release_workspaces(void);

/* Static text for a status code. */
CMP_API const char* cmp_status_string(int status);

/* ---- NsaCompressWithCache (a second workload) ------------------------------
 * "CANN ops-transformer 算子解析 NsaCompressWithCache" — 计算公式, 算法流程,
 * 参数说明, 约束说明. For each batch b with s = act_seq_len[b] (per-batch
 * lengths): if s >= compress_block_size and (s - compress_block_size) %
 * compress_stride == 0, then for every head n and channel d
 *   output_cache[slot_mapping[b], n, d] =
 *     round(sum_{j < compress_block_size} input[token s - compress_block_size + j of b, n, d] * weight[j, n])
 * with the products and the sum in fp32 and one round-to-nearest-even cast to
 * the cache dtype. Other slots are not touched. */
typedef struct {
  int64_t B;             /* batches: entries of slot_mapping and act_seq_len, at most 65535 */
  int64_t N;             /* heads, 1..64 (even when above 50) */
  int64_t D;             /* channels per head, a multiple of 16, at most 256 */
  int64_t tokens;        /* paged: block_num (input rows / page_block_size); packed: T, the input rows;
                            input rows at most INT32_MAX */
  int64_t table_stride;  /* paged: columns of block_table (pages per batch); packed: ignored */
  int64_t result_len;    /* rows of output_cache */
} cmp_nsa_dims;

enum { CMP_NSA_FP16 = 0, CMP_NSA_BF16 = 1 };
enum { CMP_NSA_PAGED = 0, CMP_NSA_PACKED = 1 };

/* input: device, dtype elements, paged [block_num, page_block_size, N, D]
 *   (a token at position p of batch b is at block block_table[b][p /
 *   page_block_size], row p % page_block_size) or packed [T, N, D] (batch b's
 *   tokens follow those of batches < b, in order); 16-byte aligned.
 * weight: device [compress_block_size, N], same dtype. slot_mapping: device
 * int32 [B], distinct values in [0, result_len). act_seq_len: device int64 [B].
 * block_table: device int32 [B, table_stride] (paged; NULL allowed when packed).
 * output_cache: device [result_len, N, D], same dtype, updated in place;
 * 16-byte aligned. The call is asynchronous on `stream` (a cudaStream_t, NULL =
 * default stream). It keeps its error word, and for the packed layout the B
 * batches' first rows (8 * B bytes), in the library's workspace for this device
 * and stream. Growing that workspace synchronises the device, so make the
 * largest call once before capturing calls into a CUDA graph, as for
 * cmp_compressor. All other memory is the caller's.
 * compress_block_size: a multiple of 16 in [16, 64], >= compress_stride;
 * compress_stride: 16, 32, 48 or 64; page_block_size: 64 or 128 (paged).
 * Returns CMP_OK, CMP_ERR_NULLPTR (a required pointer or dims is NULL),
 * CMP_ERR_INVALID (a size or alignment outside the ranges above),
 * CMP_ERR_UNSUPPORTED (dtype or layout value), CMP_ERR_CUDA (launch, or the driver
 * cannot describe the cache as a TMA tensor). B == 0
 * is a no-op. A slot outside [0, result_len), a needed table entry outside
 * [0, block_num) or packed rows past T set the device error word (the batch is
 * skipped; cmp_get_error reports CMP_ERR_DEVICE_INDEX). */
CMP_API int cmp_nsa_compress(const void* input, const void* weight, const int32_t* slot_mapping,
                             const int64_t* act_seq_len, const int32_t* block_table, int32_t layout,
                             int32_t dtype, int64_t compress_block_size, int64_t compress_stride,
                             int64_t page_block_size, void* output_cache, void* stream,
                             const cmp_nsa_dims* dims);

/* ---- the paged cache: filling it and attending over it -----------------------
 * cmp_qk_norm_rope, cmp_kv_append and cmp_paged_attention work on 16-bit tensors
 * (dtype CMP_NSA_FP16 or CMP_NSA_BF16) and on a pair of paged caches, k_cache and
 * v_cache [block_num, page_size, Hk, D]: the layout of cmp_nsa_compress's paged
 * input, so the cache that cmp_kv_append fills is one that cmp_nsa_compress
 * compresses (with pages of 64 or 128 rows). Position p of sequence b is row p % page_size of block
 * block_table[b][p / page_size]. Packed tokens: sequence b owns rows
 * cu_seqlens[b] .. cu_seqlens[b+1]-1 at positions start_pos[b], start_pos[b]+1, ...
 *
 * Tensors of tokens (q, k, v) have their last two dimensions dense and any token
 * stride that is a multiple of 8 elements (parts of one projection's output). All
 * 16-bit and float32 tensors start on 16-byte boundaries, int32 ones on 4-byte ones.
 *
 * cu_seqlens[B] may be below T: tokens behind the last sequence are skipped, their
 * rows of the caches, out and lse left as they were (batches padded to a captured
 * size). None of the three uses the library's per-stream workspace or allocates
 * memory, so they may be captured at any time and run on several streams at once.
 * What their kernels find wrong (cu_seqlens not rising from 0 or past T, a
 * negative start_pos, positions past INT32_MAX - 1 when appending and past
 * INT32_MAX - 1024 when attending, a needed table entry outside [0, block_num) or
 * past table_stride) never faults: the access is skipped and an error word of the
 * device is set, which cmp_get_error reports (on any stream of that device) and
 * clears. T == 0 is a successful no-op, with B == 0 too; tokens without any sequence
 * (B == 0, T > 0) are CMP_ERR_INVALID. */

/* The position rotation of the last `dim` channels of a head (cmp_compressor's
 * tables, one row per token):
 *   sin, cos  device [T, dim], float32 (CMP_ROPE_F32) or bf16 (CMP_ROPE_BF16)
 *   dim       a multiple of 16, at most D; 0: no rotation (sin, cos are not read)
 *   pairs     CMP_ROPE_INTERLEAVED: channels (2j, 2j+1) of the rotated part;
 *             CMP_ROPE_HALVES: channels (j, dim/2 + j). The pair (a, b) becomes
 *             (a cos[j] - b sin[j], b cos[dim/2+j] + a sin[dim/2+j]). */
enum { CMP_ROPE_INTERLEAVED = 0, CMP_ROPE_HALVES = 1 };
enum { CMP_ROPE_F32 = 0, CMP_ROPE_BF16 = 1 };
typedef struct cmp_rope {
  const void* sin;
  const void* cos;
  int32_t dim;
  int32_t pairs;
  int32_t dtype;
} cmp_rope;

typedef struct cmp_qk_dims {
  int64_t T;                      /* tokens */
  int64_t Hq, Hk;                 /* query heads 1..1024, key heads 0 (no keys)..1024 */
  int64_t D;                      /* channels per head, a multiple of 16, at most 256 */
  int64_t q_stride, k_stride;     /* elements from one token to the next */
  int64_t q_out_stride, k_out_stride;
} cmp_qk_dims;

/* Norms of queries and keys for each head with the position rotation in the same
 * pass: y = x / sqrt(mean(x^2) + eps) * weight over a head's D channels, then the
 * rotation; fp32 inside, one rounding to dtype. Heads whose squares leave fp32's
 * range (bf16 holds them) are normed in range.
 *   q, k            device [T, Hq, D], [T, Hk, D]; k, k_weight, k_out unused if Hk == 0
 *   q_weight, k_weight  device [D], dtype
 *   rope            host pointer, NULL: no rotation
 *   q_out, k_out    device, as q and k; may be q and k themselves (in place, equal
 *                   strides), must not overlap them otherwise
 * Returns CMP_OK, CMP_ERR_NULLPTR, CMP_ERR_INVALID, CMP_ERR_UNSUPPORTED (dtype,
 * rotation kind) or CMP_ERR_CUDA. */
CMP_API int cmp_qk_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight,
                             const cmp_rope* rope, float eps, int32_t dtype, void* q_out, void* k_out,
                             void* stream, const cmp_qk_dims* dims);

typedef struct cmp_kv_dims {
  int64_t B;                   /* sequences */
  int64_t T;                   /* tokens: rows of k and v */
  int64_t Hk;                  /* key heads, 1..256 */
  int64_t D;                   /* channels per head, a multiple of 16, at most 256 */
  int64_t k_stride, v_stride;  /* elements from one token to the next */
  int64_t block_num;           /* blocks of each cache; block_num * page_size <= INT32_MAX */
  int64_t page_size;           /* rows per block, 1..1024 (cmp_paged_attention reads pages that are
                                  multiples of 16 only) */
  int64_t table_stride;        /* columns of block_table */
} cmp_kv_dims;

/* Stores every token's keys (normed as in cmp_qk_norm_rope if norm_weight is not
 * NULL, rotated if rope says so) and values (unchanged) at its position of its
 * sequence's cache rows. No other row changes. Requirement that the library does
 * not check: two tokens of a call never map to one row (sequences that are
 * written do not share the blocks they are written to).
 *   k, v          device [T, Hk, D]
 *   norm_weight   device [D] or NULL
 *   block_table   device int32 [B, table_stride]; entries a call does not need are
 *                 not read
 *   cu_seqlens    device int32 [B+1];  start_pos  device int32 [B], NULL: all 0
 *   k_cache, v_cache  device [block_num, page_size, Hk, D], updated in place
 * Returns as cmp_qk_norm_rope does. */
CMP_API int cmp_kv_append(const void* k, const void* v, const void* norm_weight, const cmp_rope* rope, float eps,
                          const int32_t* block_table, const int32_t* cu_seqlens, const int32_t* start_pos,
                          int32_t dtype, void* k_cache, void* v_cache, void* stream, const cmp_kv_dims* dims);

typedef struct cmp_attn_dims {
  int64_t B;             /* sequences, at most 2^20 */
  int64_t T;             /* tokens: rows of q; T * Hq <= INT32_MAX */
  int64_t Hq, Hk;        /* query heads 1..1024, key heads 1..256; Hq = G * Hk with G <= 128 */
  int64_t D;             /* channels per head, a multiple of 16, at most 256 */
  int64_t q_stride;      /* elements from one token of q to the next */
  int64_t block_num;     /* blocks of each cache; block_num * page_size <= INT32_MAX */
  int64_t page_size;     /* rows per block: a multiple of 16, at most 1024 */
  int64_t table_stride;  /* columns of block_table */
  int64_t max_len;       /* no sequence of the call has more tokens (0: T) */
} cmp_attn_dims;

/* Attention of the call's tokens over their sequences' cached keys and values.
 * Query head h reads key head h / G. The token at position p (start_pos[b] + its
 * index) sees the first n(p) cache rows of its sequence,
 *   n(p) = 0 if p + 1 < key_block, else (p + 1 - key_block) / key_stride + 1,
 * of those the last `window` if window > 0:
 *   key_block = key_stride = 1: plain causal attention; the cache holds the chunk's
 *     own keys too (cmp_kv_append comes before);
 *   key_block = compress_block_size, key_stride = compress_stride: NSA's rows;
 *   key_block = key_stride = r: rows that each stand for r positions of their own.
 * (cmp_compressor's rows of C4A and C128A are not among them: they have 512 channels
 * and come packed, not paged.)
 *   out = sum_j softmax_j(scale q.k_j) v_j,  lse = ln sum_j exp(scale q.k_j)
 * A row that sees no key gets out = 0, lse = -inf. lse joins attentions over
 * different caches (raw and compressed rows, windows): the weights exp(lse_i - lse)
 * of their outs. Scores, statistics and sums are fp32; the weights are rounded to
 * dtype before the product with v, and out once at the end. Rounding out aside, an
 * output is off by at most about half a step of dtype of sum_j softmax_j |v_j|.
 *   q            device [T, Hq, D];  out  device [T, Hq, D], dense
 *   k_cache, v_cache  device [block_num, page_size, Hk, D]; rows that no token of
 *                the call sees may hold anything (NaN too). Inside one call a
 *                non-finite value may reach rows that do not see its key.
 *   block_table  device int32 [B, table_stride]; entries of rows that no token sees
 *                are not used (may be -1). Sequences may share blocks.
 *   cu_seqlens   device int32 [B+1];  start_pos  device int32 [B], NULL: all 0
 *   scale        finite, > 0
 *   window       keys, 0: no window;  key_block, key_stride  1..INT32_MAX
 *   lse          device float32 [T, Hq] or NULL
 *   workspace    device, workspace_bytes >= cmp_paged_attention_workspace(dims), 16-byte
 *                aligned; its contents need no preparation and mean nothing afterwards.
 *                Calls that may overlap need one each.
 * A sequence longer than max_len, whose cu_seqlens or start_pos entries are not
 * usable, or with positions past INT32_MAX - 1024 is skipped and reported (its rows
 * are left as they were); a missing table entry reads as zeros and is reported. Results do not depend on timing
 * (no floating-point atomics).
 * Returns CMP_OK, CMP_ERR_NULLPTR, CMP_ERR_INVALID, CMP_ERR_UNSUPPORTED (dtype) or
 * CMP_ERR_CUDA (launch, or the driver cannot describe the cache as a TMA tensor). */
CMP_API int cmp_paged_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                const int32_t* cu_seqlens, const int32_t* start_pos, float scale, int64_t window,
                                int64_t key_block, int64_t key_stride, int32_t dtype, void* out, float* lse,
                                void* workspace, size_t workspace_bytes, void* stream, const cmp_attn_dims* dims);

/* Bytes of workspace such a call needs on the current device (0: invalid dims).
 * Depends on D and on whether a sequence has at most 8, at most 16 or more rows per
 * key head (max_len, or T, times Hq / Hk). Host only. */
CMP_API size_t cmp_paged_attention_workspace(const cmp_attn_dims* dims);

/* ---- measurement --------------------------------------------------------
 * Kernels of the library, by id: */
enum {
  CMP_KERNEL_SCHED = 0,        /* varlen scheduler */
  CMP_KERNEL_PROJ_TC = 1,      /* prefill projection, tcgen05 / TMEM / TMA */
  CMP_KERNEL_PROJ_MMA = 2,     /* projection, warp-level mma.sync */
  CMP_KERNEL_PROJ_DECODE = 3,  /* small-T projection streaming the weights */
  CMP_KERNEL_POOL = 4,         /* pooling + RMSNorm + RoPE + Hadamard + store */
  CMP_KERNEL_FUSED = 5,        /* prefill projection with the pooling in its epilogue */
  CMP_KERNEL_FINISH = 6,       /* fused path: merge halves + RMSNorm + RoPE + Hadamard */
  CMP_KERNEL_DECODE_FUSED = 7, /* decode (T <= 64) in one cooperative kernel, K-split grid */
  CMP_KERNEL_DECODE_CP = 8,    /* decode (T <= 64) in one cooperative kernel of 4-CTA clusters
                                  that each own 16 channels */
  CMP_KERNEL_NSA = 9,          /* NsaCompressWithCache */
  CMP_KERNEL_NSA_SCAN = 10,    /* NsaCompressWithCache, packed layout: each batch's first row */
  CMP_KERNEL_QK_NORM_ROPE = 11,
  CMP_KERNEL_KV_APPEND = 12,
  CMP_KERNEL_ATTN_DECODE = 13,  /* paged attention, at most 16 rows per key head and sequence */
  CMP_KERNEL_ATTN_COMBINE = 14, /* paged attention: joins rows that were cut between CTAs */
  CMP_KERNEL_ATTN_CHUNK = 15,   /* paged attention, many rows per key head */
  CMP_KERNEL_COUNT = 16
};

/* Name of a kernel id (NULL if out of range). */
CMP_API const char* cmp_kernel_name(int kernel);

/* Total kernels this library has launched in this process (all devices). */
CMP_API int64_t cmp_launch_count(void);

/* Start per-kernel timing: every launch from now on is bracketed by CUDA
 * events on its stream. Clears earlier totals. Returns CMP_OK or CMP_ERR_CUDA. */
CMP_API int cmp_profile_start(void);

/* Stop timing; synchronise the recorded events and write, per kernel id, the
 * summed milliseconds and launch count into ms[CMP_KERNEL_COUNT] and
 * launches[CMP_KERNEL_COUNT] (host arrays; either may be NULL). */
CMP_API int cmp_profile_stop(double* ms, int64_t* launches);

/* Measurement hook of a library built with -DCMP_PHASE_STAMPS (bench.py
 * --only decode-phases builds one beside the normal library and runs it): the
 * channel-group decode kernel writes the global timer (ns) at up to 32 points
 * of its timeline; this copies those of its last launch, CTA i's phase k at
 * dst[i * 32 + k] for the first n entries (host array, n <= 512 * 32), after
 * synchronising the device. Phases: 0 entry, 1 set-up done, 2 first weight
 * stage landed, 3 last MMA issued, 4 metadata done, 5 partials sent,
 * 6 partials received, 7 pooled and arrived, 9 exchange complete, 10 rows
 * stored, 11 all CTAs arrived, 14 tails written, 15 end; 16-19 the metadata's
 * first wave, window list, second and third wave. Other builds return
 * CMP_ERR_UNSUPPORTED. */
CMP_API int cmp_debug_phase_stamps(uint64_t* dst, int64_t n);

/* Testing knob: which path calls take. 0 = automatic (for T <= 64 the
 * channel-group decode kernel, or without it (rotate, or a device that cannot
 * hold its clusters) the weight-streaming projection + pooling kernels, else
 * the K-split one-kernel decode; the fused tcgen05 pooling kernel for long
 * sequences, T >= 1024 and T >= 256*B, when its (T/256)*(C/128) work items
 * fill the SMs twice; else the tcgen05 projection + pooling kernel), 1 = force the mma.sync projection, 2 = the tcgen05 projection
 * (on CTA pairs, cta_group::2, where the device can co-schedule them),
 * 3 = weight streaming, 4 = the fused path, 5 = the K-split one-kernel decode,
 * 6 = the channel-group decode, 7 = the tcgen05 projection on single CTAs,
 * 8 = the fused path on single CTAs (4 runs on CTA pairs, cta_group::2, when
 * coff * D / 128 is even and the device co-schedules them).
 * A forced path a call cannot take falls back to 1.
 * Returns the previous value, or -1 if out of range. */
CMP_API int cmp_set_proj_kernel(int which);

/* Testing knob for failure detection: the next `launches` launches of the
 * channel-group decode kernel (CMP_KERNEL_DECODE_CP) wait for the other
 * clusters' exchange words of an epoch that no cluster publishes. Each CTA's
 * bounded wait gives up after about one second, the rows of the call come out
 * as zeros, the CTAs free their tensor memory and return, and cmp_get_error
 * then reports CMP_ERR_TIMEOUT and resets the exchange words, so the next call
 * runs normally. A cmp_paged_attention call that decodes counts as such a launch
 * too: no key tile is loaded for it, its CTAs' waits give up after two seconds,
 * its rows come out as zeros (those that span several CTAs too, lse -inf) and
 * cmp_get_error reports CMP_ERR_TIMEOUT. Nothing faults or hangs. Returns the
 * previous count, or -1 if launches < 0. */
CMP_API int cmp_debug_unreachable_barrier(int launches);

#ifdef __cplusplus
}
#endif

#endif /* CMP_H_ */
