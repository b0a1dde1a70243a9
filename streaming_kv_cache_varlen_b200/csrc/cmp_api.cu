// Host side of the C ABI: argument checks, the per-(device, stream) workspace,
// kernel launches, error reporting and per-kernel timing.
#include <algorithm>
#include <atomic>
#include <climits>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

#include <cmath>

#include "cmp_attn.cuh"
#include "cmp_internal.cuh"

namespace cmp {
cudaError_t launch_qk_norm_rope(const QkNormParams& p, cudaStream_t s, int sms);
cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t s, int sms);
cudaError_t kv_error_word(unsigned** word);
cudaError_t launch_proj_tc(const Params& p, cudaStream_t s);
cudaError_t launch_proj_decode(const Params& p, cudaStream_t s);
bool proj_tc_supported(const Params& p);
bool proj_decode_supported(const Params& p);
size_t proj_decode_workspace(const Params& p);
bool decode_fused_supported(const Params& p);
size_t decode_fused_workspace(const Params& p);
cudaError_t launch_decode_fused(const Params& p, float* part, void* bar, cudaStream_t s);
bool decode_cp_supported(const Params& p);
cudaError_t launch_decode_cp(const Params& p, void* counter, void* xch, void* u, cudaStream_t s,
                             bool unreachable);
cudaError_t launch_nsa(const NsaParams& p, cudaStream_t s, int sm_count);
cudaError_t launch_nsa_scan(const NsaParams& p, cudaStream_t s);
int noalloc_take_error(int dev, unsigned* word);
void noalloc_forget_addresses();
}  // namespace cmp

namespace {

using cmp::Params;

// ---- workspace ---------------------------------------------------------------

// The first kHeaderBytes (zeroed when the workspace is created, and after a
// timeout) hold the error word at offset 0, the K-split decode kernel's
// grid-barrier words at offset 64, the channel-group decode kernel's arrival
// counter at offset 256, its CTAs' sums (64 windows x 128 CTAs x 4 bytes) from
// offset 4096 and, for the rotation, every channel's u (64 windows x 512 x 4
// bytes) after them, then the one-kernel fused path's per-tile arrival
// counters (which that kernel puts back to zero); only those kernels write
// there.
constexpr size_t kGridBarOffset = 64;
constexpr size_t kCounterOffset = 256;
constexpr size_t kExchangeOffset = 4096;
constexpr size_t kRotateOffset = kExchangeOffset + 64 * 128 * 4;
constexpr size_t kTileCntOffset = kRotateOffset + 64 * 512 * 4;
constexpr size_t kHeaderBytes = kTileCntOffset + cmp::kFusedTileCounters * 4;

size_t zeroed_bytes() { return kHeaderBytes; }

struct WsLayout {
  size_t err, m_cu, m_s, m_off, m_tile, had, proj, ystat, ylse, part, total;
};

// fused: the pooled-halves buffers of the fused path instead of the fp32
// projection rows of the other paths.
WsLayout ws_layout(int64_t B, int64_t T, int64_t C, int64_t n_out, bool fused, size_t part_bytes) {
  WsLayout L{};
  size_t o = 0;
  auto take = [&](size_t n) {
    const size_t r = o;
    o += (n + 255) & ~size_t(255);
    return r;
  };
  L.err = take(zeroed_bytes());
  L.m_cu = take(sizeof(int32_t) * (B + 1));
  L.m_s = take(sizeof(int32_t) * std::max<int64_t>(B, 1));
  L.m_off = take(sizeof(int32_t) * (B + 1));
  L.m_tile = take(fused ? sizeof(int32_t) * (B + 1) : 0);
  L.had = take(sizeof(int32_t) * 16);  // the scheduler's verdicts on the hadamard matrix (<= 4 chunks)
  L.proj = take(fused ? 0 : sizeof(float) * (size_t)T * 2 * C);
  L.ystat = take(fused ? sizeof(float) * (size_t)std::max<int64_t>(n_out, 1) * C : 0);
  L.ylse = take(fused ? sizeof(float) * (size_t)std::max<int64_t>(n_out, 1) * C : 0);
  L.part = take(part_bytes);
  L.total = o;
  return L;
}

// Which projection path a call takes: 1 mma.sync, 2 tcgen05 (+ pooling kernel),
// 3 small-T weight streaming (+ pooling kernel), 4 fused tcgen05 pooling
// (+ finish kernel), 5 decode in one cooperative kernel (K-split grid),
// 6 decode in one cooperative kernel of channel-group clusters.
int sm_count_cached();

// The fused prefill's work items (256-position tiles x 128-channel blocks),
// estimated from the token count (the lengths are on the device).
int64_t fused_items_estimate(const Params& p) { return ((int64_t)p.T / 256) * (p.C / 128); }

int choose_path(const Params& p, int forced) {
  int which = forced;
  if (which == 0) {
    // small T: the channel-group kernel; else weight streaming, which measured
    // as fast or faster than the K-split kernel on the decode shapes (much
    // faster when each K slice would be one or two 64-column steps)
    if (cmp::decode_cp_supported(p)) which = 6;
    else if (cmp::proj_decode_supported(p)) which = 3;
    else if (cmp::decode_fused_supported(p)) which = 5;
    // the fused kernel when its items fill the SMs at least twice (narrow state
    // rows over ~10K tokens leave it half the GPU: the separate projection, with
    // twice the items, measured 17 % faster there)
    else if (cmp::fused_supported(p) && p.T >= 1024 && (int64_t)p.T >= 256LL * p.B &&
             (fused_items_estimate(p) >= 2LL * sm_count_cached() || !cmp::proj_tc_supported(p)))
      which = 4;
    else if (cmp::proj_tc_supported(p)) which = 2;
    else which = 1;
  }
  if (which == 2 && !cmp::proj_tc_supported(p)) which = 1;
  if (which == 3 && !cmp::proj_decode_supported(p)) which = 1;
  if (which == 4 && !cmp::fused_supported(p)) which = 1;
  if (which == 5 && !cmp::decode_fused_supported(p)) which = 1;
  if (which == 6 && !cmp::decode_cp_supported(p)) which = 1;
  return which;
}

int sm_count_cached() {
  static int counts[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && counts[dev]) return counts[dev];
  int n = 148;
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (dev < 64) counts[dev] = n;
  return n;
}

struct Workspace {
  unsigned char* ptr = nullptr;
  size_t bytes = 0;
};

std::mutex g_mu;
std::map<std::pair<int, cudaStream_t>, Workspace> g_ws;
std::map<std::pair<int, cudaStream_t>, unsigned> g_pending_err;  // kept across a regrow
std::atomic<int64_t> g_launches{0};
std::atomic<int> g_proj_kernel{0};
std::atomic<int> g_unreachable_barrier{0};  // launches left whose waits cannot be met

// The timeout tests' knob, consumed one launch at a time.
bool take_unreachable() {
  bool taken = false;
  for (int v = g_unreachable_barrier.load(); v > 0 && !taken;)
    taken = g_unreachable_barrier.compare_exchange_weak(v, v - 1);
  return taken;
}

// ---- profiling ---------------------------------------------------------------

struct Timed {
  cudaEvent_t a, b;
  int kernel;
};
std::mutex g_prof_mu;
bool g_prof = false;
std::vector<Timed> g_timed;
std::vector<cudaEvent_t> g_event_pool;

cudaEvent_t take_event() {
  if (!g_event_pool.empty()) {
    cudaEvent_t e = g_event_pool.back();
    g_event_pool.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
  return e;
}

template <class F>
cudaError_t launch(int kernel, cudaStream_t s, F&& f) {
  Timed t{nullptr, nullptr, kernel};
  bool prof = false;
  {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    if (g_prof) {
      t.a = take_event();
      t.b = take_event();
      prof = t.a && t.b;
    }
  }
  if (prof) cudaEventRecord(t.a, s);
  const cudaError_t e = f();
  if (prof) {
    cudaEventRecord(t.b, s);
    std::lock_guard<std::mutex> lk(g_prof_mu);
    if (e == cudaSuccess) {
      g_timed.push_back(t);
    } else {  // nothing ran: no timing record
      g_event_pool.push_back(t.a);
      g_event_pool.push_back(t.b);
    }
  }
  if (e == cudaSuccess) g_launches.fetch_add(1, std::memory_order_relaxed);
  return e;
}

int get_workspace(cudaStream_t s, size_t need, unsigned char** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return CMP_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  Workspace& w = g_ws[{dev, s}];
  if (w.bytes >= need && w.ptr) {
    *out = w.ptr;
    return CMP_OK;
  }
  if (w.ptr) {
    // keep an error word a pending call may still set: wait, read, carry over
    if (cudaDeviceSynchronize() != cudaSuccess) return CMP_ERR_CUDA;
    unsigned old = 0;
    if (cudaMemcpy(&old, w.ptr, sizeof(old), cudaMemcpyDeviceToHost) != cudaSuccess) return CMP_ERR_CUDA;
    g_pending_err[{dev, s}] |= old;
    cudaFree(w.ptr);
    w.ptr = nullptr;
    w.bytes = 0;
  }
  const size_t bytes = std::max(need, size_t(1) << 20);
  void* p = nullptr;
  if (cudaMalloc(&p, bytes) != cudaSuccess) return CMP_ERR_CUDA;
  if (cudaMemset(p, 0, zeroed_bytes()) != cudaSuccess) {
    cudaFree(p);
    return CMP_ERR_CUDA;
  }
  w.ptr = static_cast<unsigned char*>(p);
  w.bytes = bytes;
  *out = w.ptr;
  return CMP_OK;
}

// Extra workspace of the one-kernel decode paths.
size_t decode_part_bytes(const Params& p, int which) {
  if (which == 5) return cmp::decode_fused_workspace(p);
  return 0;
}

bool valid_ratio(int r) {
  return r == 1 || r == 2 || r == 4 || r == 8 || r == 16 || r == 32 || r == 64 || r == 128;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_dims(const cmp_dims* d) {
  if (!d) return CMP_ERR_NULLPTR;
  if (d->B < 0 || d->T < 0) return CMP_ERR_INVALID;
  if (d->D != 128 && d->D != 512) return CMP_ERR_INVALID;
  if (d->H < 512 || d->H > 16384 || d->H % 512) return CMP_ERR_INVALID;
  if (d->block_size < 1 || d->block_size > 1024) return CMP_ERR_INVALID;
  if (d->block_num < 1 || d->table_stride < 1) return CMP_ERR_INVALID;
  return CMP_OK;
}

// ---- paged cache operators -----------------------------------------------------

// Devices on which an operator with a device-wide error word has run.
std::atomic<uint64_t> g_word_devices{0};

void note_word_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64)
    g_word_devices.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
}

// The words are shared by all streams of the device, so a kernel of another stream may
// set bits at any time: each is read and cleared in one step.
__device__ unsigned g_taken;
__global__ void take_words_kernel(unsigned* kv, unsigned* decode, unsigned* chunk) {
  g_taken = atomicExch(kv, 0u) | atomicExch(decode, 0u) | atomicExch(chunk, 0u);
}

// The current device's words, read and cleared, by way of stream s if it is that device's.
cudaError_t take_device_words(cudaStream_t s, unsigned* word) {
  static std::mutex mu;  // g_taken belongs to one call until it is read
  std::lock_guard<std::mutex> lk(mu);
  unsigned *kv, *decode, *chunk;
  cudaError_t e = cmp::kv_error_word(&kv);
  if (e == cudaSuccess) e = cmp::attn_decode_error_word(&decode);
  if (e == cudaSuccess) e = cmp::attn_chunk_error_word(&chunk);
  int here = 0, of_s = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&here);
  if (e == cudaSuccess) e = cudaStreamGetDevice(s, &of_s);
  if (e != cudaSuccess) return e;
  if (of_s != here) s = cudaStreamPerThread;
  take_words_kernel<<<1, 1, 0, s>>>(kv, decode, chunk);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(word, g_taken, sizeof(*word), 0, cudaMemcpyDeviceToHost, s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
bool valid_head_dim(int64_t D) { return in(D, 16, 256) && D % 16 == 0; }
bool valid_dtype(int32_t t) { return t == CMP_NSA_FP16 || t == CMP_NSA_BF16; }
// tokens of `heads` dense heads, `stride` elements apart
bool valid_stride(int64_t stride, int64_t heads, int64_t D) {
  return stride % 8 == 0 && in(stride, heads * D, int64_t(1) << 40);
}

int check_rope(const cmp_rope* r, int64_t D, cmp::RopeTable* o) {
  *o = cmp::RopeTable{};
  if (!r || r->dim == 0) return CMP_OK;
  if (!in(r->dim, 16, D) || r->dim % 16) return CMP_ERR_INVALID;
  if ((r->pairs != CMP_ROPE_INTERLEAVED && r->pairs != CMP_ROPE_HALVES) ||
      (r->dtype != CMP_ROPE_F32 && r->dtype != CMP_ROPE_BF16))
    return CMP_ERR_UNSUPPORTED;
  if (!r->sin || !r->cos) return CMP_ERR_NULLPTR;
  if (!aligned(r->sin, 16) || !aligned(r->cos, 16)) return CMP_ERR_INVALID;
  o->sin = r->sin;
  o->cos = r->cos;
  o->dim = r->dim;
  o->f32 = r->dtype == CMP_ROPE_F32;
  o->halves = r->pairs == CMP_ROPE_HALVES;
  return CMP_OK;
}

int check_attn_dims(const cmp_attn_dims* d) {
  if (!d) return CMP_ERR_NULLPTR;
  if (!in(d->B, 0, cmp::kMaxSequences) || !in(d->T, 0, INT32_MAX - 1) || !in(d->Hq, 1, 1024) || !in(d->Hk, 1, 256) ||
      d->Hq % d->Hk || d->Hq / d->Hk > 128 || !valid_head_dim(d->D) || d->T * d->Hq > INT32_MAX ||
      !valid_stride(d->q_stride, d->Hq, d->D) || !in(d->page_size, 16, 1024) || d->page_size % 16 ||
      !in(d->block_num, 1, INT32_MAX / d->page_size) || !in(d->table_stride, 1, INT32_MAX) ||
      !in(d->max_len, 0, INT32_MAX) || (d->B == 0 && d->T != 0))
    return CMP_ERR_INVALID;
  return CMP_OK;
}

// How a call of paged attention runs, from its host-known sizes.
struct AttnPath {
  bool chunk;   // 128-row MMA tiles
  int m, ctas;  // rows per item; CTAs
  int key_tile;
  size_t part, ml, desc, total;
};

AttnPath attn_path(const cmp_attn_dims& d) {
  AttnPath a{};
  const int64_t len = d.max_len && d.max_len < d.T ? d.max_len : d.T;
  const int64_t rows = len * (d.Hq / d.Hk);
  a.chunk = rows > cmp::kAttnDecodeRows;
  a.m = a.chunk ? cmp::attn_chunk_rows((int)d.D) : cmp::attn_decode_rows(rows);
  a.ctas = a.chunk ? sm_count_cached() : cmp::attn_decode_ctas((int)d.D, sm_count_cached());
  a.key_tile = a.chunk ? cmp::attn_chunk_key_tile((int)d.D) : 64;
  const size_t slots = (size_t)a.ctas * 2 * a.m;
  a.part = 0;
  a.ml = a.part + slots * cmp::attn_padded((int)d.D) * sizeof(float);
  a.desc = a.ml + slots * 2 * sizeof(float);
  a.total = a.desc + (size_t)a.ctas * 2 * sizeof(int4);
  return a;
}

// Returned by run_path when the device refused a launch form before anything
// ran (the path is then disabled on that device): the caller picks again.
constexpr int kRetryOtherPath = -1000;

// Workspace and launches of one call on path `which`.
int run_path(Params& p, int which, cudaStream_t s) {
  int rc;
  const bool fused = which == 4;
  const WsLayout L = ws_layout(p.B, p.T, p.C, p.n_out, fused, decode_part_bytes(p, which));
  const size_t extra = cmp::proj_decode_workspace(p);
  unsigned char* ws = nullptr;
  rc = get_workspace(s, L.total + extra, &ws);
  if (rc != CMP_OK) return rc;
  p.err = reinterpret_cast<unsigned*>(ws + L.err);
  p.m_cu = reinterpret_cast<int32_t*>(ws + L.m_cu);
  p.m_s = reinterpret_cast<int32_t*>(ws + L.m_s);
  p.m_off = reinterpret_cast<int32_t*>(ws + L.m_off);
  p.m_tile = fused ? reinterpret_cast<int32_t*>(ws + L.m_tile) : nullptr;
  // paths with the scheduler kernel check the hadamard matrix there (the pooling
  // kernels then use the fast transform for a scaled Sylvester matrix)
  p.had_sylv = (p.rotate && which != 5 && which != 6) ? reinterpret_cast<int32_t*>(ws + L.had) : nullptr;
  p.proj = fused ? nullptr : reinterpret_cast<float*>(ws + L.proj);
  p.ystat = fused ? reinterpret_cast<float*>(ws + L.ystat) : nullptr;
  p.ylse = fused ? reinterpret_cast<float*>(ws + L.ylse) : nullptr;

  // ---- kernels ----
  if (which == 6) {  // decode: one cooperative kernel of clusters, no scheduler launch
    void* counter = ws + L.err + kCounterOffset;
    void* xch = ws + L.err + kExchangeOffset;
    void* urow = ws + L.err + kRotateOffset;
    const bool unreachable = take_unreachable();
    const cudaError_t e = launch(CMP_KERNEL_DECODE_CP, s,
                                 [&] { return cmp::launch_decode_cp(p, counter, xch, urow, s, unreachable); });
    if (e == cudaErrorNotSupported) return kRetryOtherPath;
    return e == cudaSuccess ? CMP_OK : CMP_ERR_CUDA;
  }
  if (which == 5) {  // decode: one cooperative kernel, no scheduler launch
    float* part = reinterpret_cast<float*>(ws + L.part);
    void* bar = ws + L.err + kGridBarOffset;
    if (launch(CMP_KERNEL_DECODE_FUSED, s, [&] { return cmp::launch_decode_fused(p, part, bar, s); }) !=
        cudaSuccess)
      return CMP_ERR_CUDA;
    return CMP_OK;
  }
  cudaError_t e;
  if (fused && cmp::fused_fold_supported(p)) {  // one kernel: metadata and row finish inside
    p.tile_cnt = reinterpret_cast<unsigned*>(ws + L.err + kTileCntOffset);
    const int sms = sm_count_cached();
    e = launch(CMP_KERNEL_FUSED, s, [&] { return cmp::launch_fused(p, s, sms); });
    return e == cudaSuccess ? CMP_OK : CMP_ERR_CUDA;
  }
  if (launch(CMP_KERNEL_SCHED, s, [&] { return cmp::launch_sched(p, s); }) != cudaSuccess)
    return CMP_ERR_CUDA;
  if (fused) {
    const int sms = sm_count_cached();
    e = launch(CMP_KERNEL_FUSED, s, [&] { return cmp::launch_fused(p, s, sms); });
    if (e != cudaSuccess) return CMP_ERR_CUDA;
    if (launch(CMP_KERNEL_FINISH, s, [&] { return cmp::launch_finish(p, s); }) != cudaSuccess)
      return CMP_ERR_CUDA;
    return CMP_OK;
  }
  if (which == 2)
    e = launch(CMP_KERNEL_PROJ_TC, s, [&] { return cmp::launch_proj_tc(p, s); });
  else if (which == 3)
    e = launch(CMP_KERNEL_PROJ_DECODE, s, [&] { return cmp::launch_proj_decode(p, s); });
  else
    e = launch(CMP_KERNEL_PROJ_MMA, s, [&] { return cmp::launch_proj_mma(p, s); });
  if (e != cudaSuccess) return CMP_ERR_CUDA;
  if (launch(CMP_KERNEL_POOL, s, [&] { return cmp::launch_pool(p, s); }) != cudaSuccess)
    return CMP_ERR_CUDA;
  return CMP_OK;
}

}  // namespace

extern "C" {

int64_t cmp_out_rows(int64_t B, int64_t T, int32_t ratio) {
  if (ratio < 1 || B < 0 || T < 0) return -1;
  return std::min<int64_t>(T, T / ratio + B);
}

int cmp_out_row_layout(const int32_t* cu_seqlens, const int32_t* start_pos, int32_t B, int32_t ratio,
                       int64_t n_out, int32_t* row_seq, int32_t* row_window) {
  if (!cu_seqlens || ((!row_seq || !row_window) && n_out > 0)) return CMP_ERR_NULLPTR;
  if (B < 0 || ratio < 1) return CMP_ERR_INVALID;
  if (cu_seqlens[0] != 0) return CMP_ERR_INVALID;
  for (int b = 0; b < B; ++b) {
    if (cu_seqlens[b + 1] < cu_seqlens[b]) return CMP_ERR_INVALID;
    const int64_t s = start_pos ? start_pos[b] : 0;
    if (s < 0 || s + (cu_seqlens[b + 1] - cu_seqlens[b]) > INT32_MAX) return CMP_ERR_INVALID;
  }
  if (n_out != cmp_out_rows(B, cu_seqlens[B], ratio)) return CMP_ERR_INVALID;
  for (int64_t n = 0; n < n_out; ++n) row_seq[n] = row_window[n] = -1;
  int64_t off = 0;
  for (int b = 0; b < B; ++b) {
    const int64_t L = cu_seqlens[b + 1] - cu_seqlens[b];
    const int64_t s = start_pos ? start_pos[b] : 0;
    const int64_t e = s + L;
    const int64_t nw = e / ratio - s / ratio;
    for (int64_t k = 0; k < nw; ++k) {
      row_seq[off + k] = b;
      row_window[off + k] = (int32_t)(s / ratio + k);
    }
    off += std::min<int64_t>(L, L / ratio + 1);
  }
  return CMP_OK;
}

size_t cmp_workspace_size(const cmp_dims* dims, int32_t ratio) {
  if (check_dims(dims) != CMP_OK || !valid_ratio(ratio)) return 0;
  const int coff = ratio == 4 ? 2 : 1;
  Params p{};
  p.B = dims->B;
  p.T = dims->T;
  p.H = dims->H;
  p.D = dims->D;
  p.C = coff * dims->D;
  p.coff = coff;
  p.ratio = ratio;
  p.n_out = (int)cmp_out_rows(p.B, p.T, ratio);
  const int knob = g_proj_kernel.load();
  const int which = choose_path(p, knob == 7 ? 2 : knob == 8 ? 4 : knob);
  return ws_layout(dims->B, dims->T, p.C, p.n_out, which == 4, decode_part_bytes(p, which)).total +
         cmp::proj_decode_workspace(p);
}

int cmp_release_workspaces(void) {
  std::lock_guard<std::mutex> lk(g_mu);
  int rc = CMP_OK;
  int cur = 0;
  cudaGetDevice(&cur);
  for (auto& kv : g_ws) {
    if (!kv.second.ptr) continue;
    if (cudaSetDevice(kv.first.first) != cudaSuccess) { rc = CMP_ERR_CUDA; continue; }
    cudaDeviceSynchronize();
    if (cudaFree(kv.second.ptr) != cudaSuccess) rc = CMP_ERR_CUDA;
  }
  g_ws.clear();
  cudaSetDevice(cur);
  cmp::noalloc_forget_addresses();  // looked up again by the next allocation-free call
  return rc;
}

int cmp_compressor(const cmp_bf16* x, float* kv_state, float* score_state,
                   const int32_t* kv_block_table, const int32_t* state_block_table,
                   const cmp_bf16* sin, const cmp_bf16* cos, const cmp_bf16* wkv,
                   const cmp_bf16* wgate, const float* ape, const cmp_bf16* norm_weight,
                   const cmp_bf16* hadamard, const int32_t* start_pos, const int32_t* cu_seqlens,
                   int32_t ratio, int32_t rope_head_dim, bool rotate, cmp_bf16* out,
                   void* stream, const cmp_dims* dims) {
  // ---- host checks, nothing launched before they pass ----
  if (!dims) return CMP_ERR_NULLPTR;
  if (!valid_ratio(ratio)) return CMP_ERR_UNSUPPORTED;
  int rc = check_dims(dims);
  if (rc != CMP_OK) return rc;
  if (rope_head_dim != 64 || rope_head_dim > dims->D) return CMP_ERR_INVALID;
  if (dims->B == 0 && dims->T != 0) return CMP_ERR_INVALID;
  if (dims->B == 0 || dims->T == 0) return CMP_OK;
  if (!x || !kv_state || !score_state || !kv_block_table || !state_block_table || !sin || !cos ||
      !wkv || !wgate || !ape || !norm_weight || !cu_seqlens || !out)
    return CMP_ERR_NULLPTR;
  if (rotate && !hadamard) return CMP_ERR_NULLPTR;
  if (!aligned(x, 16) || !aligned(wkv, 16) || !aligned(wgate, 16) || !aligned(kv_state, 16) ||
      !aligned(score_state, 16) || !aligned(ape, 16) || !aligned(out, 8) || !aligned(norm_weight, 8) ||
      !aligned(sin, 4) || !aligned(cos, 4) || (rotate && !aligned(hadamard, 8)) ||
      !aligned(kv_block_table, 4) || !aligned(state_block_table, 4) || !aligned(cu_seqlens, 4) ||
      (start_pos && !aligned(start_pos, 4)))
    return CMP_ERR_INVALID;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int coff = ratio == 4 ? 2 : 1;
  Params p{};
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.kv_state = kv_state;
  p.score_state = score_state;
  p.kv_tbl = kv_block_table;
  p.sc_tbl = state_block_table;
  p.sin = reinterpret_cast<const __nv_bfloat16*>(sin);
  p.cos = reinterpret_cast<const __nv_bfloat16*>(cos);
  p.wkv = reinterpret_cast<const __nv_bfloat16*>(wkv);
  p.wgate = reinterpret_cast<const __nv_bfloat16*>(wgate);
  p.ape = ape;
  p.norm_w = reinterpret_cast<const __nv_bfloat16*>(norm_weight);
  p.had = rotate ? reinterpret_cast<const __nv_bfloat16*>(hadamard) : nullptr;
  p.start_pos = start_pos;
  p.cu_in = cu_seqlens;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.B = dims->B;
  p.T = dims->T;
  p.H = dims->H;
  p.D = dims->D;
  p.C = coff * dims->D;
  p.coff = coff;
  p.ratio = ratio;
  p.rope = rope_head_dim;
  p.rotate = rotate ? 1 : 0;
  p.block_num = dims->block_num;
  p.bs = dims->block_size;
  p.stride = dims->table_stride;
  p.n_out = (int)cmp_out_rows(p.B, p.T, ratio);

  for (int attempt = 0; attempt < 2; ++attempt) {
    const int knob = g_proj_kernel.load();
    p.single_cta = (knob == 7 || knob == 8) ? 1 : 0;
    const int r2 = run_path(p, choose_path(p, knob == 7 ? 2 : knob == 8 ? 4 : knob), s);
    // the device refused the channel-group decode's launch form (nothing ran):
    // the path is now disabled there and the next choice is taken
    if (r2 != kRetryOtherPath) return r2;
  }
  return CMP_ERR_CUDA;
}


int cmp_nsa_compress(const void* input, const void* weight, const int32_t* slot_mapping,
                     const int64_t* act_seq_len, const int32_t* block_table, int32_t layout, int32_t dtype,
                     int64_t compress_block_size, int64_t compress_stride, int64_t page_block_size,
                     void* output_cache, void* stream, const cmp_nsa_dims* dims) {
  if (!dims) return CMP_ERR_NULLPTR;
  if (dtype != CMP_NSA_FP16 && dtype != CMP_NSA_BF16) return CMP_ERR_UNSUPPORTED;
  if (layout != CMP_NSA_PAGED && layout != CMP_NSA_PACKED) return CMP_ERR_UNSUPPORTED;
  const cmp_nsa_dims& d = *dims;
  const int64_t cbs = compress_block_size, st = compress_stride;
  const bool paged = layout == CMP_NSA_PAGED;
  if (d.B < 0 || d.N < 1 || d.N > 64 || (d.N > 50 && d.N % 2) || d.D < 16 || d.D > 256 || d.D % 16 ||
      d.result_len < 1 || d.tokens < 1 || cbs < 16 || cbs > 64 || cbs % 16 ||
      (st != 16 && st != 32 && st != 48 && st != 64) || cbs < st ||
      (paged && (page_block_size != 64 && page_block_size != 128)) || (paged && d.table_stride < 1) ||
      d.B > 65535 || d.tokens > (paged ? INT32_MAX / page_block_size : INT32_MAX))
    return CMP_ERR_INVALID;
  if (d.B == 0) return CMP_OK;
  if (!input || !weight || !slot_mapping || !act_seq_len || !output_cache || (paged && !block_table))
    return CMP_ERR_NULLPTR;
  if (!aligned(input, 16) || !aligned(output_cache, 16) || !aligned(weight, 2) || !aligned(slot_mapping, 4) ||
      !aligned(act_seq_len, 8) || (paged && !aligned(block_table, 4)))
    return CMP_ERR_INVALID;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned char* ws = nullptr;
  // packed: the batches' first rows follow the zeroed header
  const int rc = get_workspace(s, zeroed_bytes() + (paged ? 0 : (size_t)d.B * 8), &ws);
  if (rc != CMP_OK) return rc;
  cmp::NsaParams p{};
  p.starts = paged ? nullptr : reinterpret_cast<int64_t*>(ws + zeroed_bytes());
  p.input = static_cast<const uint16_t*>(input);
  p.weight = static_cast<const uint16_t*>(weight);
  p.slot = slot_mapping;
  p.len = act_seq_len;
  p.table = block_table;
  p.out = static_cast<uint16_t*>(output_cache);
  p.err = reinterpret_cast<unsigned*>(ws);
  p.B = (int)d.B;
  p.N = (int)d.N;
  p.D = (int)d.D;
  p.cbs = (int)cbs;
  p.stride = (int)st;
  p.pbs = paged ? (int)page_block_size : 1;
  p.packed = paged ? 0 : 1;
  p.bf16 = dtype == CMP_NSA_BF16 ? 1 : 0;
  p.tokens = d.tokens;
  p.table_stride = paged ? d.table_stride : 1;
  p.result_len = d.result_len;
  if (!paged && launch(CMP_KERNEL_NSA_SCAN, s, [&] { return cmp::launch_nsa_scan(p, s); }) != cudaSuccess)
    return CMP_ERR_CUDA;
  if (launch(CMP_KERNEL_NSA, s, [&] { return cmp::launch_nsa(p, s, sm_count_cached()); }) != cudaSuccess)
    return CMP_ERR_CUDA;
  return CMP_OK;
}

int cmp_qk_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight, const cmp_rope* rope,
                     float eps, int32_t dtype, void* q_out, void* k_out, void* stream, const cmp_qk_dims* dims) {
  if (!dims) return CMP_ERR_NULLPTR;
  if (!valid_dtype(dtype)) return CMP_ERR_UNSUPPORTED;
  const cmp_qk_dims& d = *dims;
  const bool keys = d.Hk > 0;
  if (!in(d.T, 0, INT32_MAX - 1) || !in(d.Hq, 1, 1024) || !in(d.Hk, 0, 1024) || !valid_head_dim(d.D) ||
      !valid_stride(d.q_stride, d.Hq, d.D) || !valid_stride(d.q_out_stride, d.Hq, d.D) ||
      (keys && (!valid_stride(d.k_stride, d.Hk, d.D) || !valid_stride(d.k_out_stride, d.Hk, d.D))) ||
      !(eps >= 0.f) || std::isinf(eps))
    return CMP_ERR_INVALID;
  if (d.T == 0) return CMP_OK;
  cmp::QkNormParams p{};
  const int rc = check_rope(rope, d.D, &p.rope);
  if (rc != CMP_OK) return rc;
  if (!q || !q_weight || !q_out || (keys && (!k || !k_weight || !k_out))) return CMP_ERR_NULLPTR;
  if (!aligned(q, 16) || !aligned(q_weight, 16) || !aligned(q_out, 16) ||
      (keys && (!aligned(k, 16) || !aligned(k_weight, 16) || !aligned(k_out, 16))) ||
      (q == q_out && d.q_stride != d.q_out_stride) || (keys && k == k_out && d.k_stride != d.k_out_stride))
    return CMP_ERR_INVALID;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.q_weight = static_cast<const uint16_t*>(q_weight);
  p.k_weight = static_cast<const uint16_t*>(k_weight);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.T = d.T;
  p.q_stride = d.q_stride;
  p.k_stride = d.k_stride;
  p.qo_stride = d.q_out_stride;
  p.ko_stride = d.k_out_stride;
  p.Hq = (int)d.Hq;
  p.Hk = (int)d.Hk;
  p.D = (int)d.D;
  p.bf16 = dtype == CMP_NSA_BF16 ? 1 : 0;
  p.eps = eps;
  p.inv_d = 1.f / (float)d.D;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch(CMP_KERNEL_QK_NORM_ROPE, s, [&] { return cmp::launch_qk_norm_rope(p, s, sm_count_cached()); }) ==
                 cudaSuccess
             ? CMP_OK
             : CMP_ERR_CUDA;
}

int cmp_kv_append(const void* k, const void* v, const void* norm_weight, const cmp_rope* rope, float eps,
                  const int32_t* block_table, const int32_t* cu_seqlens, const int32_t* start_pos, int32_t dtype,
                  void* k_cache, void* v_cache, void* stream, const cmp_kv_dims* dims) {
  if (!dims) return CMP_ERR_NULLPTR;
  if (!valid_dtype(dtype)) return CMP_ERR_UNSUPPORTED;
  const cmp_kv_dims& d = *dims;
  if (!in(d.B, 0, INT32_MAX - 1) || !in(d.T, 0, INT32_MAX - 1) || !in(d.Hk, 1, 256) || !valid_head_dim(d.D) ||
      !valid_stride(d.k_stride, d.Hk, d.D) || !valid_stride(d.v_stride, d.Hk, d.D) || !in(d.page_size, 1, 1024) ||
      !in(d.block_num, 1, INT32_MAX / d.page_size) || !in(d.table_stride, 1, INT32_MAX) || (d.B == 0 && d.T != 0) ||
      !(eps >= 0.f) || std::isinf(eps))
    return CMP_ERR_INVALID;
  if (d.B == 0 || d.T == 0) return CMP_OK;
  cmp::KvAppendParams p{};
  const int rc = check_rope(rope, d.D, &p.rope);
  if (rc != CMP_OK) return rc;
  if (!k || !v || !block_table || !cu_seqlens || !k_cache || !v_cache) return CMP_ERR_NULLPTR;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(norm_weight, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(block_table, 4) || !aligned(cu_seqlens, 4) || !aligned(start_pos, 4))
    return CMP_ERR_INVALID;
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.norm_weight = static_cast<const uint16_t*>(norm_weight);
  p.table = block_table;
  p.cu = cu_seqlens;
  p.start_pos = start_pos;
  p.k_cache = static_cast<uint16_t*>(k_cache);
  p.v_cache = static_cast<uint16_t*>(v_cache);
  p.T = d.T;
  p.k_stride = d.k_stride;
  p.v_stride = d.v_stride;
  p.table_stride = d.table_stride;
  p.block_num = d.block_num;
  p.B = (int)d.B;
  p.Hk = (int)d.Hk;
  p.D = (int)d.D;
  p.page = (int)d.page_size;
  p.div_page = cmp::make_fast_div(p.page);
  p.bf16 = dtype == CMP_NSA_BF16 ? 1 : 0;
  p.eps = eps;
  p.inv_d = 1.f / (float)d.D;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  note_word_device();
  return launch(CMP_KERNEL_KV_APPEND, s, [&] { return cmp::launch_kv_append(p, s, sm_count_cached()); }) ==
                 cudaSuccess
             ? CMP_OK
             : CMP_ERR_CUDA;
}

size_t cmp_paged_attention_workspace(const cmp_attn_dims* dims) {
  if (check_attn_dims(dims) != CMP_OK) return 0;
  return attn_path(*dims).total;
}

int cmp_paged_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                        const int32_t* cu_seqlens, const int32_t* start_pos, float scale, int64_t window,
                        int64_t key_block, int64_t key_stride, int32_t dtype, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream, const cmp_attn_dims* dims) {
  if (!dims) return CMP_ERR_NULLPTR;
  if (!valid_dtype(dtype)) return CMP_ERR_UNSUPPORTED;
  const int rc = check_attn_dims(dims);
  if (rc != CMP_OK) return rc;
  const cmp_attn_dims& d = *dims;
  if (!(scale > 0.f) || std::isinf(scale) || !in(window, 0, INT32_MAX) || !in(key_block, 1, INT32_MAX) ||
      !in(key_stride, 1, INT32_MAX))
    return CMP_ERR_INVALID;
  if (d.B == 0 || d.T == 0) return CMP_OK;
  if (!q || !k_cache || !v_cache || !block_table || !cu_seqlens || !out || !workspace) return CMP_ERR_NULLPTR;
  const AttnPath a = attn_path(d);
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(cu_seqlens, 4) || !aligned(start_pos, 4) || !aligned(workspace, 16) ||
      workspace_bytes < a.total)
    return CMP_ERR_INVALID;
  cmp::AttnParams p{};
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.q = static_cast<const uint16_t*>(q);
  p.table = block_table;
  p.cu = cu_seqlens;
  p.start_pos = start_pos;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.part = reinterpret_cast<float*>(ws + a.part);
  p.part_ml = reinterpret_cast<float*>(ws + a.ml);
  p.desc = reinterpret_cast<int4*>(ws + a.desc);
  p.q_stride = d.q_stride;
  p.table_stride = d.table_stride;
  p.block_num = d.block_num;
  p.B = (int)d.B;
  p.T = (int)d.T;
  p.Hq = (int)d.Hq;
  p.Hk = (int)d.Hk;
  p.G = (int)(d.Hq / d.Hk);
  p.D = (int)d.D;
  p.page = (int)d.page_size;
  p.bf16 = dtype == CMP_NSA_BF16 ? 1 : 0;
  p.key_block = (int)key_block;
  p.key_stride = (int)key_stride;
  p.window = (int)window;
  p.max_len = (int)(d.max_len && d.max_len < d.T ? d.max_len : d.T);
  p.withhold = !a.chunk && take_unreachable() ? 1 : 0;
  p.run_shift = 4;
  while ((1 << p.run_shift) < a.key_tile && p.page % (2 << p.run_shift) == 0) ++p.run_shift;
  p.div_g = cmp::make_fast_div(p.G);
  p.div_stride = cmp::make_fast_div(p.key_stride);
  p.div_page = cmp::make_fast_div(p.page);
  p.scale_log2 = scale * 1.4426950408889634f;
  CUtensorMap kmap, vmap;
  if (!cmp::attn_cache_map(&kmap, k_cache, p) || !cmp::attn_cache_map(&vmap, v_cache, p)) return CMP_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  note_word_device();
  const cudaError_t e =
      a.chunk ? launch(CMP_KERNEL_ATTN_CHUNK, s, [&] { return cmp::launch_attn_chunk(p, kmap, vmap, s, a.ctas); })
              : launch(CMP_KERNEL_ATTN_DECODE, s, [&] { return cmp::launch_attn_decode(p, kmap, vmap, s, a.ctas, a.m); });
  if (e != cudaSuccess) return CMP_ERR_CUDA;
  if (launch(CMP_KERNEL_ATTN_COMBINE, s, [&] { return cmp::launch_attn_combine(p, a.m, a.ctas, s); }) != cudaSuccess)
    return CMP_ERR_CUDA;
  return CMP_OK;
}

int cmp_debug_unreachable_barrier(int launches) {
  if (launches < 0) return -1;
  return g_unreachable_barrier.exchange(launches);
}

int cmp_get_error(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return CMP_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return CMP_ERR_CUDA;
  unsigned word = 0;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    auto pe = g_pending_err.find({dev, s});
    if (pe != g_pending_err.end()) {
      word |= pe->second;
      pe->second = 0;
    }
    auto it = g_ws.find({dev, s});
    if (it != g_ws.end() && it->second.ptr) {
      unsigned v = 0;
      if (cudaMemcpy(&v, it->second.ptr, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess)
        return CMP_ERR_CUDA;
      if (v && cudaMemset(it->second.ptr, 0, sizeof(v)) != cudaSuccess) return CMP_ERR_CUDA;
      // a wait that gave up may have left a grid barrier's count behind; the
      // decode arrival counter restarts from zero with it
      if ((v & cmp::kErrTimeout) &&
          cudaMemset(it->second.ptr + kGridBarOffset, 0, zeroed_bytes() - kGridBarOffset) != cudaSuccess)
        return CMP_ERR_CUDA;
      word |= v;
    }
  }
  unsigned na = 0;  // the allocation-free entry point's calls on this device
  if (cmp::noalloc_take_error(dev, &na) != CMP_OK) return CMP_ERR_CUDA;
  word |= na;
  if (dev < 64 && (g_word_devices.load(std::memory_order_relaxed) >> dev & 1)) {  // the paged cache operators' words
    unsigned v = 0;
    if (take_device_words(s, &v) != cudaSuccess) return CMP_ERR_CUDA;
    word |= v;
  }
  if (word & cmp::kErrTimeout) return CMP_ERR_TIMEOUT;
  if (word & cmp::kErrIndex) return CMP_ERR_DEVICE_INDEX;
  return CMP_OK;
}

const char* cmp_status_string(int status) {
  switch (status) {
    case CMP_OK: return "ok";
    case CMP_ERR_NULLPTR: return "a required pointer is NULL";
    case CMP_ERR_INVALID: return "an argument or size is outside the supported range";
    case CMP_ERR_UNSUPPORTED: return "unsupported ratio";
    case CMP_ERR_CUDA: return "CUDA runtime error";
    case CMP_ERR_DEVICE_INDEX: return "a kernel met an out-of-range index and skipped the access";
    case CMP_ERR_TIMEOUT: return "a kernel gave up waiting on its pipeline";
    default: return "unknown status";
  }
}

const char* cmp_kernel_name(int kernel) {
  static const char* names[CMP_KERNEL_COUNT] = {"sched",         "proj_tcgen05",  "proj_mma_sync",
                                                "proj_decode",   "pool_epilogue", "fused_tcgen05",
                                                "finish",        "decode_fused",  "decode_cp",
                                                "nsa_compress",  "nsa_scan",
                                                "qk_norm_rope",  "kv_append",     "attn_decode",
                                                "attn_combine",  "attn_chunk"};
  return (kernel >= 0 && kernel < CMP_KERNEL_COUNT) ? names[kernel] : nullptr;
}

int64_t cmp_launch_count(void) { return g_launches.load(); }

int cmp_profile_start(void) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  for (auto& t : g_timed) {
    g_event_pool.push_back(t.a);
    g_event_pool.push_back(t.b);
  }
  g_timed.clear();
  g_prof = true;
  return CMP_OK;
}

int cmp_profile_stop(double* ms, int64_t* launches) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  g_prof = false;
  double acc[CMP_KERNEL_COUNT] = {0};
  int64_t cnt[CMP_KERNEL_COUNT] = {0};
  int rc = CMP_OK;
  for (auto& t : g_timed) {
    float v = 0.f;
    if (cudaEventSynchronize(t.b) != cudaSuccess || cudaEventElapsedTime(&v, t.a, t.b) != cudaSuccess)
      rc = CMP_ERR_CUDA;
    acc[t.kernel] += v;
    cnt[t.kernel] += 1;
    g_event_pool.push_back(t.a);
    g_event_pool.push_back(t.b);
  }
  g_timed.clear();
  for (int k = 0; k < CMP_KERNEL_COUNT; ++k) {
    if (ms) ms[k] = acc[k];
    if (launches) launches[k] = cnt[k];
  }
  return rc;
}

int cmp_set_proj_kernel(int which) {
  if (which < 0 || which > 8) return -1;
  return g_proj_kernel.exchange(which);
}

}  // extern "C"
