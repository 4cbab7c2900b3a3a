// abi.cu - the extern "C" entry points of libasp.so declared in asp.h:
// host-side argument checks, workspace layout, launches and the device error
// word. No call here allocates memory; only asp_get_device_error synchronises.
#include <atomic>
#include <cmath>
#include <mutex>

#include "asp_internal.cuh"

namespace asp {

namespace {
constexpr int kMaxDevices = 64;
std::atomic<int> g_sm_count[kMaxDevices];

bool is_pow2_le8(int x) { return x == 1 || x == 2 || x == 4 || x == 8; }

// bf16_pages false: the call uses neither k_cache nor v_cache, and both may be missing.
asp_status check_kv(const asp_paged_kv* kv, bool bf16_pages = true) {
  if (!kv || !kv->summaries || !kv->block_table || !kv->seq_lens) return ASP_EINVAL;
  if ((!kv->k_cache || !kv->v_cache) && (bf16_pages || kv->k_cache || kv->v_cache))
    return ASP_EINVAL;
  if (kv->batch <= 0 || kv->num_q_heads <= 0 || kv->num_kv_heads <= 0 || kv->max_pages <= 0 ||
      kv->num_phys_pages <= 0)
    return ASP_EINVAL;
  if (kv->num_q_heads % kv->num_kv_heads != 0) return ASP_EINVAL;
  if (kv->head_dim != 64 && kv->head_dim != 128) return ASP_EUNSUPPORTED;
  if (kv->page_size != 16 && kv->page_size != 32 && kv->page_size != 64) return ASP_EUNSUPPORTED;
  if (!is_pow2_le8(kv->num_kv_heads)) return ASP_EUNSUPPORTED;
  if (!is_pow2_le8(kv->num_q_heads / kv->num_kv_heads)) return ASP_EUNSUPPORTED;
  if ((long long)kv->batch * kv->num_kv_heads > kMaxSegments) return ASP_EUNSUPPORTED;
  if (kv->max_pages > kMaxPages) return ASP_EUNSUPPORTED;
  // page-space (with the decode's split weights) and TMA row coordinates are int32
  if ((long long)kv->batch * kv->num_kv_heads * (kv->max_pages + kMaxPieceCost) >= (1LL << 31))
    return ASP_EUNSUPPORTED;
  if ((long long)kv->num_phys_pages * kv->num_kv_heads * kv->page_size >= (1LL << 31))
    return ASP_EUNSUPPORTED;
  // 16-byte alignment of the cache bases (bulk and tensor copies)
  if ((reinterpret_cast<uintptr_t>(kv->k_cache) | reinterpret_cast<uintptr_t>(kv->v_cache) |
       reinterpret_cast<uintptr_t>(kv->summaries)) & 15u)
    return ASP_EINVAL;
  return ASP_OK;
}

// chunk: the call needs the joins and partials at the workspace's end, which only the chunk
// calls and the prefix call do; a workspace that ends before them serves all others.
asp_status check_ws(const asp_paged_kv* kv, void* ws, size_t ws_bytes, WsLayout* lay,
                    bool chunk = false) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)) return ASP_EWORKSPACE;
  const int sms = current_device_sm_count();
  if (sms <= 0) return ASP_ECUDA;
  *lay = ws_layout(*kv, sms);
  if (ws_bytes < (chunk ? lay->total : lay->joins_off)) return ASP_EWORKSPACE;
  return ASP_OK;
}

bool misaligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

// Whether n elements of `bytes` bytes each from a and m of `mbytes` from b have one in common.
bool overlap(const void* a, size_t n, size_t bytes, const void* b, size_t m, size_t mbytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && n && m && x < y + m * mbytes && y < x + n * bytes;
}

asp_status check_q8(const asp_paged_kv* kv, const asp_q8_pages* pages) {
  const asp_status st = check_kv(kv, false);
  if (st != ASP_OK) return st;
  if (!pages || !pages->k || !pages->v || !pages->scales) return ASP_EINVAL;
  return misaligned(pages->k, 16) || misaligned(pages->v, 16) || misaligned(pages->scales, 16)
             ? ASP_EINVAL
             : ASP_OK;
}

// The packed rows of new tokens: bf16, 16-byte aligned.
asp_status check_rows(int32_t num_tokens, const uint16_t* rows) {
  if (num_tokens < 0 || !rows || misaligned(rows, 16)) return ASP_EINVAL;
  return num_tokens > ASP_MAX_NEW_TOKENS ? ASP_EUNSUPPORTED : ASP_OK;
}

asp_status check_weights(float sm_scale, float decay, const float* w_in, const float* w_out) {
  if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return ASP_EINVAL;
  if (!(decay >= 0.0f) || !std::isfinite(decay)) return ASP_EINVAL;
  return misaligned(w_in, 16) || misaligned(w_out, 16) ? ASP_EINVAL : ASP_OK;
}

// The chunk form subtracts lse / sm_scale from a product: with any lse under 2^27 that stays
// below fp32's largest value from here on.
constexpr float kMinChunkScale = 0x1p-100f;

asp_status from_cuda(cudaError_t e) { return e == cudaSuccess ? ASP_OK : ASP_ECUDA; }

// One warp; thread 0 waits on a barrier that expects one arrival which never
// comes, through the library's bounded wait, and reports the timeout.
__global__ void selftest_wait_kernel(uint32_t* err) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    mbar_fence_init();
  }
  __syncthreads();
  if (threadIdx.x == 0 && !mbar_wait(&bar, 0)) report(err, ASP_DEVERR_TIMEOUT);
}
}  // namespace

int current_device_sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
  int n = g_sm_count[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  g_sm_count[dev].store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t set_max_dynamic_smem(const void* func, int bytes) {
  // The attribute belongs to the function; setting it again is cheap but it
  // is done once per (function, device) to keep capture-time calls minimal.
  static std::mutex mu;
  static const void* done_func[256];
  static int done_dev[256];
  static int done_bytes[256];
  static int n_done = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n_done; ++i)
    if (done_func[i] == func && done_dev[i] == dev && done_bytes[i] >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  // Every kernel of the library asks for the largest shared-memory carveout,
  // so consecutive kernels never make an SM flush L1 and repartition it.
  e = cudaFuncSetAttribute(func, cudaFuncAttributePreferredSharedMemoryCarveout,
                           (int)cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  if (n_done < 256) {
    done_func[n_done] = func;
    done_dev[n_done] = dev;
    done_bytes[n_done] = bytes;
    ++n_done;
  }
  return cudaSuccess;
}

}  // namespace asp

using namespace asp;

extern "C" {

int32_t asp_abi_version(void) { return ASP_ABI_VERSION; }

const char* asp_status_string(asp_status st) {
  switch (st) {
    case ASP_OK: return "ASP_OK";
    case ASP_EINVAL: return "ASP_EINVAL: invalid argument";
    case ASP_EUNSUPPORTED: return "ASP_EUNSUPPORTED: shape outside the supported set";
    case ASP_EWORKSPACE: return "ASP_EWORKSPACE: workspace null, misaligned or too small";
    case ASP_ECUDA: return "ASP_ECUDA: CUDA runtime call or launch failed";
    case ASP_EDEVICE: return "ASP_EDEVICE: device error word set";
  }
  return "unknown asp_status";
}

asp_status asp_workspace_size(const asp_paged_kv* kv, size_t* bytes) {
  if (!bytes) return ASP_EINVAL;
  asp_status st = check_kv(kv, false);
  if (st != ASP_OK) return st;
  const int sms = current_device_sm_count();
  if (sms <= 0) return ASP_ECUDA;
  *bytes = ws_layout(*kv, sms).total;
  return ASP_OK;
}

asp_status asp_workspace_init(void* ws, size_t ws_bytes, asp_stream stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < 256) return ASP_EWORKSPACE;
  // only the error word has to start at zero; zeroing the whole buffer is
  // simplest and still cheap
  return from_cuda(cudaMemsetAsync(ws, 0, ws_bytes, static_cast<cudaStream_t>(stream)));
}

asp_status asp_page_summarize(const asp_paged_kv* kv, int32_t mode, const uint16_t* k_new,
                              const uint16_t* v_new, void* ws, size_t ws_bytes,
                              asp_stream stream) {
  NvtxRange range("asp_page_summarize");
  asp_status st = check_kv(kv);
  if (st != ASP_OK) return st;
  if (mode == ASP_SUMMARIZE_BULK) {
    if (k_new || v_new) return ASP_EINVAL;
  } else if (mode == ASP_SUMMARIZE_APPEND) {
    if (!k_new || !v_new) return ASP_EINVAL;
    if ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 7u)
      return ASP_EINVAL;
  } else {
    return ASP_EINVAL;
  }
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay)) != ASP_OK) return st;
  SummarizeArgs a{kv, mode, k_new, v_new, static_cast<uint32_t*>(ws)};
  return from_cuda(launch_summarize(a, static_cast<cudaStream_t>(stream)));
}

asp_status asp_coverage_select(const asp_paged_kv* kv, const float* q, float gamma,
                               int32_t budget, int32_t* lists, int32_t* lens, void* ws,
                               size_t ws_bytes, asp_stream stream) {
  NvtxRange range("asp_coverage_select");
  asp_status st = check_kv(kv, false);
  if (st != ASP_OK) return st;
  if (!q || !lists || !lens) return ASP_EINVAL;
  if (reinterpret_cast<uintptr_t>(q) & 15u) return ASP_EINVAL;
  if (budget < 0) return ASP_EINVAL;
  if (budget == 0 && !(gamma > 0.0f && gamma <= 1.0f)) return ASP_EINVAL;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay)) != ASP_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  SelectArgs a{kv, q, gamma, budget, lists, lens, reinterpret_cast<float*>(w + lay.scores_off),
               reinterpret_cast<uint32_t*>(w), current_device_sm_count()};
  return from_cuda(launch_select(a, static_cast<cudaStream_t>(stream)));
}

asp_status asp_select_plan(const asp_paged_kv* kv, float gamma, int32_t budget, int32_t append,
                           int32_t* kernels, int32_t* cluster_ctas) {
  asp_status st = check_kv(kv, false);
  if (st != ASP_OK) return st;
  if (!kernels || !cluster_ctas) return ASP_EINVAL;
  if (budget < 0) return ASP_EINVAL;
  if (budget == 0 && !(gamma > 0.0f && gamma <= 1.0f)) return ASP_EINVAL;
  const int sms = current_device_sm_count();
  if (sms <= 0) return ASP_ECUDA;
  const bool all = budget == 0 && gamma >= 1.0f;
  int C = 0;
  if (!all) C = cluster_select_ctas(*kv, sms);
  *cluster_ctas = C;
  *kernels = C > 0 ? 1 : (all && !append ? 1 : 2);
  return ASP_OK;
}

asp_status asp_coverage_select_append(const asp_paged_kv* kv, const uint16_t* k_new,
                                      const uint16_t* v_new, const float* q, float gamma,
                                      int32_t budget, int32_t* lists, int32_t* lens, void* ws,
                                      size_t ws_bytes, asp_stream stream) {
  NvtxRange range("asp_coverage_select_append");
  asp_status st = check_kv(kv);
  if (st != ASP_OK) return st;
  if (!q || !lists || !lens || !k_new || !v_new) return ASP_EINVAL;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_new) |
       reinterpret_cast<uintptr_t>(v_new)) & 15u)
    return ASP_EINVAL;
  if (budget < 0) return ASP_EINVAL;
  if (budget == 0 && !(gamma > 0.0f && gamma <= 1.0f)) return ASP_EINVAL;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay)) != ASP_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  SelectArgs a{kv, q, gamma, budget, lists, lens, reinterpret_cast<float*>(w + lay.scores_off),
               reinterpret_cast<uint32_t*>(w), current_device_sm_count(), k_new, v_new};
  return from_cuda(launch_select(a, static_cast<cudaStream_t>(stream)));
}

asp_status asp_page_scores(const asp_paged_kv* kv, const float* q, float* scores, void* ws,
                           size_t ws_bytes, asp_stream stream) {
  NvtxRange range("asp_page_scores");
  asp_status st = check_kv(kv, false);
  if (st != ASP_OK) return st;
  if (!q || !scores) return ASP_EINVAL;
  if ((reinterpret_cast<uintptr_t>(q) & 15u) || (reinterpret_cast<uintptr_t>(scores) & 3u))
    return ASP_EINVAL;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay)) != ASP_OK) return st;
  SelectArgs a{kv, q, 0.5f, 0, nullptr, nullptr, scores, static_cast<uint32_t*>(ws),
               current_device_sm_count()};
  return from_cuda(launch_scores(a, static_cast<cudaStream_t>(stream)));
}

asp_status asp_sparse_decode(const asp_paged_kv* kv, const float* q, const int32_t* lists,
                             const int32_t* lens, float sm_scale, float* out, float* lse,
                             void* ws, size_t ws_bytes, asp_stream stream) {
  NvtxRange range("asp_sparse_decode");
  asp_status st = check_kv(kv);
  if (st != ASP_OK) return st;
  if (!q || !lists || !lens || !out || !lse) return ASP_EINVAL;
  if (reinterpret_cast<uintptr_t>(q) & 7u) return ASP_EINVAL;
  if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return ASP_EINVAL;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay)) != ASP_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  DecodeArgs a{kv, q, lists, lens, sm_scale, out, lse,
               reinterpret_cast<float*>(w + lay.partials_off),
               reinterpret_cast<int32_t*>(w + lay.arrivals_off), reinterpret_cast<uint32_t*>(w),
               lay.decode_grid, lay.slot_floats};
  return from_cuda(launch_decode(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace asp {
namespace {
// What the three calls that append new tokens have in common. pages null: bf16 pages.
asp_status append(const asp_paged_kv* kv, const asp_q8_pages* pages, const uint16_t* qkv,
                  const int32_t* q_offsets, int32_t num_tokens, const int32_t* positions,
                  int32_t num_axes, const int32_t* pair_axis, const uint16_t* q_weight,
                  const uint16_t* k_weight, float eps, const float* inv_freq, int32_t rotary_dim,
                  int32_t interleaved, uint16_t* q_out, float* q_out_f32, void* ws,
                  size_t ws_bytes, asp_stream stream) {
  asp_status st;
  if ((st = check_rows(num_tokens, qkv)) != ASP_OK) return st;
  if (!q_offsets && num_tokens != kv->batch) return ASP_EINVAL;
  if (!q_out && !q_out_f32) return ASP_EINVAL;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return ASP_EINVAL;
  if (rotary_dim < 0 || rotary_dim > kv->head_dim || rotary_dim % 8 != 0) return ASP_EINVAL;
  if (rotary_dim > 0 && !inv_freq) return ASP_EINVAL;
  if (interleaved != 0 && interleaved != 1) return ASP_EINVAL;
  if (num_axes < 1 || num_axes > ASP_MAX_AXES) return ASP_EINVAL;
  if (misaligned(q_out, 16) || misaligned(q_out_f32, 16) || misaligned(q_weight, 8) ||
      misaligned(k_weight, 8) || misaligned(inv_freq, 4) || misaligned(pair_axis, 4))
    return ASP_EINVAL;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay)) != ASP_OK) return st;
  if (num_tokens == 0) return ASP_OK;
  NormRotateArgs a{kv, qkv, q_offsets, num_tokens, positions, q_weight, k_weight, eps, inv_freq,
                   rotary_dim, interleaved, q_out, q_out_f32, static_cast<uint32_t*>(ws),
                   current_device_sm_count(), pages, num_axes, pair_axis};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return from_cuda(pages || num_axes > 1 || pair_axis ? launch_append_rows(a, s)
                                                      : launch_norm_rotate(a, s));
}
}  // namespace
}  // namespace asp

extern "C" {

asp_status asp_norm_rotate_append(const asp_paged_kv* kv, const uint16_t* qkv,
                                  const int32_t* q_offsets, int32_t num_tokens,
                                  const int32_t* positions, const uint16_t* q_weight,
                                  const uint16_t* k_weight, float eps, const float* inv_freq,
                                  int32_t rotary_dim, int32_t interleaved, uint16_t* q_out,
                                  float* q_out_f32, void* ws, size_t ws_bytes, asp_stream stream) {
  NvtxRange range("asp_norm_rotate_append");
  const asp_status st = check_kv(kv);
  if (st != ASP_OK) return st;
  return append(kv, nullptr, qkv, q_offsets, num_tokens, positions, 1, nullptr, q_weight, k_weight,
                eps, inv_freq, rotary_dim, interleaved, q_out, q_out_f32, ws, ws_bytes, stream);
}

asp_status asp_norm_rotate_axes_append(const asp_paged_kv* kv, const uint16_t* qkv,
                                       const int32_t* q_offsets, int32_t num_tokens,
                                       const int32_t* positions, int32_t num_axes,
                                       const int32_t* pair_axis, const uint16_t* q_weight,
                                       const uint16_t* k_weight, float eps, const float* inv_freq,
                                       int32_t rotary_dim, int32_t interleaved, uint16_t* q_out,
                                       float* q_out_f32, void* ws, size_t ws_bytes,
                                       asp_stream stream) {
  NvtxRange range("asp_norm_rotate_axes_append");
  const asp_status st = check_kv(kv);
  if (st != ASP_OK) return st;
  return append(kv, nullptr, qkv, q_offsets, num_tokens, positions, num_axes, pair_axis, q_weight,
                k_weight, eps, inv_freq, rotary_dim, interleaved, q_out, q_out_f32, ws, ws_bytes,
                stream);
}

asp_status asp_q8_append(const asp_paged_kv* kv, const asp_q8_pages* pages, const uint16_t* qkv,
                         const int32_t* q_offsets, int32_t num_tokens, const int32_t* positions,
                         int32_t num_axes, const int32_t* pair_axis, const uint16_t* q_weight,
                         const uint16_t* k_weight, float eps, const float* inv_freq,
                         int32_t rotary_dim, int32_t interleaved, uint16_t* q_out,
                         float* q_out_f32, void* ws, size_t ws_bytes, asp_stream stream) {
  NvtxRange range("asp_q8_append");
  const asp_status st = check_q8(kv, pages);
  if (st != ASP_OK) return st;
  return append(kv, pages, qkv, q_offsets, num_tokens, positions, num_axes, pair_axis, q_weight,
                k_weight, eps, inv_freq, rotary_dim, interleaved, q_out, q_out_f32, ws, ws_bytes,
                stream);
}

asp_status asp_q8_read(const asp_paged_kv* kv, const asp_q8_pages* pages, uint16_t* k_out,
                       uint16_t* v_out, const int32_t* dst_table, int32_t dst_pages, void* ws,
                       size_t ws_bytes, asp_stream stream) {
  NvtxRange range("asp_q8_read");
  asp_status st = check_q8(kv, pages);
  if (st != ASP_OK) return st;
  if (!k_out || !v_out || !dst_table || misaligned(k_out, 32) || misaligned(v_out, 32))
    return ASP_EINVAL;
  if (dst_pages <= 0) return ASP_EINVAL;
  if ((long long)dst_pages * kv->num_kv_heads * kv->page_size >= (1LL << 31))
    return ASP_EUNSUPPORTED;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay)) != ASP_OK) return st;
  Q8ReadArgs a{kv, pages, k_out, v_out, dst_table, dst_pages, static_cast<uint32_t*>(ws),
               current_device_sm_count()};
  return from_cuda(launch_q8_read(a, static_cast<cudaStream_t>(stream)));
}

asp_status asp_q8_decode(const asp_paged_kv* kv, const asp_q8_pages* pages, const float* q,
                         const int32_t* lists, const int32_t* lens, float sm_scale, float* out,
                         float* lse, void* ws, size_t ws_bytes, asp_stream stream) {
  NvtxRange range("asp_q8_decode");
  asp_status st = check_q8(kv, pages);
  if (st != ASP_OK) return st;
  if (!q || !lists || !lens || !out || !lse || misaligned(q, 8)) return ASP_EINVAL;
  if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return ASP_EINVAL;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay)) != ASP_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  DecodeArgs a{kv, q, lists, lens, sm_scale, out, lse,
               reinterpret_cast<float*>(w + lay.partials_off),
               reinterpret_cast<int32_t*>(w + lay.arrivals_off), reinterpret_cast<uint32_t*>(w),
               lay.decode_grid, lay.slot_floats, pages};
  return from_cuda(launch_q8_decode(a, static_cast<cudaStream_t>(stream)));
}

asp_status asp_chunk_attention(const asp_paged_kv* kv, const uint16_t* q,
                               const int32_t* q_offsets, int32_t num_tokens, float sm_scale,
                               uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                               asp_stream stream) {
  NvtxRange range("asp_chunk_attention");
  asp_status st = check_kv(kv);
  if (st != ASP_OK) return st;
  if ((st = check_rows(num_tokens, q)) != ASP_OK) return st;
  if (!q_offsets || !out || !lse || misaligned(out, 16)) return ASP_EINVAL;
  if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return ASP_EINVAL;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay, true)) != ASP_OK) return st;
  if (num_tokens == 0) return ASP_OK;
  uint8_t* w = static_cast<uint8_t*>(ws);
  ChunkAttentionArgs a{kv, q, q_offsets, num_tokens, sm_scale, out, lse,
                       reinterpret_cast<ChunkJoin*>(w + lay.joins_off),
                       reinterpret_cast<float*>(w + lay.chunk_off), reinterpret_cast<uint32_t*>(w),
                       current_device_sm_count()};
  return from_cuda(launch_chunk_attention(a, static_cast<cudaStream_t>(stream)));
}

asp_status asp_prefix_attention(const asp_paged_kv* kv, const uint16_t* q,
                                const int32_t* row_offsets, int32_t num_rows, float sm_scale,
                                const void* own_out, int32_t own_bf16, const float* own_lse,
                                uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                                asp_stream stream) {
  NvtxRange range("asp_prefix_attention");
  asp_status st = check_kv(kv);
  if (st != ASP_OK) return st;
  if ((st = check_rows(num_rows, q)) != ASP_OK) return st;
  if (!row_offsets || !out || !lse || misaligned(out, 16)) return ASP_EINVAL;
  if ((own_out == nullptr) != (own_lse == nullptr) || misaligned(own_out, 16)) return ASP_EINVAL;
  if (own_bf16 != 0 && own_bf16 != 1) return ASP_EINVAL;
  if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return ASP_EINVAL;
  if (!ws || misaligned(ws, 256)) return ASP_EWORKSPACE;
  // A row's parts are read by other blocks than those that write it, but for a bf16 own part,
  // which only the block that replaces it reads.
  const size_t rows = (size_t)num_rows * kv->num_q_heads, all = rows * kv->head_dim;
  if (overlap(out, all, 2, q, all, 2) || overlap(lse, rows, 4, own_lse, rows, 4) ||
      (!(own_bf16 && out == own_out) && overlap(out, all, 2, own_out, all, own_bf16 ? 2 : 4)))
    return ASP_EINVAL;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay, true)) != ASP_OK) return st;
  if (num_rows == 0) return ASP_OK;
  uint8_t* w = static_cast<uint8_t*>(ws);
  ChunkAttentionArgs a{kv, q, row_offsets, num_rows, sm_scale, out, lse,
                       reinterpret_cast<ChunkJoin*>(w + lay.joins_off),
                       reinterpret_cast<float*>(w + lay.chunk_off), reinterpret_cast<uint32_t*>(w),
                       current_device_sm_count(), own_out, own_lse, own_bf16};
  return from_cuda(launch_prefix_attention(a, static_cast<cudaStream_t>(stream)));
}

asp_status asp_chunk_weights(const asp_paged_kv* kv, const uint16_t* q, const int32_t* q_offsets,
                             int32_t num_tokens, const float* lse, float sm_scale, float decay,
                             const float* w_in, float* w_out, void* ws, size_t ws_bytes,
                             asp_stream stream) {
  NvtxRange range("asp_chunk_weights");
  asp_status st = check_kv(kv);
  if (st != ASP_OK) return st;
  if ((st = check_rows(num_tokens, q)) != ASP_OK) return st;
  if (!q_offsets || !lse || !w_out) return ASP_EINVAL;
  if ((st = check_weights(sm_scale, decay, w_in, w_out)) != ASP_OK) return st;
  if (sm_scale < kMinChunkScale) return ASP_EINVAL;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay, true)) != ASP_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  WeightArgs a{kv, q, q_offsets, num_tokens, nullptr, nullptr, nullptr, lse, sm_scale, decay,
               w_in, w_out, reinterpret_cast<ChunkJoin*>(w + lay.joins_off),
               reinterpret_cast<float*>(w + lay.chunk_off), reinterpret_cast<uint32_t*>(w),
               current_device_sm_count()};
  return from_cuda(launch_chunk_weights(a, static_cast<cudaStream_t>(stream)));
}

asp_status asp_decode_weights(const asp_paged_kv* kv, const float* q, const int32_t* lists,
                              const int32_t* lens, const float* lse, float sm_scale, float decay,
                              const float* w_in, float* w_out, void* ws, size_t ws_bytes,
                              asp_stream stream) {
  NvtxRange range("asp_decode_weights");
  asp_status st = check_kv(kv);
  if (st != ASP_OK) return st;
  if (!q || !lse || !w_out || misaligned(q, 16)) return ASP_EINVAL;
  if ((lists == nullptr) != (lens == nullptr)) return ASP_EINVAL;
  if ((st = check_weights(sm_scale, decay, w_in, w_out)) != ASP_OK) return st;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay)) != ASP_OK) return st;
  WeightArgs a{kv, nullptr, nullptr, kv->batch, q, lists, lens, lse, sm_scale, decay, w_in, w_out,
               nullptr, nullptr, static_cast<uint32_t*>(ws), current_device_sm_count()};
  return from_cuda(launch_decode_weights(a, static_cast<cudaStream_t>(stream)));
}

asp_status asp_weight_evict(const asp_paged_kv* kv, const float* weights, int32_t keep,
                            int32_t recent, const int32_t* dst_table, float* w_out, int32_t* kept,
                            int32_t* new_lens, void* ws, size_t ws_bytes, asp_stream stream) {
  NvtxRange range("asp_weight_evict");
  asp_status st = check_kv(kv);
  if (st != ASP_OK) return st;
  if (!weights || !dst_table || !w_out || !kept || !new_lens) return ASP_EINVAL;
  if (new_lens == kv->seq_lens) return ASP_EINVAL;
  if (misaligned(weights, 16) || misaligned(w_out, 16)) return ASP_EINVAL;
  if (keep < 1 || (long long)keep > (long long)kv->max_pages * kv->page_size) return ASP_EINVAL;
  if (recent < 0 || recent > keep) return ASP_EINVAL;
  WsLayout lay;
  if ((st = check_ws(kv, ws, ws_bytes, &lay)) != ASP_OK) return st;
  EvictArgs a{kv, weights, keep, recent, dst_table, w_out, kept, new_lens,
              static_cast<uint32_t*>(ws), current_device_sm_count()};
  return from_cuda(launch_evict(a, static_cast<cudaStream_t>(stream)));
}

asp_status asp_selftest_wait_timeout(void* ws, size_t ws_bytes, asp_stream stream) {
  NvtxRange range("asp_selftest_wait_timeout");
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < 256) return ASP_EWORKSPACE;
  selftest_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<uint32_t*>(ws));
  return from_cuda(cudaGetLastError());
}

asp_status asp_get_device_error(void* ws, uint32_t* code_out, asp_stream stream) {
  if (!ws || !code_out) return ASP_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t code = 0;
  cudaError_t e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemcpy(&code, ws, sizeof(code), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && code) e = cudaMemset(ws, 0, sizeof(code));
  if (e != cudaSuccess) return ASP_ECUDA;
  *code_out = code;
  return code ? ASP_EDEVICE : ASP_OK;
}

}  // extern "C"
