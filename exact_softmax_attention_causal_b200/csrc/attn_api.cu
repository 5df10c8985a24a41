// The extern "C" boundary: argument validation, the decode split plan and
// dispatch to the kernels. Nothing here allocates device memory.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "internal.h"

namespace attn {

void* tensor_map_encode_fn() {
  static void* fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = f;
  });
  return fn;
}

long long wait_budget_cycles() {
  const char* s = std::getenv("ATTN_WAIT_BUDGET_CYCLES");
  const long long v = s ? std::atoll(s) : 0;
  return v > 0 ? v : 1000000000LL;
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int current_sm_count(int* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  if (cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return ATTN_ERR_CUDA;
  return ATTN_OK;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_version(void) { return 100; }

const char* attn_status_string(int status) {
  switch (status) {
    case ATTN_OK:
      return "ok";
    case ATTN_ERR_INVALID_ARG:
      return "invalid argument";
    case ATTN_ERR_UNSUPPORTED:
      return "unsupported configuration (head dimension must be 64 or 128)";
    case ATTN_ERR_CUDA:
      return "CUDA runtime or driver call failed";
    case ATTN_ERR_DEVICE_CHECK:
      return "device check failed: block-table entry or seq_len out of range";
    case ATTN_ERR_TIMEOUT:
      return "a bounded pipeline wait expired";
    case ATTN_ERR_WORKSPACE:
      return "workspace missing or too small";
    default:
      return "unknown status";
  }
}

int attn_prefill(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int N,
                 int d, int mask_kind, int window, float scale, int32_t* status, attn_stream_t stream) {
  if (!q || !k || !v || !o) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || d <= 0) return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (mask_kind != ATTN_MASK_FULL && mask_kind != ATTN_MASK_CAUSAL && mask_kind != ATTN_MASK_SLIDING_WINDOW)
    return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_SLIDING_WINDOW && window < 1) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  // TMA coordinates and the persistent kernel's item indices are int32
  if (static_cast<long long>(B) * Hq * N > (1LL << 31) - 1) return ATTN_ERR_UNSUPPORTED;
  if (mask_kind == ATTN_MASK_SLIDING_WINDOW && window >= N) mask_kind = ATTN_MASK_CAUSAL;
  return launch_prefill(q, k, v, o, lse, B, Hq, Hkv, N, d, mask_kind, window, scale, status,
                        reinterpret_cast<cudaStream_t>(stream));
}

int attn_prefill_paged(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                       const int32_t* seq_lens, void* o, float* lse, int B, int Hq, int Hkv, int Nq, int d,
                       int num_blocks, int block_size, int max_blocks_per_seq, int max_seq_len, int mask_kind,
                       int window, float scale, int32_t* status, attn_stream_t stream) {
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || d <= 0 || num_blocks <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || max_seq_len < Nq)
    return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * block_size < max_seq_len) return ATTN_ERR_INVALID_ARG;
  if (mask_kind != ATTN_MASK_FULL && mask_kind != ATTN_MASK_CAUSAL && mask_kind != ATTN_MASK_SLIDING_WINDOW)
    return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_SLIDING_WINDOW && window < 1) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return ATTN_ERR_INVALID_ARG;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hq * Nq > (1LL << 31) - 1) return ATTN_ERR_UNSUPPORTED;
  if (mask_kind == ATTN_MASK_SLIDING_WINDOW && window >= max_seq_len) mask_kind = ATTN_MASK_CAUSAL;
  return launch_prefill_paged(q, k_cache, v_cache, block_table, seq_lens, o, lse, B, Hq, Hkv, Nq, d, num_blocks,
                              block_size, max_blocks_per_seq, max_seq_len, mask_kind, window, scale, status,
                              reinterpret_cast<cudaStream_t>(stream));
}

size_t attn_prefill_paged_varlen_workspace_bytes(int d) {
  int sms = 0;
  if ((d != 64 && d != 128) || current_sm_count(&sms) != ATTN_OK) return 0;
  return varlen_workspace_bytes(d, sms);
}

int attn_prefill_paged_varlen(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                              const int32_t* cu_q, const int32_t* seq_lens, const float* sinks, void* o, float* lse,
                              int B, int T, int Hq, int Hkv, int d, int num_blocks, int block_size,
                              int max_blocks_per_seq, int max_seq_len, int mask_kind, int window, int n_sink,
                              float scale, void* workspace, size_t workspace_bytes, int32_t* status,
                              attn_stream_t stream) {
  if (!q || !k_cache || !v_cache || !block_table || !cu_q || !seq_lens || !o) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || T <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || num_blocks <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || max_seq_len <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * block_size < max_seq_len) return ATTN_ERR_INVALID_ARG;
  if (mask_kind != ATTN_MASK_FULL && mask_kind != ATTN_MASK_CAUSAL && mask_kind != ATTN_MASK_SLIDING_WINDOW)
    return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_SLIDING_WINDOW && window < 1) return ATTN_ERR_INVALID_ARG;
  if (n_sink < 0 || (n_sink > 0 && mask_kind != ATTN_MASK_SLIDING_WINDOW)) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  if (!aligned4(block_table) || !aligned4(cu_q) || !aligned4(seq_lens) || !aligned4(sinks) || !aligned4(lse))
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128) return ATTN_ERR_UNSUPPORTED;
  // row indices are int32; positions leave room for a window's and a tile's width
  if (static_cast<long long>(T) * Hq > (1LL << 31) - 1 || max_seq_len > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
  // Window and sinks that leave no gap hide nothing: a key behind the sinks is at most max_seq_len - 1 - n_sink back.
  // The others add up to less than 2^30, so the kernel's counts of keys fit 32 bits.
  if (mask_kind == ATTN_MASK_SLIDING_WINDOW && static_cast<long long>(window) + n_sink >= max_seq_len)
    mask_kind = ATTN_MASK_CAUSAL, n_sink = 0;
  int sms = 0;
  if (current_sm_count(&sms) != ATTN_OK) return ATTN_ERR_CUDA;
  if (!workspace || !aligned16(workspace) || workspace_bytes < varlen_workspace_bytes(d, sms))
    return ATTN_ERR_WORKSPACE;
  const VarlenArgs a{q,           k_cache,    v_cache,   block_table, cu_q,   seq_lens, sinks, o,
                     lse,         B,          T,         Hq,          Hkv,    d,        num_blocks,
                     block_size,  max_blocks_per_seq, max_seq_len, mask_kind, window, n_sink, sms,
                     scale,       workspace,  status};
  return launch_prefill_varlen(a, reinterpret_cast<cudaStream_t>(stream));
}

int attn_decode_plan(int B, int Hq, int Hkv, int max_seq_len, int num_sms, int* chunk_tokens, int* num_splits) {
  DecodePlan plan;
  const int rc = plan_decode(B, Hq, Hkv, max_seq_len, num_sms, &plan);
  if (rc != ATTN_OK) return rc;
  if (chunk_tokens) *chunk_tokens = plan.chunk;
  if (num_splits) *num_splits = plan.splits;
  return ATTN_OK;
}

}  // extern "C"

namespace {

// Workspace bytes of a (possibly windowed) decode, 0 for invalid sizes.
size_t decode_bytes(int B, int Hq, int Hkv, int d, int max_seq_len, int block_size, int window, int n_sink) {
  if (d != 64 && d != 128) return 0;
  if (block_size <= 0 || block_size % 16 != 0) return 0;
  if (window < 0 || n_sink < 0 || max_seq_len <= 0) return 0;
  int sms = 0;
  if (current_sm_count(&sms) != ATTN_OK) return 0;
  DecodePlan plan;
  if (plan_decode(B, Hq, Hkv, decode_plan_length(max_seq_len, window, n_sink), sms, &plan) != ATTN_OK) return 0;
  return decode_workspace_bytes(B, Hq, Hkv, d, plan);
}

int decode_common(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                  const int32_t* seq_lens, const float* sinks, void* o, float* lse, int B, int Hq, int Hkv, int d,
                  int num_blocks, int block_size, int max_blocks_per_seq, int max_seq_len, int window, int n_sink,
                  float scale, void* workspace, size_t workspace_bytes, int32_t* status, attn_stream_t stream) {
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 ||
      max_seq_len <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * block_size < max_seq_len) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  // sinks: the first n_sink positions, only beside a finite window, 0 <= n_sink <= n
  if (window < 0 || n_sink < 0 || n_sink > max_seq_len || (n_sink > 0 && window == 0)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return ATTN_ERR_INVALID_ARG;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_INVALID_ARG;
  if (sinks && (reinterpret_cast<uintptr_t>(sinks) & 3u)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (block_size % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  if (B > 65535 || static_cast<long long>(Hkv) * ((Hq / Hkv + 15) / 16) > 65535) return ATTN_ERR_UNSUPPORTED;
  // a window that covers every position hides nothing: the sink positions are inside it
  if (window >= max_seq_len) window = n_sink = 0;
  int sms = 0;
  if (current_sm_count(&sms) != ATTN_OK) return ATTN_ERR_CUDA;
  DecodePlan plan;
  if (plan_decode(B, Hq, Hkv, decode_plan_length(max_seq_len, window, n_sink), sms, &plan) != ATTN_OK)
    return ATTN_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < decode_workspace_bytes(B, Hq, Hkv, d, plan))
    return ATTN_ERR_WORKSPACE;
  // A captured call keeps its tag on every replay, so the counters would hold the last replay's counts: its graph
  // clears them first.
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(reinterpret_cast<cudaStream_t>(stream), &capture) != cudaSuccess) return ATTN_ERR_CUDA;
  if (capture != cudaStreamCaptureStatusNone && plan.splits > 1) {
    const DecodeWorkspace ws = decode_workspace_layout(B, Hq, Hkv, d, plan);
    if (cudaMemsetAsync(static_cast<uint8_t*>(workspace) + ws.counters_offset, 0, ws.bytes - ws.counters_offset,
                        reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
      return ATTN_ERR_CUDA;
  }
  const cudaError_t e = launch_decode(q, k_cache, v_cache, block_table, seq_lens, sinks, o, lse, B, Hq, Hkv, d,
                                      num_blocks, block_size, max_blocks_per_seq, max_seq_len, window, n_sink, scale,
                                      workspace, plan, status, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Table sizes: positions, slots and sums of blocks are 32-bit, and a CTA keeps
// three values per sequence in shared memory.
bool table_sizes_fit(int B, int num_blocks, int block_size, int max_blocks_per_seq) {
  const long long most = (1LL << 31) - 1;
  return B <= kMaxTableSeqs && static_cast<long long>(num_blocks) * block_size <= most &&
         static_cast<long long>(max_blocks_per_seq) * block_size <= most &&
         static_cast<long long>(B) * max_blocks_per_seq <= most;
}

// Checks shared by the norm and rotation entry points. strides: (sequence,
// token, head) of q, k, v in elements; a head row is contiguous.
int norm_rope_args(const void* q, const void* k, const void* v, const int64_t* strides, const void* q_weight,
                   const void* k_weight, int weight_bf16, const float* cos_table, const float* sin_table,
                   const int32_t* positions, int B, int N, int Hq, int Hkv, int d, int rotary_dim, int max_pos,
                   float eps, int interleaved, NormRopeArgs* a) {
  if (!strides || !cos_table || !sin_table) return ATTN_ERR_INVALID_ARG;
  if ((q_weight == nullptr) != (k_weight == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || N <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || max_pos <= 0) return ATTN_ERR_INVALID_ARG;
  if (!positions && max_pos < N) return ATTN_ERR_INVALID_ARG;
  if (q_weight && (!(eps >= 0.f) || !std::isfinite(eps))) return ATTN_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, q_weight, k_weight, (const void*)cos_table, (const void*)sin_table})
    if (!aligned16(p)) return ATTN_ERR_INVALID_ARG;
  if (!aligned4(positions)) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 9; ++i)
    if (strides[i] % 8 != 0) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (rotary_dim <= 0 || rotary_dim > d) return ATTN_ERR_INVALID_ARG;
  if (rotary_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  if (Hq > 65535 || Hkv > 65535 ||
      static_cast<long long>(B) * N > ((1LL << 31) - 1) / norm_rope_chunks(Hq, Hkv))
    return ATTN_ERR_UNSUPPORTED;
  const void* x[3] = {q, k, v};
  for (int t = 0; t < 3; ++t) {
    a->x[t] = x[t];
    a->sb[t] = strides[3 * t], a->sn[t] = strides[3 * t + 1], a->sh[t] = strides[3 * t + 2];
  }
  a->w[0] = q_weight, a->w[1] = k_weight, a->w_bf16 = weight_bf16 != 0;
  a->cos_t = cos_table, a->sin_t = sin_table, a->positions = positions;
  a->B = B, a->N = N, a->Hq = Hq, a->Hkv = Hkv, a->d = d, a->rd = rotary_dim, a->max_pos = max_pos;
  a->interleaved = interleaved != 0;
  a->eps = eps;
  return ATTN_OK;
}

}  // namespace

extern "C" {

size_t attn_decode_workspace_bytes(int B, int Hq, int Hkv, int d, int max_seq_len, int block_size) {
  return decode_bytes(B, Hq, Hkv, d, max_seq_len, block_size, 0, 0);
}

size_t attn_decode_window_workspace_bytes(int B, int Hq, int Hkv, int d, int max_seq_len, int block_size, int window,
                                          int n_sink) {
  if (window >= max_seq_len) window = n_sink = 0;
  return decode_bytes(B, Hq, Hkv, d, max_seq_len, block_size, window, n_sink);
}

int attn_decode_paged(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                      const int32_t* seq_lens, void* o, float* lse, int B, int Hq, int Hkv, int d,
                      int num_blocks, int block_size, int max_blocks_per_seq, int max_seq_len, float scale,
                      void* workspace, size_t workspace_bytes, int32_t* status, attn_stream_t stream) {
  return decode_common(q, k_cache, v_cache, block_table, seq_lens, nullptr, o, lse, B, Hq, Hkv, d, num_blocks,
                       block_size, max_blocks_per_seq, max_seq_len, 0, 0, scale, workspace, workspace_bytes, status,
                       stream);
}

int attn_decode_paged_window(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                             const int32_t* seq_lens, const float* sinks, void* o, float* lse, int B, int Hq, int Hkv,
                             int d, int num_blocks, int block_size, int max_blocks_per_seq, int max_seq_len,
                             int window, int n_sink, float scale, void* workspace, size_t workspace_bytes,
                             int32_t* status, attn_stream_t stream) {
  return decode_common(q, k_cache, v_cache, block_table, seq_lens, sinks, o, lse, B, Hq, Hkv, d, num_blocks,
                       block_size, max_blocks_per_seq, max_seq_len, window, n_sink, scale, workspace,
                       workspace_bytes, status, stream);
}

size_t attn_prefill_backward_workspace_bytes(int B, int Hq, int N) {
  if (B <= 0 || Hq <= 0 || N <= 0) return 0;
  return backward_workspace_bytes(B, Hq, N);
}

int attn_prefill_backward(const void* q, const void* k, const void* v, const void* o, const void* d_o,
                          const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int d,
                          int mask_kind, int window, float scale, void* workspace, size_t workspace_bytes,
                          int32_t* status, attn_stream_t stream) {
  if (!q || !k || !v || !o || !d_o || !lse || !dq || !dk || !dv) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || d <= 0) return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (mask_kind != ATTN_MASK_FULL && mask_kind != ATTN_MASK_CAUSAL && mask_kind != ATTN_MASK_SLIDING_WINDOW)
    return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_SLIDING_WINDOW && window < 1) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(d_o) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (B > 65535 || Hq > 65535 || static_cast<long long>(B) * Hq * N > (1LL << 31) - 1) return ATTN_ERR_UNSUPPORTED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) ||
      workspace_bytes < backward_workspace_bytes(B, Hq, N))
    return ATTN_ERR_WORKSPACE;
  if (mask_kind == ATTN_MASK_SLIDING_WINDOW && window >= N) mask_kind = ATTN_MASK_CAUSAL;
  return launch_backward(q, k, v, o, d_o, lse, dq, dk, dv, B, Hq, Hkv, N, d, mask_kind, window, scale, workspace,
                         status, reinterpret_cast<cudaStream_t>(stream));
}

size_t attn_mla_decode_workspace_bytes(int B, int H, int d_latent, int d_rope, int max_seq_len) {
  if (d_latent != 512 || d_rope != 64) return 0;
  int sms = 0;
  if (current_sm_count(&sms) != ATTN_OK) return 0;
  MlaPlan plan;
  if (plan_mla(B, H, max_seq_len, sms, &plan) != ATTN_OK) return 0;
  return mla_workspace_bytes(B, H, plan);
}

int attn_mla_decode_paged(const void* q, const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                          void* o, float* lse, int B, int H, int d_latent, int d_rope, int num_blocks, int block_size,
                          int max_blocks_per_seq, int max_seq_len, float scale, void* workspace,
                          size_t workspace_bytes, int32_t* status, attn_stream_t stream) {
  if (!q || !cache || !block_table || !seq_lens || !o) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || d_latent <= 0 || d_rope <= 0 || num_blocks <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || max_seq_len <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * block_size < max_seq_len) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return ATTN_ERR_INVALID_ARG;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_INVALID_ARG;
  if (d_latent != 512 || d_rope != 64) return ATTN_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128) return ATTN_ERR_UNSUPPORTED;
  if (B > 65535 || (H + 63) / 64 > 65535) return ATTN_ERR_UNSUPPORTED;
  int sms = 0;
  if (current_sm_count(&sms) != ATTN_OK) return ATTN_ERR_CUDA;
  MlaPlan plan;
  if (plan_mla(B, H, max_seq_len, sms, &plan) != ATTN_OK) return ATTN_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < mla_workspace_bytes(B, H, plan))
    return ATTN_ERR_WORKSPACE;
  return launch_mla_decode(q, cache, block_table, seq_lens, o, lse, B, H, num_blocks, block_size,
                           max_blocks_per_seq, max_seq_len, scale, workspace, plan, status,
                           reinterpret_cast<cudaStream_t>(stream));
}

int attn_paged_extend(const int32_t* seq_lens, const int32_t* new_lens, int32_t* block_table,
                      const int32_t* free_blocks, const int32_t* num_free, int32_t* seq_lens_out,
                      int32_t* num_free_out, int32_t* cu_q, int32_t* positions, int32_t* slots, int B, int num_blocks,
                      int block_size, int max_blocks_per_seq, int free_capacity, int max_tokens, int32_t* status,
                      attn_stream_t stream) {
  if (!seq_lens || !new_lens || !block_table || !free_blocks || !num_free || !seq_lens_out || !num_free_out || !cu_q)
    return ATTN_ERR_INVALID_ARG;
  if (max_tokens < 0 || (max_tokens > 0 && (!positions || !slots))) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 || free_capacity <= 0)
    return ATTN_ERR_INVALID_ARG;
  for (const void* p : {(const void*)seq_lens, (const void*)new_lens, (const void*)block_table,
                        (const void*)free_blocks, (const void*)num_free, (const void*)seq_lens_out,
                        (const void*)num_free_out, (const void*)cu_q, (const void*)positions, (const void*)slots})
    if (!aligned4(p)) return ATTN_ERR_INVALID_ARG;
  if (!table_sizes_fit(B, num_blocks, block_size, max_blocks_per_seq)) return ATTN_ERR_UNSUPPORTED;
  return launch_paged_extend(seq_lens, new_lens, block_table, free_blocks, num_free, seq_lens_out, num_free_out, cu_q,
                             positions, slots, B, num_blocks, block_size, max_blocks_per_seq, free_capacity,
                             max_tokens, status, reinterpret_cast<cudaStream_t>(stream));
}

int attn_paged_release(const int32_t* seq_lens, const int32_t* finished, const int32_t* block_table,
                       int32_t* free_blocks, const int32_t* num_free, int32_t* seq_lens_out, int32_t* num_free_out,
                       int B, int num_blocks, int block_size, int max_blocks_per_seq, int free_capacity,
                       int32_t* status, attn_stream_t stream) {
  if (!seq_lens || !finished || !block_table || !free_blocks || !num_free || !seq_lens_out || !num_free_out)
    return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 || free_capacity <= 0)
    return ATTN_ERR_INVALID_ARG;
  for (const void* p : {(const void*)seq_lens, (const void*)finished, (const void*)block_table,
                        (const void*)free_blocks, (const void*)num_free, (const void*)seq_lens_out,
                        (const void*)num_free_out})
    if (!aligned4(p)) return ATTN_ERR_INVALID_ARG;
  if (!table_sizes_fit(B, num_blocks, block_size, max_blocks_per_seq)) return ATTN_ERR_UNSUPPORTED;
  return launch_paged_release(seq_lens, finished, block_table, free_blocks, num_free, seq_lens_out, num_free_out, B,
                              num_blocks, block_size, max_blocks_per_seq, free_capacity, status,
                              reinterpret_cast<cudaStream_t>(stream));
}

int attn_qk_norm_rope(const void* q, const void* k, const void* v, const int64_t* strides, const void* q_weight,
                      const void* k_weight, int weight_bf16, const float* cos_table, const float* sin_table,
                      const int32_t* positions, void* q_out, void* k_out, void* v_out, int B, int N, int Hq, int Hkv,
                      int d, int rotary_dim, int max_pos, float eps, int interleaved, int32_t* status,
                      attn_stream_t stream) {
  NormRopeArgs a;
  const int rc = norm_rope_args(q, k, v, strides, q_weight, k_weight, weight_bf16, cos_table, sin_table, positions, B,
                                N, Hq, Hkv, d, rotary_dim, max_pos, eps, interleaved, &a);
  if (rc != ATTN_OK) return rc;
  if (!q_out || !k_out || !v_out || !aligned16(q_out) || !aligned16(k_out) || !aligned16(v_out))
    return ATTN_ERR_INVALID_ARG;
  if (!q || !k || !v) return ATTN_ERR_INVALID_ARG;
  if (current_sm_count(&a.sms) != ATTN_OK) return ATTN_ERR_CUDA;
  return launch_norm_rope(a, q_out, k_out, v_out, nullptr, 0, status, reinterpret_cast<cudaStream_t>(stream));
}

int attn_qk_norm_rope_paged(const void* q, const void* k, const void* v, const int64_t* strides, const void* q_weight,
                            const void* k_weight, int weight_bf16, const float* cos_table, const float* sin_table,
                            const int32_t* positions, const int32_t* slots, void* q_out, void* k_cache, void* v_cache,
                            int T, int Hq, int Hkv, int d, int num_blocks, int block_size, int rotary_dim,
                            int max_pos, float eps, int interleaved, int32_t* status, attn_stream_t stream) {
  if (!strides) return ATTN_ERR_INVALID_ARG;
  const int64_t dense[9] = {0, strides[0], strides[1], 0, strides[2], strides[3], 0, strides[4], strides[5]};
  NormRopeArgs a;
  const int rc = norm_rope_args(q, k, v, dense, q_weight, k_weight, weight_bf16, cos_table, sin_table, positions, 1,
                                T, Hq, Hkv, d, rotary_dim, max_pos, eps, interleaved, &a);
  if (rc != ATTN_OK) return rc;
  if (!q || !k || !v || !positions || !slots || !q_out || !k_cache || !v_cache || num_blocks <= 0 || block_size <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned4(slots)) return ATTN_ERR_INVALID_ARG;
  if (current_sm_count(&a.sms) != ATTN_OK) return ATTN_ERR_CUDA;
  return launch_norm_rope(a, q_out, k_cache, v_cache, slots, static_cast<long long>(num_blocks) * block_size, status,
                          reinterpret_cast<cudaStream_t>(stream));
}

size_t attn_qk_norm_rope_backward_workspace_bytes(int B, int N, int Hq, int Hkv, int d) {
  if (B <= 0 || N <= 0 || Hq <= 0 || Hkv <= 0 || (d != 64 && d != 128)) return 0;
  int sms = 0;
  if (current_sm_count(&sms) != ATTN_OK) return 0;
  return norm_rope_bwd_workspace(norm_rope_bwd_ctas(static_cast<long long>(B) * N, Hq, Hkv, d, sms), d);
}

int attn_qk_norm_rope_backward(const void* q, const void* k, const int64_t* strides, const void* q_weight,
                               const void* k_weight, int weight_bf16, const float* cos_table, const float* sin_table,
                               const int32_t* positions, const void* d_q, const void* d_k, const void* d_v, void* dq,
                               void* dk, void* dv, const int64_t* grad_strides, float* dq_weight, float* dk_weight,
                               int B, int N, int Hq, int Hkv, int d, int rotary_dim, int max_pos, float eps,
                               int interleaved, void* workspace, size_t workspace_bytes, int32_t* status,
                               attn_stream_t stream) {
  if (!strides || !grad_strides) return ATTN_ERR_INVALID_ARG;
  const int64_t three[9] = {strides[0], strides[1], strides[2], strides[3], strides[4], strides[5], 0, 0, 0};
  NormRopeArgs a;
  const int rc = norm_rope_args(q, k, nullptr, three, q_weight, k_weight, weight_bf16, cos_table, sin_table,
                                positions, B, N, Hq, Hkv, d, rotary_dim, max_pos, eps, interleaved, &a);
  if (rc != ATTN_OK) return rc;
  const bool norm = q_weight != nullptr;
  if (!d_q || !d_k || !d_v || !dq || !dk || !dv) return ATTN_ERR_INVALID_ARG;
  if (norm && (!q || !k || !dq_weight || !dk_weight)) return ATTN_ERR_INVALID_ARG;
  for (const void* p : {d_q, d_k, d_v, (const void*)dq, (const void*)dk, (const void*)dv})
    if (!aligned16(p)) return ATTN_ERR_INVALID_ARG;
  if (!aligned4(dq_weight) || !aligned4(dk_weight)) return ATTN_ERR_INVALID_ARG;
  int64_t sb[3], sn[3], sh[3];
  for (int t = 0; t < 3; ++t) {
    sb[t] = grad_strides[3 * t], sn[t] = grad_strides[3 * t + 1], sh[t] = grad_strides[3 * t + 2];
    if (sb[t] % 8 != 0 || sn[t] % 8 != 0 || sh[t] % 8 != 0) return ATTN_ERR_INVALID_ARG;
  }
  if (current_sm_count(&a.sms) != ATTN_OK) return ATTN_ERR_CUDA;
  const int ctas = norm_rope_bwd_ctas(static_cast<long long>(B) * N, Hq, Hkv, d, a.sms);
  if (norm &&
      (!workspace || !aligned16(workspace) || workspace_bytes < norm_rope_bwd_workspace(ctas, d)))
    return ATTN_ERR_WORKSPACE;
  const void* const dz[3] = {d_q, d_k, d_v};
  void* const dx[3] = {dq, dk, dv};
  return launch_norm_rope_backward(a, dz, dx, sb, sn, sh, dq_weight, dk_weight, static_cast<float*>(workspace), ctas,
                                   status, reinterpret_cast<cudaStream_t>(stream));
}

int attn_paged_gather(const void* cache, const int32_t* block_table, const int32_t* seq_lens, void* out, int B,
                      int Hkv, int d, int num_blocks, int block_size, int max_blocks_per_seq, int max_seq_len,
                      int32_t* status, attn_stream_t stream) {
  if (!cache || !block_table || !seq_lens || !out) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hkv <= 0 || d <= 0 || num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 ||
      max_seq_len <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * block_size < max_seq_len) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(cache) || !aligned16(out)) return ATTN_ERR_INVALID_ARG;
  if (d % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  const cudaError_t e = launch_paged_gather(cache, block_table, seq_lens, out, B, Hkv, d, num_blocks, block_size,
                                            max_blocks_per_seq, max_seq_len, status,
                                            reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
