// hisa_cache_keep: the rows of each sequence to keep within a budget, by accumulated weight.
#include "common.cuh"
#include "internal.h"
#include "select.cuh"

namespace hisa {
namespace {

constexpr int kThreads = 1024;

// Order-preserving key of a weight: every NaN above +inf.  No weight's key is 0 (the selection's empty mark).
__device__ __forceinline__ uint32_t weight_key(float w) { return w == w ? score_key(w) : 0xFFFFFFFFu; }

__global__ void __launch_bounds__(kThreads)
    cache_keep_kernel(const float* __restrict__ weight, const int32_t* kv_len, int64_t n_kv, int budget, int n_first,
                      int n_recent, int32_t* __restrict__ keep_idx, int32_t* kept_len, int32_t* __restrict__ status) {
  __shared__ SelectShared<kThreads> sm;
  const int64_t seq = blockIdx.x;
  int32_t* out = keep_idx + seq * budget;
  int64_t L = kv_len[seq];
  __syncthreads();  // kept_len may be kv_len
  if (L < 0 || L > n_kv) {
    if (threadIdx.x == 0 && status) atomicOr(status, kStatusBadIndex);
    L = 0;
  }
  const int kept = (int)min((int64_t)budget, L);
  if (threadIdx.x == 0) kept_len[seq] = kept;
  for (int j = kept + threadIdx.x; j < budget; j += kThreads) out[j] = -1;
  if (L <= budget) {
    for (int j = threadIdx.x; j < kept; j += kThreads) out[j] = j;
    return;
  }
  for (int j = threadIdx.x; j < n_first; j += kThreads) out[j] = j;
  for (int j = threadIdx.x; j < n_recent; j += kThreads) out[budget - n_recent + j] = (int32_t)(L - n_recent + j);
  const int K = budget - n_first - n_recent;
  if (K == 0) return;
  const int n = (int)(L - n_first - n_recent);
  const float* w = weight + seq * n_kv + n_first;
  auto key = [&](int i) { return weight_key(w[i]); };
  const SelectResult sel = radix_select<kThreads>(key, n, K, sm);
  emit_selected<kThreads>(key, n, sel, sm, [&](int i, int rank) { out[n_first + rank] = n_first + i; });
}

}  // namespace

size_t cache_keep_workspace_bytes(const Shape&) { return 0; }

cudaError_t launch_cache_keep(const Shape& s, const float* weight, const int32_t* kv_len, int budget, int n_first,
                              int n_recent, int32_t* keep_idx, int32_t* kept_len, int32_t* status, void*,
                              cudaStream_t st) {
  cache_keep_kernel<<<(unsigned)s.batch, kThreads, 0, st>>>(weight, kv_len, s.n_kv, budget, n_first, n_recent,
                                                            keep_idx, kept_len, status);
  return cudaGetLastError();
}

}  // namespace hisa
