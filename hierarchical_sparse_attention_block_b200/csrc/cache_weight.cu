// hisa_cache_weight: the attention weight each cached row receives.
#include <math.h>

#include "common.cuh"
#include "draft_tree.cuh"
#include "internal.h"

namespace hisa {
namespace {

constexpr int kThreads = 256;

// One warp per cache row: sum over heads and counted slots of exp(z - lse).
template <int D>
__global__ void __launch_bounds__(kThreads)
    cache_weight_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                        const int32_t* __restrict__ kv_len, const int32_t* __restrict__ parent,
                        const int32_t* __restrict__ path, const float* __restrict__ lse, float* __restrict__ weight,
                        int32_t* __restrict__ status, int T, int64_t n_kv, int H, int Hkv, float scale) {
  constexpr int NW = kThreads / 32, E = D / 32;
  __shared__ DraftTree tree;
  __shared__ uint32_t counted[kDraftWords];
  const int64_t seq = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t L = context_len(kv_len, seq, T, n_kv);
  bool bad = draft_tree_build<kThreads>(tree, parent ? parent + seq * T : nullptr, T, tid, [] { __syncthreads(); });
  if (tid < kDraftWords) counted[tid] = path ? 0u : 0xFFFFFFFFu;
  __syncthreads();
  if (path && tid == 0) {
    int last = -1;
    for (int j = 0; j < T; ++j) {
      const int p = path[seq * T + j];
      if (p == -1) continue;
      if (p <= last || p >= T) {
        bad = true;
        continue;
      }
      last = p;
      counted[p >> 5] |= 1u << (p & 31);
    }
  }
  __syncthreads();
  bad = bad || L < 0;
  if (bad && status) atomicOr(status, kStatusBadIndex);
  if (L < 0) return;
  for (int64_t t = (int64_t)blockIdx.x * NW + warp; t < L + T; t += (int64_t)gridDim.x * NW) {
    float sum = 0.f;
    for (int g = 0; g < Hkv; ++g) {
      float kf[E];
      for (int e = 0; e < E; ++e)
        kf[e] = __bfloat162float(k[((seq * n_kv + t) * Hkv + g) * D + lane + 32 * e]) * scale;
      for (int i = 0; i < T; ++i) {
        if (tree.up[i] != kRoot || !((counted[i >> 5] >> (i & 31)) & 1u)) continue;
        if (t >= L && !((tree.anc[i][(t - L) >> 5] >> ((t - L) & 31)) & 1u)) continue;
        for (int h = g * (H / Hkv); h < (g + 1) * (H / Hkv); ++h) {
          const int64_t row = (seq * T + i) * H + h;
          float z = 0.f;
          for (int e = 0; e < E; ++e) z += kf[e] * __bfloat162float(q[row * D + lane + 32 * e]);
          z = warp_sum(z);
          if (lse[row] != -INFINITY) sum += expf(z - lse[row]);
        }
      }
    }
    if (lane == 0) weight[seq * n_kv + t] = t < L ? weight[seq * n_kv + t] + sum : sum;
  }
}

}  // namespace

size_t cache_weight_workspace_bytes(const Shape&) { return 0; }

cudaError_t launch_cache_weight(const Shape& s, const void* q, const void* k, const int32_t* kv_len,
                                const int32_t* parent, const int32_t* path, const float* lse, float* weight,
                                int32_t* status, void*, cudaStream_t st) {
  using bf = __nv_bfloat16;
  const int64_t want = (s.n_kv + 7) / 8;
  const dim3 grid((unsigned)(want < 4096 ? want : 4096), (unsigned)s.batch);
  const auto kern = s.d == 64 ? cache_weight_kernel<64> : cache_weight_kernel<128>;
  kern<<<grid, kThreads, 0, st>>>(static_cast<const bf*>(q), static_cast<const bf*>(k), kv_len, parent, path, lse,
                                  weight, status, (int)s.n_q, s.n_kv, s.H, s.Hkv, s.scale);
  return cudaGetLastError();
}

}  // namespace hisa
