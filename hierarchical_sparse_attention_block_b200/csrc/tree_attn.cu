// hisa_tree_attn_fwd: attention of drafted tokens over a cache.
#include <math.h>

#include "common.cuh"
#include "draft_tree.cuh"
#include "internal.h"

namespace hisa {
namespace {

constexpr int kThreads = 256;

// One CTA per (slot, head, sequence): warps take keys in turn with an online softmax each, merged at the end.
template <int D>
__global__ void __launch_bounds__(kThreads)
    tree_attn_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                     const __nv_bfloat16* __restrict__ v, const int32_t* __restrict__ kv_len,
                     const int32_t* __restrict__ parent, __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                     int32_t* __restrict__ status, int T, int64_t n_kv, int H, int Hkv, float scale) {
  constexpr int NW = kThreads / 32, E = D / 32;
  __shared__ DraftTree tree;
  __shared__ float sm_m[NW], sm_l[NW], sm_o[NW][D];
  const int i = blockIdx.x, h = blockIdx.y, g = h / (H / Hkv);
  const int64_t seq = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t L = context_len(kv_len, seq, T, n_kv);
  bool bad = draft_tree_build<kThreads>(tree, parent ? parent + seq * T : nullptr, T, tid, [] { __syncthreads(); });
  bad = bad || L < 0;
  if (bad && status) atomicOr(status, kStatusBadIndex);
  const int64_t row = (seq * T + i) * H + h;
  const bool token = L >= 0 && tree.up[i] == kRoot;
  float qf[E], acc[E];
  for (int e = 0; e < E; ++e) {
    qf[e] = __bfloat162float(q[row * D + lane + 32 * e]) * scale;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  if (token) {
    for (int64_t t = warp; t < L + T; t += NW) {
      if (t >= L && !((tree.anc[i][(t - L) >> 5] >> ((t - L) & 31)) & 1u)) continue;
      const int64_t at = ((seq * n_kv + t) * Hkv + g) * D + lane;
      float z = 0.f;
      for (int e = 0; e < E; ++e) z += qf[e] * __bfloat162float(k[at + 32 * e]);
      z = warp_sum(z);
      const float mn = fmaxf(m, z);
      const float a = m == -INFINITY ? 0.f : __expf(m - mn), p = z == -INFINITY ? 0.f : __expf(z - mn);
      m = mn;
      l = l * a + p;
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + p * __bfloat162float(v[at + 32 * e]);
    }
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
  for (int e = 0; e < E; ++e) sm_o[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  if (tid >= D) return;
  float M = -INFINITY, sum = 0.f, out = 0.f;
  for (int w = 0; w < NW; ++w) M = fmaxf(M, sm_m[w]);
  for (int w = 0; w < NW; ++w) {
    const float a = sm_m[w] == -INFINITY ? 0.f : __expf(sm_m[w] - M);
    sum += sm_l[w] * a;
    out += sm_o[w][tid] * a;
  }
  o[row * D + tid] = __float2bfloat16(sum == 0.f ? 0.f : out / sum);
  if (tid == 0 && lse) lse[row] = sum == 0.f ? -INFINITY : M + logf(sum);
}

}  // namespace

size_t tree_attn_workspace_bytes(const Shape& s, bool with_weight) {
  return with_weight ? (size_t)s.batch * s.n_q * s.H * sizeof(float) : 0;
}

cudaError_t launch_tree_attn(const Shape& s, const void* q, const void* k, const void* v, const int32_t* kv_len,
                             const int32_t* parent, void* o, float* lse, float* weight, int32_t* status, void* ws,
                             cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (weight && !lse) lse = static_cast<float*>(ws);
  const dim3 grid((unsigned)s.n_q, (unsigned)s.H, (unsigned)s.batch);
  const auto kern = s.d == 64 ? tree_attn_kernel<64> : tree_attn_kernel<128>;
  kern<<<grid, kThreads, 0, st>>>(static_cast<const bf*>(q), static_cast<const bf*>(k), static_cast<const bf*>(v),
                                  kv_len, parent, static_cast<bf*>(o), lse, status, (int)s.n_q, s.n_kv, s.H, s.Hkv,
                                  s.scale);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !weight) return e;
  return launch_cache_weight(s, q, k, kv_len, parent, nullptr, lse, weight, nullptr, nullptr, st);
}

}  // namespace hisa
