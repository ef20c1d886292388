// hisa_cache_keep: the rows of each sequence to keep within a budget, by accumulated weight.
//
// Between the first n_first and the last n_recent rows, the K = budget - n_first - n_recent rows
// with the largest weight (ties: the lower row) are kept: an exact selection of the K-th largest key
// by radix, 8 bits a pass from the top, then one counting and one emitting sweep in row order.
//
// A cluster of up to 16 CTAs takes one sequence, a contiguous part of its rows each, so that a single
// long cache is not left to one SM; the first 47K rows of a part stay in shared memory, each sweep reads
// the others again (L2).  A pass counts into 32 copies of the 256 counters, copy =
// lane: the atomics of a warp never meet, whatever the weights' distribution (accumulated weights
// share few exponents, equal ones are frequent).  The CTAs exchange their 256 sums through
// distributed shared memory.  The bound is the sweeps' latency, not the 4 bytes a row.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace hisa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kUnroll = 16;  // keys a thread reads at once
constexpr int kMaxCluster = 16;
constexpr int kStaged = 47 * 1024;  // rows a CTA holds in shared memory

struct Shared {
  uint32_t copies[256][32];  // counters of the running pass, copy = lane
  uint32_t sums[2][256];     // this CTA's sums, of the passes in turn (read by the whole cluster)
  uint32_t totals[256];      // the cluster's
  uint32_t counts[2];        // this CTA's keys above and at the threshold
  uint32_t warp_gt[kWarps], warp_eq[kWarps];
  uint32_t digit, above, at;
};

static_assert(sizeof(Shared) + 4 * kStaged <= 227 * 1024, "shared memory budget");

// Order-preserving key of a weight: every NaN above +inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(__fadd_rn(w, 0.0f));  // -0 + 0 = +0
  return u ^ ((u & 0x80000000u) ? 0xFFFFFFFFu : 0x80000000u);
}

__global__ void __launch_bounds__(kThreads, 1)
    cache_keep_kernel(const float* __restrict__ weight, const int32_t* kv_len, int64_t n_kv, int budget, int n_first,
                      int n_recent, int32_t* __restrict__ keep_idx, int32_t* kept_len, int32_t* __restrict__ status) {
  extern __shared__ uint8_t smem[];
  Shared& sm = *reinterpret_cast<Shared*>(smem);
  uint32_t* held = reinterpret_cast<uint32_t*>(smem + sizeof(Shared));
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t seq = blockIdx.x / nc;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* out = keep_idx + seq * budget;
  int64_t L = kv_len[seq];
  cluster.sync();  // kept_len may be kv_len
  if (L < 0 || L > n_kv) {
    if (rank == 0 && tid == 0 && status) atomicOr(status, kStatusBadIndex);
    L = 0;
  }
  const int kept = (int)min((int64_t)budget, L);
  if (rank == 0 && tid == 0) kept_len[seq] = kept;
  // The rows that need no choice, and the padding.
  const int at = rank * kThreads + tid, step = nc * kThreads;
  for (int64_t j = (int64_t)kept + at; j < budget; j += step) out[j] = -1;
  if (L <= budget) {
    for (int64_t j = at; j < kept; j += step) out[j] = (int32_t)j;
    return;
  }
  for (int64_t j = at; j < n_first; j += step) out[j] = (int32_t)j;
  for (int64_t j = at; j < n_recent; j += step) out[budget - n_recent + j] = (int32_t)(L - n_recent + j);
  const int K = budget - n_first - n_recent;
  if (K == 0) return;

  // This CTA's part [b0, b0 + n) of the rows between.
  const int64_t all = L - n_first - n_recent;
  const int64_t b0 = all * rank / nc;
  const int n = (int)(all * (rank + 1) / nc - b0);
  const float* w = weight + seq * n_kv + n_first + b0;
  const int staged = min(n, kStaged);  // the first rows' keys stay here
  auto key = [&](int i) { return i < staged ? held[i] : weight_key(w[i]); };

  uint32_t prefix = 0, mask = 0, krem = (uint32_t)K;
  bool tie = true;  // of the keys equal to the prefix under the mask the first krem are taken, else all
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < 256 * 32; i += kThreads) (&sm.copies[0][0])[i] = 0;
    __syncthreads();
    if (pass == 0) {
      for (int i0 = 0; i0 < n; i0 += kUnroll * kThreads) {
        float x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int i = i0 + u * kThreads + tid;
          x[u] = i < n ? w[i] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int i = i0 + u * kThreads + tid;
          if (i >= n) continue;
          const uint32_t k = weight_key(x[u]);
          if (i < staged) held[i] = k;
          atomicAdd(&sm.copies[k >> 24][lane], 1u);
        }
      }
    } else {
      for (int i0 = 0; i0 < n; i0 += kUnroll * kThreads) {
        uint32_t x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int i = i0 + u * kThreads + tid;
          x[u] = i < n ? key(i) : ~prefix;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if ((x[u] & mask) == prefix) atomicAdd(&sm.copies[(x[u] >> shift) & 255u][lane], 1u);
      }
    }
    __syncthreads();
    // the copies' sums: a warp takes 8 counters, its lanes their copies
    uint32_t* mine = sm.sums[pass & 1];
#pragma unroll
    for (int b = 0; b < 256 / kWarps; ++b) {
      const int bin = warp * (256 / kWarps) + b;
      const uint32_t c = __reduce_add_sync(0xFFFFFFFFu, sm.copies[bin][lane]);
      if (lane == 0) mine[bin] = c;
    }
    cluster.sync();
    if (tid < 256) {
      uint32_t c[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) c[r] = r < nc ? cluster.map_shared_rank(mine, r)[tid] : 0u;
#pragma unroll
      for (int r = 1; r < kMaxCluster; ++r) c[0] += c[r];
      sm.totals[tid] = c[0];
    }
    __syncthreads();
    if (warp == 0) {
      // digits 255 - 8 lane - b, from the highest; the digit that holds the krem-th largest key
      uint32_t c[8], tot = 0;
#pragma unroll
      for (int b = 0; b < 8; ++b) c[b] = sm.totals[255 - 8 * lane - b];
#pragma unroll
      for (int b = 0; b < 8; ++b) tot += c[b];
      uint32_t incl = tot;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
      }
      uint32_t acc = incl - tot;
      if (acc < krem && krem <= incl) {
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          if (acc < krem && krem <= acc + c[b]) {
            sm.digit = 255u - 8u * lane - b;
            sm.above = acc;
            sm.at = c[b];
          }
          acc += c[b];
        }
      }
    }
    __syncthreads();
    krem -= sm.above;
    prefix |= sm.digit << shift;
    mask |= 255u << shift;
    if (sm.at == krem) {
      tie = false;
      break;
    }
  }

  // Every warp counts, then emits, a contiguous range of the part.
  const int span = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int w0 = min(warp * span, n), w1 = min(w0 + span, n);
  uint32_t gt = 0, eq = 0;
  for (int c0 = w0; c0 < w1; c0 += 256) {
    uint32_t x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = c0 + 32 * u + lane;
      x[u] = i < w1 ? key(i) : 0u;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = c0 + 32 * u + lane < w1;
      gt += in && (x[u] & mask) > prefix;
      eq += in && (x[u] & mask) == prefix;
    }
  }
  gt = __reduce_add_sync(0xFFFFFFFFu, gt);
  eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  if (lane == 0) {
    sm.warp_gt[warp] = gt;
    sm.warp_eq[warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {
    const uint32_t g = __reduce_add_sync(0xFFFFFFFFu, sm.warp_gt[lane]);
    const uint32_t e = __reduce_add_sync(0xFFFFFFFFu, sm.warp_eq[lane]);
    if (lane == 0) {
      sm.counts[0] = g;
      sm.counts[1] = e;
    }
  }
  cluster.sync();
  // keys above and at the threshold in front of this warp's range
  uint32_t above = 0, ties = 0;
  if (lane < rank) {  // rank <= 15
    const uint32_t* theirs = cluster.map_shared_rank(sm.counts, lane);
    above = theirs[0];
    ties = theirs[1];
  }
  above += lane < warp ? sm.warp_gt[lane] : 0u;
  ties += lane < warp ? sm.warp_eq[lane] : 0u;
  above = __reduce_add_sync(0xFFFFFFFFu, above);
  ties = __reduce_add_sync(0xFFFFFFFFu, ties);
  cluster.sync();  // no CTA leaves while its counts are read
  const uint32_t quota = tie ? krem : 0xFFFFFFFFu;
  uint32_t place = n_first + above + min(ties, quota);
  const uint32_t below = (1u << lane) - 1u;
  const int32_t row0 = (int32_t)(n_first + b0);
  for (int c0 = w0; c0 < w1; c0 += 256) {
    uint32_t x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = c0 + 32 * u + lane;
      x[u] = i < w1 ? key(i) : 0u;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = c0 + 32 * u + lane;
      const bool is_eq = i < w1 && (x[u] & mask) == prefix;
      const uint32_t be = __ballot_sync(0xFFFFFFFFu, is_eq);
      const bool take = i < w1 && ((x[u] & mask) > prefix || (is_eq && ties + __popc(be & below) < quota));
      const uint32_t bt = __ballot_sync(0xFFFFFFFFu, take);
      if (take) out[place + __popc(bt & below)] = row0 + i;
      place += __popc(bt);
      ties += __popc(be);
    }
  }
}

}  // namespace

size_t cache_keep_workspace_bytes(const Shape&) { return 0; }

cudaError_t launch_cache_keep(const Shape& s, const float* weight, const int32_t* kv_len, int budget, int n_first,
                              int n_recent, int32_t* keep_idx, int32_t* kept_len, int32_t* status, void*,
                              cudaStream_t st) {
  // CTAs per sequence: as many as leave every CTA 4096 rows or more while the call stays on one wave
  // of the 148 SMs.
  int nc = 1;
  while (nc < kMaxCluster && (int64_t)s.batch * nc * 2 <= 148 && s.n_kv >= (int64_t)nc * 2 * 4096) nc *= 2;
  const int64_t part = (s.n_kv + nc - 1) / nc;
  const size_t smem = sizeof(Shared) + 4 * (size_t)(part < kStaged ? part : kStaged);
  cudaError_t e = ensure_smem((const void*)cache_keep_kernel, (int)(sizeof(Shared) + 4 * (size_t)kStaged));
  if (e != cudaSuccess) return e;
  if (nc > 8) {
    e = cudaFuncSetAttribute(cache_keep_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(s.batch * nc));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)nc;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_keep_kernel, weight, kv_len, s.n_kv, budget, n_first, n_recent, keep_idx,
                            kept_len, status);
}

}  // namespace hisa
