// hisa_cache_keep: the rows of each sequence to keep within a budget, by accumulated weight.
//
// Between the first n_first and the last n_recent rows, the K = budget - n_first - n_recent rows
// with the largest weight (ties: the lower row) are kept: an exact selection of the K-th largest key
// by radix, 8 bits a pass from the top, and a sweep that emits the taken rows in order.
//
// A cluster of up to 16 CTAs takes one sequence, a contiguous part of its rows each, so that a single
// long cache is not left to one SM, and for a few very long ones a cooperative grid shares the whole GPU
// among them (their counters then meet in the workspace); the first 46K keys of a part stay in shared
// memory, each sweep reads the others again (L2).  A pass counts into 32 copies of the 256 counters, copy = lane: the
// atomics of a warp never meet, whatever the weights' distribution (accumulated weights share few
// exponents, equal ones are frequent).  The CTAs exchange their 256 sums through distributed shared
// memory.  Two passes fix 16 bits of the threshold; where few keys share them (the usual case), one
// more sweep counts the keys above and collects those few, and the last two passes and the split of
// the ties work on them alone; else they are sweeps too.  Keys are read four at a time: the bound is
// the number of instructions a key and the cluster's barriers, not the 4 bytes a row.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace hisa {
namespace {

namespace cg = cooperative_groups;
using tc::global_ns;
using tc::kStatusTimeout;
using tc::kWaitNs;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kClusters16 = 7;      // clusters of 16 CTAs of an SM each that run at a time
constexpr int kStaged = 46 * 1024;  // keys a CTA holds in shared memory
constexpr int kFew = 1024;          // keys of the cluster that are collected
// A cooperative grid takes sequences from kWideRows rows on that get kMinWide CTAs or more, of kWidePart rows
// at least.  Its barriers and the counters in global memory cost about 8 us more than a cluster's: 1 x 256K rows
// 21.9 us against 20.3; 1 x 512K 24.6 against 28; 1 x 1M 31 against 47; 1 x 8M 69 against 415; 4 x 2M 52 against
// 106.  With parts of 8192 rows 1 x 1M takes 39 us: the counters' atomics of 122 CTAs meet.
constexpr int64_t kWideRows = 524288, kWidePart = 16384;
constexpr int kMinWide = 16;

struct alignas(16) Shared {
  uint32_t copies[256][32];  // counters of the running pass, copy = lane
  uint32_t sums[2][256];     // this CTA's sums, of the passes in turn (read by the whole cluster)
  uint32_t totals[256];      // the cluster's
  uint32_t counts[2];        // this CTA's keys above and at the threshold
  uint32_t warp_gt[kWarps], warp_eq[kWarps];
  uint32_t digit, above, at;
  uint32_t n_few;             // collected keys of this CTA
  uint32_t few_key[kFew];
  uint16_t few_warp[kFew];    // the warp whose range the key lies in
};
static_assert(sizeof(Shared) + 4 * kStaged <= 227 * 1024, "shared memory budget");

// Order-preserving key of a weight: every NaN above +inf.  No weight's key is 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(__fadd_rn(w, 0.0f));  // -0 + 0 = +0
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return w != w ? 0xFFFFFFFFu : k;
}

// Adds 1 to a shared counter where `hit` holds, without a branch.
__device__ __forceinline__ void count_if(bool hit, uint32_t counter) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %0, 0;\n @p red.shared.add.u32 [%1], 1;\n}\n" ::"r"((uint32_t)hit),
               "r"(counter)
               : "memory");
}

// What the CTAs of one sequence share where they are no cluster.
struct Global {
  uint32_t totals[4][256];  // a pass's counters
  uint32_t arrived;         // CTAs at the barriers so far
  uint32_t counts[][2];     // [CTA] keys above and at the threshold
};
__host__ __device__ constexpr size_t global_bytes(int nc) { return sizeof(uint32_t) * (4 * 256 + 1 + 2 * (size_t)nc); }

// WIDE: nc CTAs of a cooperative grid share a sequence, else a cluster.
template <bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    cache_keep_kernel(const float* __restrict__ weight, const int32_t* kv_len, int64_t n_kv, int budget, int n_first,
                      int n_recent, int32_t* __restrict__ keep_idx, int32_t* kept_len, int32_t* __restrict__ status,
                      int nc, uint8_t* ws) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sm = *reinterpret_cast<Shared*>(smem);
  uint4* held = reinterpret_cast<uint4*>(smem + sizeof(Shared));
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)blockIdx.x % nc;  // a cluster's CTAs follow one another
  const int64_t seq = blockIdx.x / nc;
  Global* const global = WIDE ? reinterpret_cast<Global*>(ws + seq * global_bytes(nc)) : nullptr;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // A barrier of the sequence's CTAs.  A cooperative grid's CTAs are all there, so its wait ends; should one not
  // come within a second, the others stop too.
  uint32_t due = 0;
  auto sync = [&]() {
    if constexpr (WIDE) {
      __shared__ int gone;
      due += (uint32_t)nc;
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        atomicAdd(&global->arrived, 1u);
        const uint64_t t0 = global_ns();
        uint32_t n;
        do {
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(&global->arrived) : "memory");
        } while (n < due && global_ns() - t0 < kWaitNs);
        gone = n < due;
        if (gone && status) atomicOr(status, kStatusTimeout);
      }
      __syncthreads();
      return gone == 0;
    } else {
      cluster.sync();
      return true;
    }
  };
  int32_t* out = keep_idx + seq * budget;
  int64_t L = kv_len[seq];
  for (int i = tid; i < 256 * 32 / 4; i += kThreads) reinterpret_cast<uint4*>(sm.copies)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) sm.n_few = 0;
  if (tid < kWarps) sm.warp_gt[tid] = sm.warp_eq[tid] = 0;
  if constexpr (WIDE) {
    if (rank == 0) (&global->totals[0][0])[tid] = 0;
    if (rank == 0 && tid == 0) global->arrived = 0;
    cg::this_grid().sync();
  } else {
    cluster.sync();  // kept_len may be kv_len
  }
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

  // The rows between, in groups of four from a 16-byte boundary at or before the first; this CTA has the
  // groups [0, n) of its part.  Rows outside the range get key 0, which is never taken.
  const float* row = weight + seq * n_kv;
  const int lead = (int)((reinterpret_cast<uintptr_t>(row + n_first) >> 2) & 3);
  const int64_t begin = n_first - lead, end = L - n_recent;
  const int64_t groups = (end - begin + 3) / 4, g0 = groups * rank / nc;
  const int n = (int)(groups * (rank + 1) / nc - g0);
  const int64_t t0 = begin + 4 * g0;  // row of the part's first key
  const int staged = min(n, kStaged / 4);
  auto fetch = [&](int q) {  // keys of group q
    const int64_t t = t0 + 4 * (int64_t)q;
    if (t >= n_first && t + 4 <= end) {
      const float4 w = *reinterpret_cast<const float4*>(row + t);
      return make_uint4(weight_key(w.x), weight_key(w.y), weight_key(w.z), weight_key(w.w));
    }
    uint32_t k[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) k[i] = t + i >= n_first && t + i < end ? weight_key(row[t + i]) : 0u;
    return make_uint4(k[0], k[1], k[2], k[3]);
  };
  auto keys = [&](int q) { return q < staged ? held[q] : fetch(q); };
  // Every warp has a contiguous range of groups in the sweeps that keep the order.
  const int span = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int q0 = min(warp * span, n), q1 = min(q0 + span, n);

  uint32_t prefix = 0, mask = 0, krem = (uint32_t)K;
  bool tie = true;   // of the keys equal to the prefix under the mask the first krem are taken, else all
  bool few = false;  // the keys that match 16 bits of the threshold are collected
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    const uint32_t mine_at = (uint32_t)__cvta_generic_to_shared(&sm.copies[0][lane]);
    auto count = [&](uint32_t k) { count_if((k & mask) == prefix, mine_at + ((k >> shift) & 255u) * 128u); };
    if (pass == 0) {
      for (int c0 = 0; c0 < n; c0 += 4 * kThreads) {
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int q = c0 + u * kThreads + tid;
          if (q < n) x[u] = fetch(q);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int q = c0 + u * kThreads + tid;
          if (q >= n) continue;
          if (q < staged) held[q] = x[u];
          count(x[u].x);
          count(x[u].y);
          count(x[u].z);
          count(x[u].w);
        }
      }
    } else if (few) {
      for (int i = tid; i < (int)sm.n_few; i += kThreads) count(sm.few_key[i]);
    } else {
      auto four = [&](uint4 x) {
        count(x.x);
        count(x.y);
        count(x.z);
        count(x.w);
      };
#pragma unroll 4
      for (int q = tid; q < staged; q += kThreads) four(held[q]);
      for (int c0 = staged; c0 < n; c0 += 4 * kThreads) {
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int q = c0 + u * kThreads + tid;
          x[u] = q < n ? fetch(q) : make_uint4(0u, 0u, 0u, 0u);  // (0 may match only where no key is taken)
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) four(x[u]);
      }
    }
    __syncthreads();
    // the copies' sums: a warp takes 8 counters, its lanes their copies, which are then free again
    uint32_t* mine = sm.sums[pass & 1];
#pragma unroll
    for (int b = 0; b < 256 / kWarps; ++b) {
      const int bin = warp * (256 / kWarps) + b;
      const uint32_t c = __reduce_add_sync(0xFFFFFFFFu, sm.copies[bin][lane]);
      sm.copies[bin][lane] = 0;
      if (lane != 0) continue;
      if (!WIDE)
        mine[bin] = c;
      else if (c != 0)
        atomicAdd(&global->totals[pass][bin], c);
    }
    if (!sync()) return;
    if (WIDE) {
      if (tid < 256) sm.totals[tid] = __ldcg(&global->totals[pass][tid]);
    } else if (tid < 256) {
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
    if (pass == 1 && sm.at <= kFew) {
      // few keys share the 16 bits: count what lies above, collect them
      few = true;
      uint32_t gt = 0;
      for (int c0 = q0; c0 < q1; c0 += 128) {
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int q = c0 + 32 * u + lane;
          x[u] = q < q1 ? keys(q) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t k[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          bool hit = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            gt += (k[i] & mask) > prefix;
            hit |= (k[i] & mask) == prefix;
          }
          if (hit) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if ((k[i] & mask) == prefix && k[i] != 0u) {
                const uint32_t p = atomicAdd(&sm.n_few, 1u);
                sm.few_key[p] = k[i];
                sm.few_warp[p] = (uint16_t)warp;
              }
            }
          }
        }
      }
      gt = __reduce_add_sync(0xFFFFFFFFu, gt);
      if (lane == 0) sm.warp_gt[warp] = gt;
      __syncthreads();
    }
  }

  // What every warp's range holds above and at the threshold.
  if (few) {
    for (int i = tid; i < (int)sm.n_few; i += kThreads) {
      const uint32_t k = sm.few_key[i] & mask;
      if (k > prefix) atomicAdd(&sm.warp_gt[sm.few_warp[i]], 1u);
      if (k == prefix) atomicAdd(&sm.warp_eq[sm.few_warp[i]], 1u);
    }
  } else {
    uint32_t gt = 0, eq = 0;
    for (int c0 = q0; c0 < q1; c0 += 128) {
      uint4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int q = c0 + 32 * u + lane;
        x[u] = q < q1 ? keys(q) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t k[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          gt += (k[i] & mask) > prefix;
          eq += (k[i] & mask) == prefix && k[i] != 0u;
        }
      }
    }
    gt = __reduce_add_sync(0xFFFFFFFFu, gt);
    eq = __reduce_add_sync(0xFFFFFFFFu, eq);
    if (lane == 0) {
      sm.warp_gt[warp] = gt;
      sm.warp_eq[warp] = eq;
    }
  }
  __syncthreads();
  if (warp == 0) {
    const uint32_t g = __reduce_add_sync(0xFFFFFFFFu, sm.warp_gt[lane]);
    const uint32_t e = __reduce_add_sync(0xFFFFFFFFu, sm.warp_eq[lane]);
    if (lane == 0) {
      uint32_t* counts = WIDE ? global->counts[rank] : sm.counts;
      counts[0] = g;
      counts[1] = e;
    }
  }
  if (!sync()) return;
  // keys above and at the threshold in front of this warp's range
  uint32_t above = 0, ties = 0;
  for (int r = lane; r < rank; r += 32) {
    if (WIDE) {
      above += __ldcg(&global->counts[r][0]);
      ties += __ldcg(&global->counts[r][1]);
    } else {  // r <= 15
      const uint32_t* theirs = cluster.map_shared_rank(sm.counts, r);
      above = theirs[0];
      ties = theirs[1];
    }
  }
  above += lane < warp ? sm.warp_gt[lane] : 0u;
  ties += lane < warp ? sm.warp_eq[lane] : 0u;
  above = __reduce_add_sync(0xFFFFFFFFu, above);
  ties = __reduce_add_sync(0xFFFFFFFFu, ties);
  if (!WIDE) cluster.sync();  // no CTA leaves while its counts are read
  const uint32_t quota = tie ? krem : 0xFFFFFFFFu;
  uint32_t place = n_first + above + min(ties, quota);
  const uint32_t below = (1u << lane) - 1u;
  for (int c0 = q0; c0 < q1; c0 += 64) {
    uint4 x[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int q = c0 + 32 * u + lane;
      x[u] = q < q1 ? keys(q) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t k[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      bool take[4];
      bool eq[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        take[i] = (k[i] & mask) > prefix;
        eq[i] = (k[i] & mask) == prefix && k[i] != 0u;
      }
      if (__any_sync(0xFFFFFFFFu, eq[0] | eq[1] | eq[2] | eq[3])) {
        // keys at the threshold, in row order: lane by lane, four a lane
        uint32_t before = 0, total = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t b = __ballot_sync(0xFFFFFFFFu, eq[i]);
          before += __popc(b & below);
          total += __popc(b);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!eq[i]) continue;
          take[i] = ties + before < quota;
          ++before;
        }
        ties += total;
      }
      uint32_t p = place, total = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = __ballot_sync(0xFFFFFFFFu, take[i]);
        p += __popc(b & below);
        total += __popc(b);
      }
      const int32_t t = (int32_t)(t0 + 4 * (int64_t)(c0 + 32 * u + lane));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (take[i]) out[p++] = t + i;
      place += total;
    }
  }
}

// CTAs of a cooperative grid per sequence, or 0 where a cluster takes it.
int wide_ctas(const Shape& s) {
  const int64_t nc = std::min<int64_t>(148 / s.batch, s.n_kv / kWidePart);
  return s.n_kv >= kWideRows && nc >= kMinWide ? (int)nc : 0;
}

}  // namespace

size_t cache_keep_workspace_bytes(const Shape& s) {
  const int nc = wide_ctas(s);
  return nc > 0 ? (size_t)s.batch * global_bytes(nc) : 0;
}

cudaError_t launch_cache_keep(const Shape& s, const float* weight, const int32_t* kv_len, int budget, int n_first,
                              int n_recent, int32_t* keep_idx, int32_t* kept_len, int32_t* status, void* ws,
                              cudaStream_t st) {
  const int wide = wide_ctas(s);
  int nc = wide;
  if (wide == 0) {
    // Clusters: as many CTAs as leave every one 4096 rows or more while the call stays on one wave of the SMs
    // (1 x 16K rows: 12.6 us with 4 CTAs, 16.1 with one; 8 x 64K: 14.4 with 8); 16 only for 8192 rows each and
    // where so many clusters run at a time (6 x 64K: 17.1 us with 16, 15.1 with 8; 6 x 256K: 21 and 25;
    // 8 x 256K: 34 in two waves, 25 with 8).
    nc = 1;
    while (nc < kMaxCluster / 2 && (int64_t)s.batch * nc * 2 <= 148 && s.n_kv >= (int64_t)nc * 2 * 4096) nc *= 2;
    if (nc == kMaxCluster / 2 && s.batch <= kClusters16 && s.n_kv >= kMaxCluster * 8192) nc = kMaxCluster;
  }
  const int64_t part = (s.n_kv + 3 + nc - 1) / nc + 4;  // keys of a part at the most: whole groups of four
  const size_t smem = sizeof(Shared) + 4 * (size_t)(part < kStaged ? (part + 3) / 4 * 4 : kStaged);
  const auto kern = wide > 0 ? cache_keep_kernel<true> : cache_keep_kernel<false>;
  cudaError_t e = ensure_smem((const void*)kern, (int)(sizeof(Shared) + 4 * (size_t)kStaged));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  if (wide > 0) {
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
  } else {
    if (nc > 8) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)nc;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(s.batch * nc));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, weight, kv_len, s.n_kv, budget, n_first, n_recent, keep_idx, kept_len, status,
                            nc, static_cast<uint8_t*>(ws));
}

}  // namespace hisa
