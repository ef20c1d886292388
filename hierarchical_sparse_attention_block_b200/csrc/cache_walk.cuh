// How the kernels over a cache share their work: every key tile of every item (a part of one
// sequence's work that reads all its key tiles) is a unit, the units lie in the order sequence, item,
// key tile, and CTA c takes the c-th of equal contiguous ranges.  The ranges follow from the lengths
// on the device, so ragged caches balance and one long cache covers every SM.  An item starts with a few
// units more that hold no tile: what it costs a CTA to go over to another item (its query rows, the
// products' start and end), so that a CTA with the ends of two items gets fewer tiles.
#pragma once

#include "common.cuh"
#include "draft_tree.cuh"

namespace hisa {

constexpr int kTileKeys = 128;  // cache rows per key tile
constexpr int kMaxCtas = 148;   // one CTA per SM

__device__ __forceinline__ int64_t key_tiles(int64_t L, int T) {
  return L < 0 ? 0 : (L + T + kTileKeys - 1) / kTileKeys;
}

// CTA c of `ctas` takes the units [range_begin(c), range_begin(c + 1)), at least one each: with fewer
// units than CTAs the CTAs behind the last unit take none.
__device__ __forceinline__ int64_t range_ctas(int64_t units, int64_t grid) { return units < grid ? units : grid; }
__device__ __forceinline__ int64_t range_begin(int64_t c, int64_t units, int64_t ctas) { return c * units / ctas; }
// The CTA whose range holds unit u.
__device__ __forceinline__ int64_t range_of(int64_t u, int64_t units, int64_t ctas) {
  return ((u + 1) * ctas - 1) / units;
}

// One CTA's walk through its range, in segments: consecutive key tiles of one item.
struct Walk {
  const int32_t* kv_len;
  int64_t n_kv, u, u1, first;  // first: the range's begin
  int64_t P;                   // units per item of the sequences before s, summed
  int64_t L, tiles;
  int64_t L_next;              // of sequence s + 1: its load is long over when the walk gets there
  int s, T, per_seq, batch;    // per_seq: items of a sequence
  int lead;                    // units without a tile in front of an item
  // the segment: key tiles [j0, j0 + n) of the item
  int item, j0, n;
  int64_t start;

  __device__ int64_t length() const { return tiles > 0 ? tiles + lead : 0; }  // units of an item
  __device__ void at(int seq, int64_t len) {
    s = seq;
    L = len;
    tiles = key_tiles(L, T);
    if (seq + 1 < batch) L_next = context_len(kv_len, seq + 1, T, n_kv);
  }
  __device__ bool next() {
    do {
      if (u >= u1) return false;
      while (u >= (P + length()) * per_seq) {
        P += length();
        at(s + 1, L_next);
      }
      const int64_t rel = u - P * per_seq;
      item = (int)(rel / length());
      const int64_t from = rel - item * length(), to = min(length(), from + (u1 - u));
      j0 = (int)max((int64_t)0, from - lead);
      n = (int)max((int64_t)0, to - lead) - j0;
      start = u;
      u += to - from;
    } while (n == 0);
    return true;
  }
  __device__ bool whole() const { return j0 == 0 && n == tiles; }
  // Which of the CTA's segments that are not whole this one is: the range's first, or its last.
  __device__ int slot() const { return start == first ? 0 : 1; }
};

template <int NT>
struct WalkShared {
  int64_t sums[NT / 32], found[2];
};

// Key tiles (low 44 bits) and sequences that have any (high 20 bits), as one number to be summed.
__device__ __forceinline__ int64_t tile_sum(int64_t L, int T) {
  const int64_t n = key_tiles(L, T);
  return n | (n > 0 ? (int64_t)1 << 44 : 0);
}
__device__ __forceinline__ int64_t tiles_of(int64_t sum) { return sum & (((int64_t)1 << 44) - 1); }
__device__ __forceinline__ int64_t units_of(int64_t sum, int lead) { return tiles_of(sum) + lead * (sum >> 44); }

// The CTA's walk; all NT threads call, two barriers.  lead: units without a tile in front of an item, where the
// call has a tile for each SM (else none).  us without them and with them, by tiles a CTA, in a replayed graph:
//   4 x n rows, 16 heads on 4, 32 tokens, d = 128:    0.6: 24.1, 22.9   1.4: 35.2, 29.0   3: 37.2, 31.1   12: 51, 46
//   4 x n rows, 16 heads on 2, 64 tokens, d = 128:    0.6: 31.0, 33.5   1.4: 47.3, 37.2   3: 51.4, 41.2   12: 78, 63
//   4 x n rows, 8 heads on 4, one token, d = 64:      0.6: 16.9, 17.2   1.4: 21.0, 19.5   3: 24.9, 23.9   12: 38, 38
//   received weight, 16 heads on 4, 32 tokens:        0.6: 16.8, 18.6   1.4: 23.3, 20.7   3: 24.3, 22.5   12: 33, 32
// prefix (nullable, [batch + 2]): CTA 0 writes the units per item of the sequences before each, of all, and the
// lead; it also flags lengths out of range.
template <int NT>
__device__ Walk walk_begin(const int32_t* kv_len, int64_t n_kv, int T, int batch, int per_seq, int lead,
                           WalkShared<NT>& sm, int64_t* prefix, int32_t* status) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // every thread counts the key tiles of a run of sequences
  const int run = (batch + NT - 1) / NT;
  const int s0 = min(tid * run, batch), s1 = min(s0 + run, batch);
  int64_t mine = 0;
  bool bad = false;
  for (int s = s0; s < s1; ++s) {
    const int64_t L = context_len(kv_len, s, T, n_kv);
    bad = bad || L < 0;
    mine += tile_sum(L, T);
  }
  if (bad && status && blockIdx.x == 0) atomicOr(status, kStatusBadIndex);
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) sm.sums[warp] = incl;
  __syncthreads();
  int64_t before_sum = incl - mine, total_sum = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const int64_t x = sm.sums[w];
    if (w < warp) before_sum += x;
    total_sum += x;
  }
  if (tiles_of(total_sum) * per_seq < kMaxCtas) lead = 0;
  const int64_t before = units_of(before_sum, lead), total = units_of(total_sum, lead);
  const int64_t units = total * per_seq, ctas = range_ctas(units, gridDim.x);
  const bool busy = blockIdx.x < ctas;
  Walk walk;
  walk.kv_len = kv_len;
  walk.n_kv = n_kv;
  walk.T = T;
  walk.per_seq = per_seq;
  walk.batch = batch;
  walk.lead = lead;
  walk.u = walk.first = busy ? range_begin(blockIdx.x, units, ctas) : 0;
  walk.u1 = busy ? range_begin(blockIdx.x + 1, units, ctas) : 0;
  if (busy && walk.u >= before * per_seq && walk.u < (before + units_of(mine, lead)) * per_seq) {
    int64_t P = before;
    for (int s = s0; s < s1; ++s) {
      const int64_t n = units_of(tile_sum(context_len(kv_len, s, T, n_kv), T), lead);
      if (walk.u < (P + n) * per_seq) {
        sm.found[0] = s;
        sm.found[1] = P;
        break;
      }
      P += n;
    }
  }
  if (prefix && blockIdx.x == 0) {
    int64_t P = before;
    for (int s = s0; s < s1; ++s) {
      prefix[s] = P;
      P += units_of(tile_sum(context_len(kv_len, s, T, n_kv), T), lead);
    }
    if (tid == 0) {
      prefix[batch] = total;
      prefix[batch + 1] = lead;
    }
  }
  __syncthreads();
  if (busy) {
    walk.P = sm.found[1];
    walk.at((int)sm.found[0], context_len(kv_len, (int)sm.found[0], T, n_kv));
  }
  return walk;
}

// 32 bits of a tail tile's mask: keys off .. off + 31 relative to the context's end.
__device__ __forceinline__ uint32_t mask_word(const uint32_t* anc, int off) {
  if (off <= -32) return 0xFFFFFFFFu;
  if (off >= kMaxDraft) return 0u;
  if (off < 0) return (anc[0] << -off) | ((1u << -off) - 1u);
  const int w = off >> 5, sh = off & 31;
  const uint32_t lo = anc[w], hi = w + 1 < kDraftWords ? anc[w + 1] : 0u;
  return __funnelshift_r(lo, hi, sh);
}
// The same for a chain: slot i sees the keys off <= i.
__device__ __forceinline__ uint32_t chain_word(int i, int off) {
  const int n = i - off + 1;  // visible keys of the word
  return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}

// A launch that may be scheduled while the kernel before it drains; that kernel's results are
// waited for inside (griddepcontrol.wait).
template <class... P, class... A>
inline cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, cudaStream_t st, int smem, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace hisa
