// What the two kernels of hisa_tree_attn_fwd share.
#pragma once

#include "attn_math.cuh"
#include "cache_walk.cuh"
#include "common.cuh"
#include "draft_tree.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace hisa {

constexpr int kRows = kTileKeys;    // query rows per tile = keys per key tile
constexpr int kHalf = kRows * 128;  // 64 columns of 128 rows of 16-bit values: one 128-byte swizzle span
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;

// What the CTAs share with the merge: the unit ranges and the partial results.
struct Work {
  int64_t* prefix;  // [b + 2] units per item of the sequences before, of all, units in front of an item's tiles
  float4* part_o;   // [cta][2][D / 4][rows of an item]: four columns of a row; neighbours are rows
  float2* part_ml;  // [cta][2][rows of an item]: max (log2 domain), sum; (+inf, 0): the row's slot is empty
};

// The call's tensors and shape.
struct TreeArgs {
  const uint16_t* q;
  const uint16_t* v;
  const int32_t* kv_len;
  const int32_t* parent;  // nullable: a chain
  uint16_t* o;
  float* lse;     // nullable
  float* scores;  // nullable: every score kept, log2 domain [b][Hkv][R][score_stride] (few rows only)
  int64_t score_stride;
  Work work;
  int32_t* status;
  int batch, T;
  int64_t n_kv;
  int H, Hkv;
  float qscale;  // softmax scale in the log2 domain
};

// V rows of a tile that reaches behind the context (row L - t0 of the tile on): rows that no token holds
// become 0, and so do values that are no finite numbers, whose rows are noted in `odd`.  Threads r of
// kRows call; the tile is D / 64 spans of 64 columns.
template <int D>
__device__ __forceinline__ void clear_tail_values(uint8_t* tile, int t0, int L, int T, bool listed,
                                                  const DraftTree& tree, uint32_t* odd, int r) {
  constexpr int CH = D / 8;  // 16 bytes each, CH to a row
  for (int e = max(0, L - t0) * CH + r; e < kRows * CH; e += kRows) {
    const int row = e / CH, c = e % CH, j = t0 + row - L;
    const bool held = j < T && (!listed || tree.end[j] == kRoot);
    uint4* p = reinterpret_cast<uint4*>(tile + (c >> 3) * kHalf + row * 128 + (c & 7) * 16);
    if (!held) {
      *p = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    uint4 w = *p;
    uint32_t* a = reinterpret_cast<uint32_t*>(&w);
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((a[i] & 0x7F80u) == 0x7F80u) {
        a[i] &= 0xFFFF0000u;
        found = true;
      }
      if ((a[i] & 0x7F800000u) == 0x7F800000u) {
        a[i] &= 0xFFFFu;
        found = true;
      }
    }
    if (found) {
      *p = w;
      atomicOr(&odd[j >> 5], 1u << (j & 31));
    }
  }
}

// Whether drafted token i sees drafted row j.
__device__ __forceinline__ bool sees(const DraftTree& tree, bool listed, int i, int j) {
  return listed ? (tree.anc[i][j >> 5] >> (j & 31)) & 1u : j <= i;
}

// The walk's next segment: its query rows (up to `rows` of an item) and its tree brought into the L2,
// by the threads r of kRows.
template <int D>
__device__ __forceinline__ void prefetch_next(Walk walk, const TreeArgs& a, int np, int rows, int r) {
  if (!walk.next()) return;
  const int G = a.H / a.Hkv, R = a.T * G, g = walk.item / np, base = (walk.item - g * np) * rows;
  for (int e = r; e < min(rows, R - base) * (D / 64); e += kRows) {
    const int rr = base + e / (D / 64), i = rr / G;
    prefetch_l2(a.q + (((int64_t)walk.s * a.T + i) * a.H + g * G + (rr - i * G)) * D + (e % (D / 64)) * 64);
  }
  if (a.parent && r * 32 < a.T) prefetch_l2(a.parent + (int64_t)walk.s * a.T + r * 32);
}

// Up to kFewRows query rows per KV head (tree_attn_few.cu), which are also an item's rows in the partial results.
constexpr int kFewRows = 16;
cudaError_t launch_tree_attn_few(const Shape& s, const void* k, const void* v, const TreeArgs& a, int ctas,
                                 cudaStream_t st);

}  // namespace hisa
