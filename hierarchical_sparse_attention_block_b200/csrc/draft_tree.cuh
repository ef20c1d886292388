// The tree of drafted tokens: which slots of a sequence are tokens, and the ancestors of each.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace hisa {

constexpr int kDraftWords = kMaxDraft / 32;

// Context rows of sequence `seq` (0 <= L, L + T <= n_kv), or -1 where the caller's length breaks that.
__device__ __forceinline__ int64_t context_len(const int32_t* kv_len, int64_t seq, int64_t T, int64_t n_kv) {
  const int64_t L = kv_len[seq];
  return L < 0 || L + T > n_kv ? -1 : L;
}

// One sequence's tree in shared memory.
struct DraftTree {
  uint32_t anc[kMaxDraft][kDraftWords];  // bit j of row i: slot j is slot i or one of its ancestors
  int16_t up[kMaxDraft];                 // slot the walk stands at; kRoot, kEmpty at its end
};
constexpr int kRoot = -1, kEmpty = -2;

// Fills `t` from parent[0 .. T) (null: a chain) with NT threads, tid of each; sync() is a barrier
// over them.  A slot is a token iff t.up[i] == kRoot afterwards; the rows of empty slots are 0.  Returns
// whether this thread saw a parent that is no parent, no root and no empty mark.
// Each round joins every slot's set with the set of the slot its walk has reached and doubles the
// walk's step, so ceil(log2 T) rounds reach the root from any depth.
template <int NT, class Sync>
__device__ bool draft_tree_build(DraftTree& t, const int32_t* parent, int T, int tid, Sync sync) {
  constexpr int kPer = (kMaxDraft + NT - 1) / NT;
  const int nw = (T + 31) / 32;
  bool bad = false;
  for (int i = tid; i < T; i += NT) {
    if (parent == nullptr) {
      for (int w = 0; w < kDraftWords; ++w) {
        const int hi = i - 32 * w;  // bits 0 .. hi of word w
        t.anc[i][w] = hi < 0 ? 0u : hi >= 31 ? 0xFFFFFFFFu : (2u << hi) - 1u;
      }
      t.up[i] = kRoot;
      continue;
    }
    const int p = parent[i];
    const bool ok = p >= -1 && p < i;
    bad = bad || (!ok && p != -2);
    for (int w = 0; w < kDraftWords; ++w) t.anc[i][w] = w == (i >> 5) ? 1u << (i & 31) : 0u;
    t.up[i] = (int16_t)(ok ? p : kEmpty);
  }
  sync();
  if (parent == nullptr) return false;
  for (int reach = 1; reach < T; reach *= 2) {
    // the sets and steps of this round are read before any of them is written
    uint32_t set[kPer][kDraftWords];
    int step[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const int i = tid + c * NT;
      const int j = i < T ? t.up[i] : kRoot;
      step[c] = j >= 0 ? t.up[j] : j;
#pragma unroll
      for (int w = 0; w < kDraftWords; ++w) set[c][w] = j >= 0 && w < nw ? t.anc[j][w] : 0u;
    }
    sync();
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const int i = tid + c * NT;
      if (i >= T) continue;
      t.up[i] = (int16_t)step[c];
#pragma unroll
      for (int w = 0; w < kDraftWords; ++w)
        if (w < nw) t.anc[i][w] |= set[c][w];
    }
    sync();
  }
  for (int i = tid; i < T; i += NT)
    if (t.up[i] != kRoot)
      for (int w = 0; w < nw; ++w) t.anc[i][w] = 0u;
  sync();
  return bad;
}

}  // namespace hisa
