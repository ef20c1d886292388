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
struct alignas(16) DraftTree {
  uint32_t anc[kMaxDraft][kDraftWords];  // bit j of row i: slot j is slot i or one of its ancestors
  int16_t parent[kMaxDraft];             // kRoot, kEmpty or the slot before
  int16_t end[kMaxDraft];                // where the walk up from the slot ends: kRoot, kEmpty
};
constexpr int kRoot = -1, kEmpty = -2;

// Fills `t` from parent[0 .. T) with NT threads, tid of each; sync() is a barrier over them, the last
// thing done.  A slot is a token iff t.end[i] == kRoot; the rows of empty slots are 0.  Returns whether
// this thread saw a parent that is no parent, no root and no empty mark.  Every slot walks up to its
// root by itself (a parent lies in front of its child, so the walk ends): as many steps in shared
// memory as the tree is deep, and two barriers.
template <int NT, class Sync>
__device__ bool draft_tree_build(DraftTree& t, const int32_t* parent, int T, int tid, Sync sync) {
  bool bad = false;
  for (int i = tid; i < T; i += NT) {
    const int p = parent[i];
    const bool ok = p >= -1 && p < i;
    bad = bad || (!ok && p != kEmpty);
    t.parent[i] = (int16_t)(ok ? p : kEmpty);
    uint4* row = reinterpret_cast<uint4*>(t.anc[i]);
    row[0] = row[1] = make_uint4(0u, 0u, 0u, 0u);
  }
  sync();
  for (int i = tid; i < T; i += NT) {
    int j = i, word = i >> 5;
    uint32_t bits = 0;
    while (j >= 0) {
      if ((j >> 5) != word) {
        t.anc[i][word] = bits;
        bits = 0;
        word = j >> 5;
      }
      bits |= 1u << (j & 31);
      j = t.parent[j];
    }
    t.anc[i][word] = bits;
    t.end[i] = (int16_t)j;
    if (j != kRoot) {
      uint4* row = reinterpret_cast<uint4*>(t.anc[i]);
      row[0] = row[1] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  sync();
  return bad;
}

}  // namespace hisa
