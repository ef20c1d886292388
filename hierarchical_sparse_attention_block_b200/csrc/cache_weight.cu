// hisa_cache_weight: the attention weight each cached row receives, on the 5th-generation tensor
// cores.
//
//   a(t) = sum over counted slots i that see t, heads h, of exp(scale q[i,h].k[t,g] - lse[i,h])
//   w(t) = (t < L ? w(t) : 0) + a(t),  t < L + T
//
// The keys are the rows of the product: S^T = K Q^T, a tile of 128 keys (the M of the MMA, one TMEM
// lane each) against the N = 16 .. 128 query rows of one KV head (counted slots x the head's G query
// heads, padded to 16).  So few query rows cost little, and a thread, which owns one key, adds its
// row of weights up in registers: no sum crosses threads, and its order is fixed.  K is read once:
// bound by HBM for few rows, by the exponentials (16 a clock and SM) from about 128 rows a KV head.
//
// Work: a unit is one key tile of one sequence for a group of KV heads (all of them, unless the
// call has fewer key tiles than SMs: then the heads are split, each group's sums go to the workspace
// and cache_weight_join_kernel adds them in order).  A CTA takes its range two key tiles at a time,
// one for each of its two readout groups, and streams their K heads through a ring; the query rows
// of as many heads as fit 128 rows stay in shared memory for all key tiles of the segment (two
// buffers: the next heads' rows arrive meanwhile).  A head with more than 128 rows takes several
// passes over the segment's keys.
// Roles (448 threads): warps 0-3 and 4-7 readout groups, thread = key; warps 8-11 the counted slots,
// the tree and the query rows (a gather: the counted slots lie anywhere); one thread each for the K
// loads (TMA) and the MMAs.  Every wait is bounded (1 s): a timeout sets status bit 1.
#include <math.h>

#include "attn_math.cuh"
#include "cache_walk.cuh"
#include "common.cuh"
#include "draft_tree.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace hisa {
namespace {

using namespace tc;

constexpr int kKeys = kTileKeys;
constexpr int kQRows = 128;         // query rows of one buffer
constexpr int kHalf = kKeys * 128;  // 64 columns of 128 rows of 16-bit values: one 128-byte swizzle span
constexpr int kReadout = 256, kLoaders = 128;
constexpr int kThreads = kReadout + kLoaders + 64;
constexpr int kWarpQ = 8, kWarpK = 12, kWarpMMA = 13;
constexpr uint32_t kTmemCols = 512;  // score buffer b at 128 b; readout group e uses buffers 2 e, 2 e + 1
constexpr float kLog2e = 1.4426950408889634f;

// What a query row of a buffer adds: lse in the log2 domain (+inf: nothing) and its slot.
struct Row {
  float lse2;
  int slot;
};

template <int D>
struct Cfg {
  static constexpr int kTile = kHalf * (D / 64);
  static constexpr int KS = D == 64 ? 8 : 4;  // K ring
  static constexpr int K_OFF = 2 * kTile;     // Q buffer b at b * kTile (kQRows rows)
  static constexpr int TREE_OFF = K_OFF + KS * kTile;
  static constexpr int ROW_OFF = (TREE_OFF + (int)sizeof(DraftTree) + 15) / 16 * 16;  // Row [2][kQRows]
  static constexpr int LIST_OFF = ROW_OFF + 2 * kQRows * (int)sizeof(Row);            // counted slots: int16 [kMaxDraft]
  static constexpr int BAR_OFF = LIST_OFF + 2 * kMaxDraft;
  enum : int {
    B_KFULL = 0,             // [KS]
    B_KEMPTY = B_KFULL + KS, // [KS]
    B_QFULL = B_KEMPTY + KS, // [2]
    B_QEMPTY = B_QFULL + 2,  // [2]
    B_SFULL = B_QEMPTY + 2,  // [4]
    B_SFREE = B_SFULL + 4,   // [4]
    B_SEGFULL = B_SFREE + 4, // the segment's slots and tree are there
    B_SEGFREE,               // ... and read out
    B_LSYNC,                 // the loader warps among themselves
    B_DRAIN,
    kNBar
  };
  static constexpr int WALK_OFF = BAR_OFF + kNBar * 8;
  static constexpr int MISC_OFF = WALK_OFF + (int)sizeof(WalkShared<kThreads>);
  static constexpr int kSmem = MISC_OFF + 4 * (3 + 2 * kDraftWords) + 1024;
  static_assert(BAR_OFF % 8 == 0 && kSmem <= 227 * 1024, "shared memory budget");
};

// How the query rows of a head group pass through the buffers: in `chunks` fills.
struct Chunks {
  int h0, nh, R, subs, heads, chunks;
  __device__ Chunks(int h0_, int nh_, int R_) : h0(h0_), nh(nh_), R(R_) {
    subs = max(1, (R + kQRows - 1) / kQRows);              // fills of one head
    heads = R == 0 ? 1 : max(1, kQRows / ((R + 15) & ~15));  // heads of one fill
    chunks = R == 0 ? 0 : subs == 1 ? (nh + heads - 1) / heads : nh * subs;
  }
  // fill c: heads [head, head + n), rows [row0, row0 + rows) of each, at pitch `pitch` in the buffer
  int head, n, row0, rows, pitch;
  __device__ void at(int c) {
    if (subs == 1) {
      head = h0 + c * heads;
      n = min(heads, h0 + nh - head);
      row0 = 0;
      rows = R;
    } else {
      head = h0 + c / subs;
      n = 1;
      row0 = c % subs * kQRows;
      rows = min(kQRows, R - row0);
    }
    pitch = (rows + 15) & ~15;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cache_weight_kernel(const __grid_constant__ CUtensorMap map_k, const uint16_t* __restrict__ q,
                        const int32_t* __restrict__ kv_len, const int32_t* __restrict__ parent,
                        const int32_t* __restrict__ path, const float* __restrict__ lse, float* __restrict__ weight,
                        float* __restrict__ part, int32_t* __restrict__ status, int batch, int T, int64_t n_kv, int H,
                        int Hkv, int groups, float qscale) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) { return sb + (uint32_t)C::BAR_OFF + 8u * (uint32_t)i; };
  DraftTree& tree = *reinterpret_cast<DraftTree*>(smem + C::TREE_OFF);
  Row* rows_of = reinterpret_cast<Row*>(smem + C::ROW_OFF);
  int16_t* list = reinterpret_cast<int16_t*>(smem + C::LIST_OFF);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  uint32_t* tmem_slot = misc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* n_counted = reinterpret_cast<volatile int*>(misc + 2);
  auto fail = [&]() {
    *abort_flag = 1;
    if (status) atomicOr(status, kStatusTimeout);
  };
  if (warp == kWarpMMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < C::kNBar; ++i) {
      int n = 1;
      if (i >= C::B_QFULL && i < C::B_QEMPTY) n = kLoaders;
      if (i >= C::B_QEMPTY && i < C::B_SFULL) n = kReadout + 1;
      if (i >= C::B_SFREE && i < C::B_SEGFULL) n = kKeys;
      if (i == C::B_SEGFULL || i == C::B_LSYNC) n = kLoaders;
      if (i == C::B_SEGFREE) n = kReadout + 2;  // and the K and MMA threads
      mbar_init(bar(i), (uint32_t)n);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  tc_fence_before();
  Walk walk = walk_begin<kThreads>(kv_len, n_kv, T, batch, groups,
                                   *reinterpret_cast<WalkShared<kThreads>*>(smem + C::WALK_OFF), nullptr, status);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int G = H / Hkv;
  auto chunks_of = [&](int item) {  // item: the group of KV heads
    const int h0 = (int)((int64_t)item * Hkv / groups), h1 = (int)((int64_t)(item + 1) * Hkv / groups);
    return Chunks(h0, h1 - h0, *n_counted * G);
  };

  if (warp >= kWarpQ && warp < kWarpK) {
    // ---------------- the counted slots, the tree and the query rows ----------------
    const int lt = tid - kReadout;
    bool ok = true;
    uint32_t lphase = 0;
    int seg = 0, fill = 0;
    auto sync = [&]() {
      mbar_arrive(bar(C::B_LSYNC));
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_LSYNC), lphase, abort_flag)) && ok;
      lphase ^= 1u;
    };
    while (ok && walk.next()) {
      const int64_t seq = walk.s;
      if (seg > 0) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_SEGFREE), (uint32_t)(seg - 1) & 1u, abort_flag));
        if (!ok) break;
      }
      bool bad = false;
      if (parent) bad = draft_tree_build<kLoaders>(tree, parent + seq * T, T, lt, sync);
      if (!ok) break;
      if (lt < 32) {
        // slots 8 lane .. 8 lane + 7 of this lane: a bit each for the counted ones
        const int32_t* p = path ? path + seq * T : nullptr;
        if (p) {
          // the list's entries in the same split: kept if in range and above every in-range entry before
          int e[8], top = -1;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            e[x] = 8 * lane + x < T ? p[8 * lane + x] : -1;
            if (e[x] < -1 || e[x] >= T) {
              bad = true;
              e[x] = -1;
            }
            top = max(top, e[x]);
          }
          int above = top;  // inclusive maximum over the lanes, then exclusive
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, above, off);
            if (lane >= off) above = max(above, y);
          }
          above = __shfl_up_sync(0xFFFFFFFFu, above, 1);
          if (lane == 0) above = -1;
          int kept = 0;
          uint32_t keep = 0;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            if (e[x] < 0) continue;
            if (e[x] <= above) {
              bad = true;
              continue;
            }
            above = e[x];
            if (!parent || tree.up[e[x]] == kRoot) {
              keep |= 1u << x;
              ++kept;
            }
          }
          int at = kept;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, at, off);
            if (lane >= off) at += y;
          }
          const int all = __shfl_sync(0xFFFFFFFFu, at, 31);
          at -= kept;
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if ((keep >> x) & 1u) list[at++] = (int16_t)e[x];
          if (lane == 0) *n_counted = all;
        } else {
          int n = 0;
          for (int i0 = 0; i0 < T; i0 += 32) {
            const int i = i0 + lane;
            const bool c = i < T && (!parent || tree.up[i] == kRoot);
            const uint32_t b = __ballot_sync(0xFFFFFFFFu, c);
            if (c) list[n + __popc(b & ((1u << lane) - 1u))] = (int16_t)i;
            n += __popc(b);
          }
          if (lane == 0) *n_counted = n;
        }
      }
      if (bad && status) atomicOr(status, kStatusBadIndex);
      sync();
      if (!ok) break;
      mbar_arrive(bar(C::B_SEGFULL));
      ++seg;
      Chunks ch = chunks_of(walk.item);
      for (int c = 0; ok && c < ch.chunks; ++c, ++fill) {
        ch.at(c);
        const int b = fill & 1;
        if (fill >= 2) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_QEMPTY + b), (uint32_t)((fill >> 1) - 1) & 1u, abort_flag));
          if (!ok) break;
        }
        constexpr int CH = D / 8;  // 16-byte chunks of a row
        uint8_t* qb = smem + b * C::kTile;
        const int total = ch.n * ch.pitch;  // buffer rows
        // all copies of the fill in flight at once (16 bytes each, CH threads a row)
        for (int e = lt; e < total * CH; e += kLoaders) {
          const int row = e / CH, x = e % CH, hd = row / ch.pitch, rr = row - hd * ch.pitch;
          const uint16_t* src = q;
          const bool held = rr < ch.rows;
          if (held) {
            const int r = ch.row0 + rr, ci = r / G;
            src = q + ((seq * T + list[ci]) * H + (ch.head + hd) * G + (r - ci * G)) * D + x * 8;
          }
          cp_async16(qb + (x >> 3) * kHalf + row * 128 + (((x & 7) ^ (row & 7)) << 4), src, held);
        }
        cp_async_commit();
        for (int row = lt; row < total; row += kLoaders) {
          const int hd = row / ch.pitch, rr = row - hd * ch.pitch;
          Row out = {INFINITY, 0};
          if (rr < ch.rows) {
            const int r = ch.row0 + rr, ci = r / G;
            out.slot = list[ci];
            const float l = lse[(seq * T + out.slot) * H + (ch.head + hd) * G + (r - ci * G)];
            out.lse2 = l == -INFINITY ? INFINITY : l * kLog2e;
          }
          rows_of[b * kQRows + row] = out;
        }
        cp_async_wait<0>();
        fence_async_smem();
        mbar_arrive(bar(C::B_QFULL + b));
      }
    }
    if (!ok && lane == 0) fail();
  } else if (warp == kWarpK) {
    // ---------------- K tiles ----------------
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
      bool ok = true;
      int seg = 0, issued = 0;
      while (ok && walk.next()) {
        ok = mbar_wait_or_abort(bar(C::B_SEGFULL), (uint32_t)seg & 1u, abort_flag);
        ++seg;
        if (!ok) break;
        Chunks ch = chunks_of(walk.item);
        mbar_arrive(bar(C::B_SEGFREE));
        for (int c = 0; ok && c < ch.chunks; ++c) {
          ch.at(c);
          for (int x = 0; ok && x < walk.n; x += 2)
            for (int hd = 0; ok && hd < ch.n; ++hd)
              for (int e = 0; e < 2 && x + e < walk.n; ++e) {
                const int s = issued % C::KS;
                if (issued >= C::KS &&
                    !mbar_wait_or_abort(bar(C::B_KEMPTY + s), (uint32_t)(issued / C::KS - 1) & 1u, abort_flag)) {
                  ok = false;
                  break;
                }
                const uint32_t dst = sb + (uint32_t)(C::K_OFF + s * C::kTile);
                mbar_expect_tx(bar(C::B_KFULL + s), C::kTile);
#pragma unroll
                for (int h2 = 0; h2 < D / 64; ++h2)
                  tma_load_4d(dst + h2 * kHalf, &map_k, 64 * h2, ch.head + hd, (walk.j0 + x + e) * kKeys, walk.s,
                              bar(C::B_KFULL + s));
                ++issued;
              }
        }
      }
      if (!ok) fail();
      // The copies in flight land before the CTA may exit.
      for (int x = max(0, issued - C::KS); x < issued; ++x)
        mbar_wait(bar(C::B_KFULL + x % C::KS), (uint32_t)(x / C::KS) & 1u);
    }
  } else if (warp == kWarpMMA) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      bool ok = true;
      int seg = 0, fill = 0, kit = 0;
      int made[2] = {0, 0};  // products handed to each readout group
      while (ok && walk.next()) {
        ok = mbar_wait_or_abort(bar(C::B_SEGFULL), (uint32_t)seg & 1u, abort_flag);
        ++seg;
        if (!ok) break;
        Chunks ch = chunks_of(walk.item);
        mbar_arrive(bar(C::B_SEGFREE));
        for (int c = 0; ok && c < ch.chunks; ++c, ++fill) {
          ch.at(c);
          const int qb = fill & 1;
          ok = mbar_wait_or_abort(bar(C::B_QFULL + qb), (uint32_t)(fill >> 1) & 1u, abort_flag);
          const uint32_t idesc = idesc_bf16(kKeys, ch.pitch, false, false);
          for (int x = 0; ok && x < walk.n; x += 2)
            for (int hd = 0; ok && hd < ch.n; ++hd)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (!ok || x + e >= walk.n) continue;
                const int s = kit % C::KS, buf = 2 * e + (made[e] & 1);
                ok = mbar_wait_or_abort(bar(C::B_KFULL + s), (uint32_t)(kit / C::KS) & 1u, abort_flag) &&
                     (made[e] < 2 ||
                      mbar_wait_or_abort(bar(C::B_SFREE + buf), (uint32_t)((made[e] >> 1) - 1) & 1u, abort_flag));
                if (!ok) continue;
                tc_fence_after();
                const uint32_t kt = sb + (uint32_t)(C::K_OFF + s * C::kTile);
                const uint32_t qt = sb + (uint32_t)(qb * C::kTile + hd * ch.pitch * 128);
#pragma unroll
                for (int h2 = 0; h2 < D / 64; ++h2)
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk)
                    umma_bf16(tmem + 128u * (uint32_t)buf, desc_kmajor_sw128(kt + h2 * kHalf + kk * 32),
                              desc_kmajor_sw128(qt + h2 * kHalf + kk * 32), idesc, (h2 | kk) ? 1u : 0u);
                umma_commit(bar(C::B_SFULL + buf));
                umma_commit(bar(C::B_KEMPTY + s));
                ++made[e];
                ++kit;
              }
          if (ok) umma_commit(bar(C::B_QEMPTY + qb));
        }
      }
      if (!ok) fail();
      umma_commit(bar(C::B_DRAIN));
      mbar_wait(bar(C::B_DRAIN), 0);
    }
  } else {
    // ---------------- readout: group e, thread = key ----------------
    const int e = warp >> 2, r = tid & (kKeys - 1);
    const uint32_t ts = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256u * (uint32_t)e;
    bool ok = true;
    int seg = 0, fill = 0, got = 0;
    while (ok && walk.next()) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_SEGFULL), (uint32_t)seg & 1u, abort_flag));
      ++seg;
      if (!ok) break;
      const int64_t seq = walk.s;
      const int L = (int)walk.L;
      Chunks ch = chunks_of(walk.item);
      float* out = groups == 1 ? weight + seq * n_kv : part + ((int64_t)walk.item * batch + seq) * n_kv;
      // One fill's sum of a key joins what the fills before left; nothing counted leaves 0.
      auto add = [&](int c, int t, float sum) {
        if (t >= L + T) return;
        if (c > 0 || (groups == 1 && t < L)) sum += out[t];
        out[t] = sum;
      };
      if (ch.chunks == 0)
        for (int x = e; x < walk.n; x += 2) add(0, (walk.j0 + x) * kKeys + r, 0.f);
      for (int c = 0; ok && c < ch.chunks; ++c, ++fill) {
        ch.at(c);
        const int qb = fill & 1;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_QFULL + qb), (uint32_t)(fill >> 1) & 1u, abort_flag));
        for (int x = e; ok && x < walk.n; x += 2) {
          const int t = (walk.j0 + x) * kKeys + r;
          const bool tail = (walk.j0 + x + 1) * kKeys > L;
          const int j = t - L;  // drafted row, from the context's end on
          float sum = 0.f;
          for (int hd = 0; ok && hd < ch.n; ++hd, ++got) {
            const int buf = got & 1;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_SFULL + 2 * e + buf), (uint32_t)(got >> 1) & 1u, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const Row* rows = rows_of + qb * kQRows + hd * ch.pitch;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            for (int c0 = 0; c0 < ch.rows; c0 += 16) {
              uint32_t s[16];
              __syncwarp();  // the load takes the whole warp
              tmem_ld<16>(ts + 128u * (uint32_t)buf + (uint32_t)c0, s);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const Row row = rows[c0 + i];
                bool see = row.lse2 < INFINITY || row.lse2 != row.lse2;  // padding and rows that count nothing: +inf
                if (tail && j >= 0)
                  see = see && (parent ? j < T && ((tree.anc[row.slot][j >> 5] >> (j & 31)) & 1u) : j <= row.slot);
                const float p = fast_exp2(fmaf(__uint_as_float(s[i]), qscale, -row.lse2));
                acc[i & 3] += see ? p : 0.f;
              }
            }
            tc_fence_before();
            mbar_arrive(bar(C::B_SFREE + 2 * e + buf));
            sum += (acc[0] + acc[1]) + (acc[2] + acc[3]);
          }
          if (ok) add(c, t, sum);
        }
        mbar_arrive(bar(C::B_QEMPTY + qb));
      }
      mbar_arrive(bar(C::B_SEGFREE));
    }
    if (!ok && lane == 0) fail();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

// The head groups' sums joined, in order, with the weights.
__global__ void __launch_bounds__(256)
    cache_weight_join_kernel(const float* __restrict__ part, const int32_t* __restrict__ kv_len,
                             float* __restrict__ weight, int batch, int T, int64_t n_kv, int groups) {
  const int64_t seq = blockIdx.y, L = context_len(kv_len, seq, T, n_kv);
  if (L < 0) return;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < L + T; t += (int64_t)gridDim.x * 256) {
    float sum = t < L ? weight[seq * n_kv + t] : 0.f;
    for (int g = 0; g < groups; ++g) sum += part[((int64_t)g * batch + seq) * n_kv + t];
    weight[seq * n_kv + t] = sum;
  }
}

// KV-head groups: one, unless the key tiles alone leave SMs idle.
int head_groups(const Shape& s) {
  const int64_t tiles = (int64_t)s.batch * ((s.n_kv + kKeys - 1) / kKeys);
  if (tiles >= kMaxCtas) return 1;
  const int64_t g = (kMaxCtas + tiles - 1) / tiles;
  return (int)(g < s.Hkv ? g : s.Hkv);
}

template <int D>
cudaError_t launch(const Shape& s, const void* q, const void* k, const int32_t* kv_len, const int32_t* parent,
                   const int32_t* path, const float* lse, float* weight, int32_t* status, float* part,
                   cudaStream_t st) {
  CUtensorMap mk;
  if (!map_cache_rows(&mk, k, D, (uint64_t)s.Hkv, (uint64_t)s.n_kv, (uint64_t)s.batch, kKeys))
    return cudaErrorNotSupported;
  cudaError_t e = ensure_smem((const void*)cache_weight_kernel<D>, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  const int groups = head_groups(s);
  const int64_t most = (int64_t)s.batch * groups * ((s.n_kv + kKeys - 1) / kKeys);
  cache_weight_kernel<D><<<(unsigned)(most < kMaxCtas ? most : kMaxCtas), kThreads, Cfg<D>::kSmem, st>>>(
      mk, static_cast<const uint16_t*>(q), kv_len, parent, path, lse, weight, part, status, s.batch, (int)s.n_q, s.n_kv,
      s.H, s.Hkv, groups, s.scale * kLog2e);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (groups > 1) {
    const int64_t want = (s.n_kv + 255) / 256;
    cache_weight_join_kernel<<<dim3((unsigned)want, (unsigned)s.batch), 256, 0, st>>>(part, kv_len, weight, s.batch,
                                                                                      (int)s.n_q, s.n_kv, groups);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

size_t cache_weight_workspace_bytes(const Shape& s) {
  const int g = head_groups(s);
  return g == 1 ? 0 : (size_t)g * s.batch * s.n_kv * sizeof(float);
}

cudaError_t launch_cache_weight(const Shape& s, const void* q, const void* k, const int32_t* kv_len,
                                const int32_t* parent, const int32_t* path, const float* lse, float* weight,
                                int32_t* status, void* ws, cudaStream_t st) {
  const auto run = s.d == 64 ? launch<64> : launch<128>;
  return run(s, q, k, kv_len, parent, path, lse, weight, status, static_cast<float*>(ws), st);
}

}  // namespace hisa
