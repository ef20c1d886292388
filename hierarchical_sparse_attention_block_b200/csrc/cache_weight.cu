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
// Work: a unit is one key tile of one sequence for a group of KV heads: as many heads as have their
// query rows in one buffer of 128 (fewer heads where the call has fewer units than SMs).  So a CTA
// keeps its query rows for all key tiles of a segment; each group's sums (4 bytes a key against its
// heads' 2 d bytes of K) go to the workspace and cache_weight_join_kernel adds them in order.  A CTA
// takes its range two key tiles at a time, one for each of its two readout groups.  A head with more
// than 128 rows takes several passes over the segment's keys.
// Roles (448 threads): warps 0-3 and 4-7 readout groups, thread = key; warps 8-11 the counted slots,
// the tree and the query rows (a gather: the counted slots lie anywhere); one thread each for the K
// loads (TMA) and the MMAs.  Every wait is bounded (1 s): a timeout sets status bit 1.
#include <math.h>

#include <algorithm>

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
constexpr int kLead = 2;  // what another item costs a CTA, in key tiles
constexpr int kReadout = 256, kLoaders = 128;
constexpr int kThreads = kReadout + kLoaders + 64;
constexpr int kWarpQ = 8, kWarpK = 12, kWarpMMA = 13;
constexpr uint32_t kTmemCols = 512;  // score buffer b at 128 b; readout group e uses buffers 2 e, 2 e + 1
constexpr float kLog2e = 1.4426950408889634f;

// What the query rows of a buffer add: minus their LSE in the log2 domain (-inf: nothing), their slots.
struct Rows {
  float nlse2[kQRows];
  int16_t slot[kQRows];
  uint32_t none[kQRows / 32];  // bit per row: padding, or a row that adds nothing
};

template <int D>
struct Cfg {
  static constexpr int kTile = kHalf * (D / 64);
  static constexpr int KS = D == 64 ? 8 : 4;  // K ring
  static constexpr int K_OFF = 2 * kTile;     // Q buffer b at b * kTile (kQRows rows)
  static constexpr int TREE_OFF = K_OFF + KS * kTile;
  static constexpr int ROW_OFF = (TREE_OFF + 2 * (int)sizeof(DraftTree) + 15) / 16 * 16;  // Rows [2]
  static constexpr int LIST_OFF = ROW_OFF + 2 * (int)sizeof(Rows);  // counted slots: int16 [2][kMaxDraft]
  static constexpr int BAR_OFF = LIST_OFF + 2 * 2 * kMaxDraft;
  enum : int {
    B_KFULL = 0,             // [KS]
    B_KEMPTY = B_KFULL + KS, // [KS]
    B_QFULL = B_KEMPTY + KS, // [2]
    B_QEMPTY = B_QFULL + 2,  // [2]
    B_SFULL = B_QEMPTY + 2,  // [4]
    B_SFREE = B_SFULL + 4,   // [4]
    B_SEGFULL = B_SFREE + 4,     // [2]: a segment's slots and tree are there
    B_SEGFREE = B_SEGFULL + 2,   // [2]: ... and read out
    B_GO = B_SEGFREE + 2,        // the first query rows are asked for
    B_LSYNC,                     // the loader warps among themselves
    B_DRAIN,
    kNBar
  };
  static constexpr int WALK_OFF = BAR_OFF + kNBar * 8;
  static constexpr int MISC_OFF = WALK_OFF + (int)sizeof(WalkShared<kThreads>);
  static constexpr int kSmem = MISC_OFF + 4 * 4 + 1024;
  static_assert(BAR_OFF % 8 == 0 && kSmem <= 227 * 1024, "shared memory budget");
};

// How the query rows of a head group pass through the buffers: in `chunks` fills.
struct Chunks {
  int h0, nh, R, subs, heads, chunks;
  __device__ Chunks(int h0_, int nh_, int R_) : h0(h0_), nh(nh_), R(R_) {
    subs = max(1, (R + kQRows - 1) / kQRows);                     // fills of one head
    heads = min(nh, max(1, kQRows / max(16, (R + 15) & ~15)));  // heads of one fill
    chunks = subs == 1 ? (nh + heads - 1) / heads : nh * subs;
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
    pitch = max(16, (rows + 15) & ~15);  // nothing counted: padding alone
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
  DraftTree* trees = reinterpret_cast<DraftTree*>(smem + C::TREE_OFF);  // [2]: of the segments in turn, as the lists
  Rows* rows_of = reinterpret_cast<Rows*>(smem + C::ROW_OFF);
  int16_t* lists = reinterpret_cast<int16_t*>(smem + C::LIST_OFF);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  uint32_t* tmem_slot = misc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* n_counted = reinterpret_cast<volatile int*>(misc + 2);  // [2]
  auto fail = [&]() {
    *abort_flag = 1;
    if (status) atomicOr(status, kStatusTimeout);
  };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int G = H / Hkv;
  const bool wide = T * G > kQRows;  // how often K is read depends on the counted slots
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
      if ((i >= C::B_SEGFULL && i < C::B_SEGFREE) || i == C::B_GO || i == C::B_LSYNC) n = kLoaders;
      if (i >= C::B_SEGFREE && i < C::B_GO) n = kReadout + (wide ? 2 : 1);  // and the MMA thread, the K thread
      mbar_init(bar(i), (uint32_t)n);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what the kernels before wrote, and read of the workspace
  tc_fence_before();
  Walk walk = walk_begin<kThreads>(kv_len, n_kv, T, batch, groups, kLead,
                                   *reinterpret_cast<WalkShared<kThreads>*>(smem + C::WALK_OFF), nullptr, status);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto chunks_of = [&](int item, int rows) {  // item: the group of KV heads; rows: query rows of a head
    const int h0 = (int)((int64_t)item * Hkv / groups), h1 = (int)((int64_t)(item + 1) * Hkv / groups);
    return Chunks(h0, h1 - h0, rows);
  };

  if (warp >= kWarpQ && warp < kWarpK) {
    // ---------------- the counted slots, the tree and the query rows ----------------
    const int lt = tid - kReadout;
    bool ok = true;
    uint32_t lphase = 0;
    int seg = 0, fill = 0;
    auto sync = [&]() {
      mbar_arrive(bar(C::B_LSYNC));
      ok = warp_wait_or_abort(bar(C::B_LSYNC), lphase, abort_flag) && ok;
      lphase ^= 1u;
    };
    while (ok && walk.next()) {
      // one segment ahead of the readout
      const int64_t seq = walk.s;
      const int sp = seg & 1;
      DraftTree& tree = trees[sp];
      int16_t* list = lists + sp * kMaxDraft;
      if (seg >= 2) {
        ok = warp_wait_or_abort(bar(C::B_SEGFREE + sp), (uint32_t)((seg >> 1) - 1) & 1u, abort_flag);
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
            if (!parent || tree.end[e[x]] == kRoot) {
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
          if (lane == 0) n_counted[sp] = all;
        } else {
          int n = 0;
          for (int i0 = 0; i0 < T; i0 += 32) {
            const int i = i0 + lane;
            const bool c = i < T && (!parent || tree.end[i] == kRoot);
            const uint32_t b = __ballot_sync(0xFFFFFFFFu, c);
            if (c) list[n + __popc(b & ((1u << lane) - 1u))] = (int16_t)i;
            n += __popc(b);
          }
          if (lane == 0) n_counted[sp] = n;
        }
      }
      if (bad && status) atomicOr(status, kStatusBadIndex);
      sync();
      if (!ok) break;
      mbar_arrive(bar(C::B_SEGFULL + sp));
      ++seg;
      Chunks ch = chunks_of(walk.item, n_counted[sp] * G);
      for (int c = 0; ok && c < ch.chunks; ++c, ++fill) {
        ch.at(c);
        const int b = fill & 1;
        if (fill >= 2) {
          ok = warp_wait_or_abort(bar(C::B_QEMPTY + b), (uint32_t)((fill >> 1) - 1) & 1u, abort_flag);
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
        Rows& rows = rows_of[b];
        float nl = -INFINITY;
        if (lt < total) {
          const int hd = lt / ch.pitch, rr = lt - hd * ch.pitch;
          int slot = 0;
          if (rr < ch.rows) {
            const int r = ch.row0 + rr, ci = r / G;
            slot = list[ci];
            const float l = lse[(seq * T + slot) * H + (ch.head + hd) * G + (r - ci * G)];
            nl = l == -INFINITY ? -INFINITY : l * -kLog2e;
          }
          rows.nlse2[lt] = nl;
          rows.slot[lt] = (int16_t)slot;
        }
        const uint32_t none = __ballot_sync(0xFFFFFFFFu, nl == -INFINITY);
        if (lane == 0) rows.none[lt >> 5] = none;
        if (fill == 0) mbar_arrive(bar(C::B_GO));
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
      const uint64_t policy = l2_evict_first();
      int seg = 0, issued = 0;
      while (ok && walk.next()) {
        int rows = 0;  // any number up to kQRows passes the group's heads in one fill
        if (wide) {
          ok = mbar_wait_or_abort(bar(C::B_SEGFULL + (seg & 1)), (uint32_t)(seg >> 1) & 1u, abort_flag);
          if (!ok) break;
          rows = n_counted[seg & 1] * G;
          mbar_arrive(bar(C::B_SEGFREE + (seg & 1)));
          ++seg;
        }
        Chunks ch = chunks_of(walk.item, rows);
        for (int c = 0; ok && c < ch.chunks; ++c) {
          ch.at(c);
          for (int x = 0; ok && x < walk.n; x += 2)
            for (int hd = 0; ok && hd < ch.n; ++hd)
              for (int e = 0; e < 2 && x + e < walk.n; ++e) {
                const int s = issued % C::KS;
                // The first query rows go before all but one K tile: behind the first tiles of every SM
                // they would wait for all of those.
                if (issued == 1 && !mbar_wait_or_abort(bar(C::B_GO), 0, abort_flag)) {
                  ok = false;
                  break;
                }
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
                              bar(C::B_KFULL + s), policy);
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
    {
      auto waited = [&](uint32_t barrier, uint32_t parity) {
        return warp_wait_or_abort(barrier, parity, abort_flag);
      };
      bool ok = true;
      int seg = 0, fill = 0, kit = 0;
      int made[2] = {0, 0};  // products handed to each readout group
      while (ok && walk.next()) {
        ok = waited(bar(C::B_SEGFULL + (seg & 1)), (uint32_t)(seg >> 1) & 1u);
        if (!ok) break;
        Chunks ch = chunks_of(walk.item, n_counted[seg & 1] * G);
        if (lane == 0) mbar_arrive(bar(C::B_SEGFREE + (seg & 1)));
        ++seg;
        for (int c = 0; ok && c < ch.chunks; ++c, ++fill) {
          ch.at(c);
          const int qb = fill & 1;
          ok = waited(bar(C::B_QFULL + qb), (uint32_t)(fill >> 1) & 1u);
          const uint32_t idesc = idesc_bf16(kKeys, ch.pitch, false, false);
          for (int x = 0; ok && x < walk.n; x += 2)
            for (int hd = 0; ok && hd < ch.n; ++hd)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (!ok || x + e >= walk.n) continue;
                const int s = kit % C::KS, buf = 2 * e + (made[e] & 1);
                ok = waited(bar(C::B_KFULL + s), (uint32_t)(kit / C::KS) & 1u) &&
                     (made[e] < 2 ||
                      waited(bar(C::B_SFREE + buf), (uint32_t)((made[e] >> 1) - 1) & 1u));
                if (!ok) continue;
                tc_fence_after();
                const uint32_t kt = sb + (uint32_t)(C::K_OFF + s * C::kTile);
                const uint32_t qt = sb + (uint32_t)(qb * C::kTile + hd * ch.pitch * 128);
                if (elect_one()) {
#pragma unroll
                  for (int h2 = 0; h2 < D / 64; ++h2)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                      umma_bf16(tmem + 128u * (uint32_t)buf, desc_kmajor_sw128(kt + h2 * kHalf + kk * 32),
                                desc_kmajor_sw128(qt + h2 * kHalf + kk * 32), idesc, (h2 | kk) ? 1u : 0u);
                  umma_commit(bar(C::B_SFULL + buf));
                  umma_commit(bar(C::B_KEMPTY + s));
                }
                ++made[e];
                ++kit;
              }
          if (ok && elect_one()) umma_commit(bar(C::B_QEMPTY + qb));
        }
      }
      if (!ok && lane == 0) fail();
      if (elect_one()) umma_commit(bar(C::B_DRAIN));
      mbar_wait(bar(C::B_DRAIN), 0);
    }
  } else {
    // ---------------- readout: group e, thread = key ----------------
    const int e = warp >> 2, r = tid & (kKeys - 1);
    const uint32_t ts = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256u * (uint32_t)e;
    bool ok = true;
    int seg = 0, fill = 0, got = 0;
    while (ok && walk.next()) {
      const int sp = seg & 1;
      ok = warp_wait_or_abort(bar(C::B_SEGFULL + sp), (uint32_t)(seg >> 1) & 1u, abort_flag);
      ++seg;
      if (!ok) break;
      const DraftTree& tree = trees[sp];
      const int64_t seq = walk.s;
      const int L = (int)walk.L;
      Chunks ch = chunks_of(walk.item, n_counted[sp] * G);
      float* out = groups == 1 ? weight + seq * n_kv : part + ((int64_t)walk.item * batch + seq) * n_kv;
      for (int c = 0; ok && c < ch.chunks; ++c, ++fill) {
        ch.at(c);
        const int qb = fill & 1;
        ok = warp_wait_or_abort(bar(C::B_QFULL + qb), (uint32_t)(fill >> 1) & 1u, abort_flag);
        for (int x = e; ok && x < walk.n; x += 2) {
          const int t = (walk.j0 + x) * kKeys + r;
          const bool tail = (walk.j0 + x + 1) * kKeys > L;
          const int j = t - L;  // drafted row, from the context's end on
          const int j_word = min(max(j, 0) >> 5, kDraftWords - 1), j_bit = j & 31;
          // One fill's sum of a key joins what the fills before left; read while the products are formed.
          float sum = t < L + T && (c > 0 || (groups == 1 && t < L)) ? out[t] : 0.f;
          for (int hd = 0; ok && hd < ch.n; ++hd, ++got) {
            const int buf = got & 1;
            ok = warp_wait_or_abort(bar(C::B_SFULL + 2 * e + buf), (uint32_t)(got >> 1) & 1u, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const Rows& rows = rows_of[qb];
            const int first = hd * ch.pitch;
            const float2 qs2 = {qscale, qscale};
            float2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
            const uint32_t tb = ts + 128u * (uint32_t)buf;
            auto take = [&](int c0, uint32_t(&s)[32]) {  // columns c0 .. c0 + 31, those below the pitch
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int at = first + c0 + 16 * h;
                if (c0 + 16 * h >= ch.pitch) break;
                float nl[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                  *reinterpret_cast<float4*>(nl + i) = *reinterpret_cast<const float4*>(rows.nlse2 + at + i);
                const uint32_t none = rows.none[at >> 5] >> (at & 16) & 0xFFFFu;
                if (none == 0 && !tail) {
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    const uint32_t* z = s + 16 * h + 2 * i;
                    const float2 x = ffma2(make_float2(__uint_as_float(z[0]), __uint_as_float(z[1])), qs2,
                                           make_float2(nl[2 * i], nl[2 * i + 1]));
                    acc[i & 1] = fadd2(acc[i & 1], make_float2(fast_exp2(x.x), fast_exp2(x.y)));
                  }
                  continue;
                }
                // Padding, rows that add nothing, and, for a drafted row, the slots not below it in the tree.
                // No branch a column: a CTA with a tile behind the context is the one all others wait for
                // (1 x 8K keys, 1024 rows a KV head: 170 us with a test for each column, 93 this way).
                uint32_t hidden = none;
                if (tail) {
                  uint32_t seen = 0;
                  if (parent) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                      seen |= (tree.anc[rows.slot[at + i]][j_word] >> j_bit & 1u) << i;
                  } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) seen |= (j <= rows.slot[at + i] ? 1u : 0u) << i;
                  }
                  hidden |= j < 0 ? 0u : ~seen;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float p = fast_exp2(fmaf(__uint_as_float(s[16 * h + i]), qscale, nl[i]));
                  acc[i & 1].x += (hidden >> i) & 1u ? 0.f : p;
                }
              }
            };
#pragma unroll 1
            for (int c0 = 0; c0 < ch.pitch; c0 += 32) {  // a load may reach behind the pitch, within the buffer
              uint32_t x[32];
              __syncwarp();
              tmem_ld32_issue(tb + (uint32_t)c0, x);
              tmem_wait_ld(x);
              take(c0, x);
            }
            tc_fence_before();
            mbar_arrive(bar(C::B_SFREE + 2 * e + buf));
            acc[0] = fadd2(acc[0], acc[1]);
            sum += acc[0].x + acc[0].y;
          }
          if (ok && t < L + T) out[t] = sum;
        }
        mbar_arrive(bar(C::B_QEMPTY + qb));
      }
      mbar_arrive(bar(C::B_SEGFREE + sp));
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t seq = blockIdx.y, L = context_len(kv_len, seq, T, n_kv);
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (L < 0 || t >= L + T) return;
  float sum = t < L ? weight[seq * n_kv + t] : 0.f;
#pragma unroll 8
  for (int g = 0; g < groups; ++g) sum += part[((int64_t)g * batch + seq) * n_kv + t];
  weight[seq * n_kv + t] = sum;
}

// KV-head groups: of as many heads as have their query rows in one buffer, and at least as many
// groups as give every SM a unit.
int head_groups(const Shape& s) {
  const int64_t R = s.n_q * (s.H / s.Hkv), pitch = (R + 15) / 16 * 16;
  const int64_t heads = R > kQRows ? 1 : kQRows / pitch;
  const int64_t tiles = (int64_t)s.batch * ((s.n_kv + kKeys - 1) / kKeys);
  const int64_t g = std::max((s.Hkv + heads - 1) / heads, (kMaxCtas + tiles - 1) / tiles);
  return (int)std::min<int64_t>(g, s.Hkv);
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
  e = launch_after(cache_weight_kernel<D>, dim3((unsigned)(most < kMaxCtas ? most : kMaxCtas)), kThreads, st,
                   Cfg<D>::kSmem, mk, static_cast<const uint16_t*>(q), kv_len, parent, path, lse, weight, part, status,
                   s.batch, (int)s.n_q, s.n_kv, s.H, s.Hkv, groups, s.scale * kLog2e);
  if (e != cudaSuccess) return e;
  if (groups > 1)
    e = launch_after(cache_weight_join_kernel, dim3((unsigned)((s.n_kv + 255) / 256), (unsigned)s.batch), 256, st, 0, part,
                     kv_len, weight, s.batch, (int)s.n_q, s.n_kv, groups);
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
