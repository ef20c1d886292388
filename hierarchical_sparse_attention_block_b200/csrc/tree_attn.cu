// hisa_tree_attn_fwd: attention of drafted tokens over a cache, on the 5th-generation tensor cores.
//
//   z(t) = scale q[i,h].k[t,g],  lse = ln sum_{t in V(i)} e^z(t),  o = sum_{t in V(i)} e^(z(t) - lse) v[t,g],
//   V(i) = the context's rows [0, L) and the drafted rows L + j of i's ancestors and itself.
//
// The T tokens of a sequence and the G = H / Hk heads of one KV head make R = T G query rows that
// read the same K and V.  With few rows the call is bound by the cache's bytes, with many (R above
// about 128) by the tensor cores; one kernel serves both: tiles of 128 query rows (padded) against
// tiles of 128 keys.  A tile of 128 x 128 costs the tensor cores about half the time that its K and V
// take from HBM, so the padding of few rows costs nothing; R above 128 puts two row tiles on one CTA,
// which then reads every K/V tile once for 256 rows.
//
// Work.  A unit is one key tile of one (sequence, KV head, row-tile pair) item.  All units of the
// call, in that order, are cut into equal contiguous ranges, one per CTA (one CTA per SM), from the
// lengths on the device: ragged caches balance, and a long cache of a single sequence covers every
// SM.  An item that one CTA holds whole is written by it; the others leave (max, sum, unnormalised
// output) per range in the workspace, merged by tree_attn_merge_kernel.
//
// Roles of a CTA (NT row tiles): warps 0 .. 4 NT - 1 softmax and output, one thread per query row
// (TMEM lane = row); then one thread each for the K loads (TMA), the MMAs (tcgen05) and the V loads.
// One row tile: two score buffers take the key tiles in turn, so the next tile's scores are formed
// while this one's weights are.  Two row tiles: each has its score buffer, and the two alternate.
// Scores and weights share columns of tensor memory: a row's 128 scores are read, and its weights
// written over them as two bf16 numbers each (w = hi + lo to 16 significant bits: with one bf16 the
// weights' rounding would equal the output's own), the A operands of two products with V.
//
// Rows that a slot does not see get weight 0 by a bit mask in the key tiles from L on; there, V rows
// that no token holds are zeroed in shared memory, and values that are no finite numbers are taken out
// and added, at the end, to the rows that see them (0 x inf would reach the others).
// Every wait is bounded (1 s): a timeout sets status bit 1 and the CTA stops.
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

constexpr int kRows = kTileKeys;  // query rows per tile = keys per key tile
constexpr uint32_t kTmemCols = 512;
constexpr int kHalf = kRows * 128;  // 64 columns of 128 rows of 16-bit values: one 128-byte swizzle span
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int NT>
struct Cfg {
  static constexpr int kSoftmax = 128 * NT;
  static constexpr int kThreads = kSoftmax + 96;
  static constexpr int kWarpK = 4 * NT, kWarpMMA = kWarpK + 1, kWarpV = kWarpK + 2;
  static constexpr int kTile = kHalf * (D / 64);
  // ring slots of K and of V: what 227 KB hold beside Q and the tree
  static constexpr int KS = D == 64 ? 4 : NT == 1 ? 3 : 2, VS = D == 64 ? 4 : 2;
  static constexpr int K_OFF = NT * kTile, V_OFF = K_OFF + KS * kTile, TREE_OFF = V_OFF + VS * kTile;
  static constexpr int BAR_OFF = (TREE_OFF + (int)sizeof(DraftTree) + 15) / 16 * 16;
  enum : int {
    B_QFULL = 0,               // [NT]
    B_KFULL = B_QFULL + NT,    // [KS]
    B_KEMPTY = B_KFULL + KS,   // [KS]
    B_VFULL = B_KEMPTY + KS,   // [VS]
    B_VEMPTY = B_VFULL + VS,   // [VS]
    B_SFULL = B_VEMPTY + VS,   // [2]: per score buffer
    B_PREADY = B_SFULL + 2,    // [2]
    B_PFREE = B_PREADY + 2,    // [NT]
    B_SYNC = B_PFREE + NT,     // the softmax warps among themselves
    B_DRAIN,
    kNBar
  };
  static constexpr int WALK_OFF = BAR_OFF + kNBar * 8;
  static constexpr int MISC_OFF = WALK_OFF + (int)sizeof(WalkShared<kThreads>);
  static constexpr int kSmem = MISC_OFF + 4 * (2 + 2 * kDraftWords) + 1024;  // + slack for the 1024-byte alignment
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static __host__ __device__ constexpr uint32_t col_o(int t) { return 256u + 128u * (uint32_t)t; }
};

// What the CTAs share with the merge: the unit ranges and the partial results.
struct Work {
  int64_t* prefix;  // [b + 1] key tiles of the sequences before; the total at the end
  float* part_o;    // [cta][2][NT * 128][D]
  float2* part_ml;  // [cta][2][NT * 128]: max (log2 domain), sum
};

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const uint16_t* __restrict__ q, const uint16_t* __restrict__ v,
                     const int32_t* __restrict__ kv_len, const int32_t* __restrict__ parent, uint16_t* __restrict__ o,
                     float* __restrict__ lse, Work work, int32_t* __restrict__ status, int batch, int T, int64_t n_kv, int H, int Hkv, float qscale) {
  using C = Cfg<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) { return sb + (uint32_t)C::BAR_OFF + 8u * (uint32_t)i; };
  DraftTree& tree = *reinterpret_cast<DraftTree*>(smem + C::TREE_OFF);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  uint32_t* tmem_slot = misc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  uint32_t* odd_rows = misc + 2;  // [2][kDraftWords]: drafted V rows with values that are not finite, per segment parity
  auto fail = [&]() {
    *abort_flag = 1;
    if (status) atomicOr(status, kStatusTimeout);
  };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == C::kWarpMMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < C::kNBar; ++i) {
      const bool soft = (i >= C::B_PREADY && i < C::B_PFREE) || (i >= C::B_QFULL && i < C::B_KFULL);
      mbar_init(bar(i), soft ? kRows : i == C::B_SYNC ? C::kSoftmax : 1);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (tid < 2 * kDraftWords) odd_rows[tid] = 0u;
  const int G = H / Hkv, R = T * G, np = (R + NT * kRows - 1) / (NT * kRows);  // items: (KV head, row-tile pair)
  tc_fence_before();
  Walk walk = walk_begin<C::kThreads>(kv_len, n_kv, T, batch, Hkv * np,
                                      *reinterpret_cast<WalkShared<C::kThreads>*>(smem + C::WALK_OFF), work.prefix, status);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == C::kWarpK || warp == C::kWarpV) {
    // ---------------- TMA producers ----------------
    if (lane == 0) {
      const bool is_k = warp == C::kWarpK;
      const CUtensorMap* map = is_k ? &map_k : &map_v;
      const int full = is_k ? C::B_KFULL : C::B_VFULL, empty = is_k ? C::B_KEMPTY : C::B_VEMPTY;
      const int NS = is_k ? C::KS : C::VS;
      const uint32_t base = sb + (uint32_t)(is_k ? C::K_OFF : C::V_OFF);
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
      int slot = 0, issued = 0;
      uint32_t phase = 1;  // parity of the slot's last release
      bool ok = true;
      while (ok && walk.next()) {
        const int g = walk.item / np;
        for (int x = 0; x < walk.n; ++x) {
          if (issued >= NS && !mbar_wait_or_abort(bar(empty + slot), phase, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          const uint32_t dst = base + (uint32_t)(slot * C::kTile);
          mbar_expect_tx(bar(full + slot), C::kTile);
#pragma unroll
          for (int h2 = 0; h2 < D / 64; ++h2)
            tma_load_4d(dst + h2 * kHalf, map, 64 * h2, g, (walk.j0 + x) * kRows, walk.s, bar(full + slot));
          ++issued;
          if (++slot == NS) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      // The copies in flight land before the CTA may exit.
      for (int x = max(0, issued - NS); x < issued; ++x) mbar_wait(bar(full + x % NS), (uint32_t)(x / NS) & 1u);
    }
  } else if (warp == C::kWarpMMA) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);  // Q and K both K-major
      constexpr uint32_t kIdO = idesc_bf16(128, D, false, true);     // weights (tensor memory), V MN-major
      bool ok = true;
      int kit = 0, vit = 0, seg = 0;  // K and V tiles taken so far, segments
      int cnt = 0;                    // key tiles multiplied so far (by each row tile that has rows)
      int cnt1 = 0;                   // the same of row tile B
      auto scores_of = [&](int t, int buf) {  // scores of row tile t and the K tile kit -> buffer buf
        const uint32_t kt = sb + (uint32_t)(C::K_OFF + (kit % C::KS) * C::kTile);
        const uint32_t qb = sb + (uint32_t)(t * C::kTile);
#pragma unroll
        for (int h2 = 0; h2 < D / 64; ++h2)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem + 128u * (uint32_t)buf, desc_kmajor_sw128(qb + h2 * kHalf + kk * 32),
                      desc_kmajor_sw128(kt + h2 * kHalf + kk * 32), kIdS, (h2 | kk) ? 1u : 0u);
        umma_commit(bar(C::B_SFULL + buf));
      };
      auto wait_k = [&]() {
        const bool r = mbar_wait_or_abort(bar(C::B_KFULL + kit % C::KS), (uint32_t)(kit / C::KS) & 1u, abort_flag);
        tc_fence_after();
        return r;
      };
      auto free_k = [&]() {
        umma_commit(bar(C::B_KEMPTY + kit % C::KS));
        ++kit;
      };
      auto output_of = [&](int t, int buf, bool first) {  // O_t += weights of buffer buf x V tile vit
        const uint32_t vt = sb + (uint32_t)(C::V_OFF + (vit % C::VS) * C::kTile);
#pragma unroll
        for (int part = 0; part < 2; ++part)  // the weights' high and low parts
#pragma unroll
          for (int kk = 0; kk < kRows / 16; ++kk)
            umma_bf16_ta(tmem + C::col_o(t), tmem + 128u * (uint32_t)buf + (uint32_t)(64 * part + 8 * kk),
                         desc_mnmajor_sw128(vt + kk * 2048, kHalf), kIdO, (!first || part || kk) ? 1u : 0u);
        umma_commit(bar(C::B_PFREE + t));
      };
      while (ok && walk.next()) {
        const int n = walk.n;
        if constexpr (NT == 1) {
          ok = mbar_wait_or_abort(bar(C::B_QFULL), (uint32_t)seg & 1u, abort_flag) && wait_k();
          if (!ok) break;
          tc_fence_after();
          scores_of(0, cnt & 1);
          free_k();
          for (int x = 0; ok && x < n; ++x, ++cnt) {
            const int buf = cnt & 1;
            if (x + 1 < n) {  // buffer buf ^ 1: its weights were multiplied with the V tile before
              ok = wait_k();
              if (!ok) break;
              scores_of(0, buf ^ 1);
              free_k();
            }
            ok = mbar_wait_or_abort(bar(C::B_VFULL + vit % C::VS), (uint32_t)(vit / C::VS) & 1u, abort_flag) &&
                 mbar_wait_or_abort(bar(C::B_PREADY + buf), (uint32_t)(cnt >> 1) & 1u, abort_flag);
            if (!ok) break;
            tc_fence_after();
            output_of(0, buf, x == 0);
            umma_commit(bar(C::B_VEMPTY + vit % C::VS));
            ++vit;
          }
        } else {
          const int pair = walk.item % np;
          const bool two = R - pair * 256 > kRows;
          ok = mbar_wait_or_abort(bar(C::B_QFULL), (uint32_t)seg & 1u, abort_flag) &&
               mbar_wait_or_abort(bar(C::B_QFULL + NT - 1), (uint32_t)seg & 1u, abort_flag) && wait_k();
          if (!ok) break;
          tc_fence_after();
          scores_of(0, 0);
          if (two) scores_of(1, 1);
          free_k();
          for (int x = 0; ok && x < n; ++x) {
            ok = mbar_wait_or_abort(bar(C::B_VFULL + vit % C::VS), (uint32_t)(vit / C::VS) & 1u, abort_flag) &&
                 mbar_wait_or_abort(bar(C::B_PREADY), (uint32_t)cnt & 1u, abort_flag);
            if (!ok) break;
            tc_fence_after();
            output_of(0, 0, x == 0);
            ++cnt;
            const bool more = x + 1 < n;
            if (more) {
              ok = wait_k();
              if (!ok) break;
              scores_of(0, 0);
            }
            if (two) {
              ok = mbar_wait_or_abort(bar(C::B_PREADY + 1), (uint32_t)cnt1 & 1u, abort_flag);
              if (!ok) break;
              tc_fence_after();
              output_of(NT - 1, 1, x == 0);
              ++cnt1;
              if (more) scores_of(1, 1);
            }
            umma_commit(bar(C::B_VEMPTY + vit % C::VS));
            ++vit;
            if (more) free_k();
          }
        }
        ++seg;
      }
      if (!ok) fail();
      umma_commit(bar(C::B_DRAIN));
      mbar_wait(bar(C::B_DRAIN), 0);
    }
  } else {
    // ---------------- softmax and output: warps 4 t .. 4 t + 3 row tile t, thread = query row ----------------
    const int t = warp >> 2;
    const int r = tid & (kRows - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lanes + C::col_o(t);
    const float lim = 8.f / qscale;
    const float2 qs2 = {qscale, qscale};
    bool ok = true;
    int cnt = 0, seg = 0;
    uint32_t sync_phase = 0;
    int vit = 0;  // V tiles so far
    auto sync = [&]() {
      mbar_arrive(bar(C::B_SYNC));
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_SYNC), sync_phase, abort_flag)) && ok;
      sync_phase ^= 1u;
    };
    while (ok && walk.next()) {
      const int64_t seq = walk.s;
      const int g = walk.item / np, pair = walk.item - g * np;
      const int L = (int)walk.L;
      const int base = pair * (NT * kRows) + t * kRows;  // first query row of the tile
      const int nr = min(kRows, R - base);                     // rows of the tile (none: below 1)
      // Q rows of the tile; the last use of its buffer ended with the segment before
      if (nr > 0) {
        const int fill = (nr + 31) & ~31;  // the rows of warps that take part
        constexpr int CH = D / 8;          // 16-byte chunks of a row
        for (int e = r; e < fill * CH; e += kRows) {
          const int row = e / CH, c = e % CH;
          const bool held = row < nr;
          const int i = (base + row) / G, hg = (base + row) - i * G;
          cp_async16(smem + t * C::kTile + (c >> 3) * kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                     held ? q + ((seq * T + i) * H + g * G + hg) * D + c * 8 : q, held);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_async_smem();
      }
      mbar_arrive(bar(C::B_QFULL + t));
      sync();  // the segment before is read out everywhere
      if (tid < kDraftWords) odd_rows[((seg + 1) & 1) * kDraftWords + tid] = 0u;
      uint32_t* odd = odd_rows + (seg & 1) * kDraftWords;
      if (parent) {
        if (draft_tree_build<C::kSoftmax>(tree, parent + seq * T, T, tid, sync) && status)
          atomicOr(status, kStatusBadIndex);
      }
      if (!ok) break;
      ++seg;
      if (nr <= 0) {  // this row tile has no rows here
        vit += walk.n;
        continue;
      }
      const int slot_i = min(base + r, R - 1) / G;  // drafted token of this row
      const bool token = !parent || tree.up[slot_i] == kRoot;
      const bool warp_rows = (warp & 3) * 32 < nr;  // the warp has rows
      float m_run = -INFINITY;                      // running max of the row's scores
      float2 l2 = {0.f, 0.f};                       // sum of the row's weights, relative to m_run
      for (int x = 0; x < walk.n; ++x, ++cnt, ++vit) {
        const int buf = NT == 2 ? t : cnt & 1;
        const uint32_t par = (uint32_t)(NT == 2 ? cnt : cnt >> 1) & 1u;
        const uint32_t ts = tmem + lanes + 128u * (uint32_t)buf;
        const int t0 = (walk.j0 + x) * kRows;
        const bool tail = t0 + kRows > L;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_SFULL + buf), par, abort_flag));
        if (!ok) break;
        tc_fence_after();
        if (tail && t == 0) {
          // V rows behind the context: thread = row of the V tile.  The scores are in, so the V tile two
          // before has been multiplied and the wait below cannot take an earlier fill of the slot for this one.
          const int vs = vit % C::VS;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_VFULL + vs), (uint32_t)(vit / C::VS) & 1u, abort_flag));
          if (!ok) break;
          const int j = t0 + r - L;
          if (j >= 0) {
            uint8_t* row = smem + C::V_OFF + vs * C::kTile + r * 128;
            const bool held = j < T && (!parent || tree.up[j] == kRoot);
            bool any = false;
#pragma unroll 1
            for (int c = 0; c < D / 8; ++c) {
              uint4* p = reinterpret_cast<uint4*>(row + (c >> 3) * kHalf + (c & 7) * 16);
              uint4 w = *p;
              uint32_t* a = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((a[e] & 0x7F80u) == 0x7F80u) {
                  a[e] &= 0xFFFF0000u;
                  any = true;
                }
                if ((a[e] & 0x7F800000u) == 0x7F800000u) {
                  a[e] &= 0xFFFFu;
                  any = true;
                }
                if (!held) a[e] = 0u;
              }
              if (any || !held) *p = w;
            }
            if (held && any) atomicOr(&odd[j >> 5], 1u << (j & 31));
          }
          fence_async_smem();
        }
        if (warp_rows) {
          uint32_t raw[4][32];
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) tmem_ld32_issue(ts + (uint32_t)(32 * c4), raw[c4]);
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) tmem_wait_ld(raw[c4]);
          if (tail) {
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) {
              const int off = t0 + 32 * c4 - L;
              const uint32_t w = parent ? mask_word(tree.anc[slot_i], off) : chain_word(slot_i, off);
#pragma unroll
              for (int c = 0; c < 32; ++c) raw[c4][c] = ((w >> c) & 1u) ? raw[c4][c] : 0xFF800000u;  // -inf
            }
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4)
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              m4[(c >> 1) & 3] = fmax3(m4[(c >> 1) & 3], __uint_as_float(raw[c4][c]), __uint_as_float(raw[c4][c + 1]));
          const float tmax = fmax3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
          // the max moves only when a weight would exceed 2^8
          const bool raise = tmax > m_run + lim;  // also the first visible key of the row (m_run = -inf)
          float alpha = 1.f;
          bool resc = false;
          if (raise) {
            if (m_run != -INFINITY) {
              alpha = exp2f((m_run - tmax) * qscale);
              l2.x *= alpha;
              l2.y *= alpha;
              resc = true;
            }
            m_run = tmax;
          }
          const float nmq = m_run == -INFINITY ? 0.f : -m_run * qscale;
          const float2 nmq2 = {nmq, nmq};
          // the weights over the scores: pairs (2 i, 2 i + 1), high parts in columns 0-63, low parts in 64-127
          float2 ls[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 e = ffma2(make_float2(__uint_as_float(raw[c4][2 * i]), __uint_as_float(raw[c4][2 * i + 1])),
                                     qs2, nmq2);
              const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));  // 0 where masked
              ls[i & 1] = fadd2(ls[i & 1], p);
              hi[i] = pack_bf16(p.x, p.y);
              lo[i] = pack_bf16(p.x - bf16_lo(hi[i]), p.y - bf16_hi(hi[i]));
            }
            tmem_st16_issue(ts + (uint32_t)(16 * c4), hi);
            tmem_st16_issue(ts + (uint32_t)(64 + 16 * c4), lo);
          }
          l2 = fadd2(l2, fadd2(ls[0], ls[1]));
          if (__any_sync(0xFFFFFFFFu, resc)) {  // O holds earlier tiles (x > 0): rescale it once they are in
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_PFREE + t), (uint32_t)(cnt - 1) & 1u, abort_flag))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t ov[16];
              tmem_ld<16>(to + c, ov);
#pragma unroll
              for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
              tmem_st16_issue(to + c, ov);
            }
          }
          tmem_wait_st();
        }
        // Two score buffers: these scores say only that the product before the last one is in.  The wait
        // behind the segment's last tile can tell its product from that of the tile before alone, so
        // that one is waited for here.
        if (NT == 1 && x + 1 == walk.n && cnt > 0) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_PFREE + t), (uint32_t)(cnt - 1) & 1u, abort_flag));
          if (!ok) break;
        }
        tc_fence_before();
        mbar_arrive(bar(C::B_PREADY + buf));
      }
      if (!ok) break;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar(C::B_PFREE + t), (uint32_t)(cnt - 1) & 1u, abort_flag));
      if (!ok) break;
      tc_fence_after();
      if (!warp_rows) continue;
      float l = l2.x + l2.y;
      if (!token) {
        l = 0.f;
        m_run = -INFINITY;
      }
      const bool whole = walk.whole();
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const int64_t row = (seq * T + slot_i) * H + g * G + (base + r - slot_i * G);
      const int64_t prow = ((int64_t)blockIdx.x * 2 + walk.slot()) * (NT * kRows) + t * kRows + r;
      const uint32_t any_odd = odd[0] | odd[1] | odd[2] | odd[3] | odd[4] | odd[5] | odd[6] | odd[7];
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t ov[32];
        __syncwarp();  // the load below takes the whole warp
        tmem_ld32_issue(to + c0, ov);
        tmem_wait_ld(ov);
        if (r >= nr) continue;
        if (l == 0.f) {
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = 0u;
        }
        if (any_odd && token) {
          // values that are not finite, of the rows this token sees in this segment
#pragma unroll 1
          for (int j = 0; j < T; ++j) {
            if (!((odd[j >> 5] >> (j & 31)) & 1u)) continue;
            if (parent ? !((tree.anc[slot_i][j >> 5] >> (j & 31)) & 1u) : j > slot_i) continue;
            const uint32_t* vr = reinterpret_cast<const uint32_t*>(v + (((seq * n_kv + L + j) * Hkv) + g) * D + c0);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t w = vr[i];
              if ((w & 0x7F80u) == 0x7F80u) ov[2 * i] = __float_as_uint(__uint_as_float(ov[2 * i]) + bf16_lo(w));
              if ((w & 0x7F800000u) == 0x7F800000u)
                ov[2 * i + 1] = __float_as_uint(__uint_as_float(ov[2 * i + 1]) + bf16_hi(w));
            }
          }
        }
        if (whole) {
          uint16_t* orow = o + row * D + c0;
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            uint4 w;
            w.x = pack_bf16(__uint_as_float(ov[8 * q4 + 0]) * inv, __uint_as_float(ov[8 * q4 + 1]) * inv);
            w.y = pack_bf16(__uint_as_float(ov[8 * q4 + 2]) * inv, __uint_as_float(ov[8 * q4 + 3]) * inv);
            w.z = pack_bf16(__uint_as_float(ov[8 * q4 + 4]) * inv, __uint_as_float(ov[8 * q4 + 5]) * inv);
            w.w = pack_bf16(__uint_as_float(ov[8 * q4 + 6]) * inv, __uint_as_float(ov[8 * q4 + 7]) * inv);
            *reinterpret_cast<uint4*>(orow + 8 * q4) = w;
          }
        } else {
          float* prt = work.part_o + prow * D + c0;
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(prt + i) = make_uint4(ov[i], ov[i + 1], ov[i + 2], ov[i + 3]);
        }
      }
      __syncwarp();
      if (r < nr) {
        if (!whole)
          work.part_ml[prow] = make_float2(m_run == -INFINITY ? -INFINITY : m_run * qscale, l);
        else if (lse)
          lse[row] = l == 0.f ? -INFINITY : (m_run * qscale + log2f(l)) * kLn2;
      }
    }
    if (!ok && lane == 0) fail();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarpMMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

// Rows whose item several CTAs hold: the parts joined; rows of sequences whose length is out of
// range: 0 and -inf.  SPLIT = false: a warp per row takes the parts one after another (items on few
// CTAs each); true: a CTA per row, its warps share the parts (few items, each on many CTAs).
constexpr int kMergeThreads = 256;
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kMergeThreads)
    tree_attn_merge_kernel(Work work, uint16_t* __restrict__ o,
                           float* __restrict__ lse, int batch, int T, int H, int Hkv, int tile_rows, int grid) {
  constexpr int NW = kMergeThreads / 32, LN = D / 4, PER = 32 / LN;  // lanes of a row, parts a warp takes at once
  __shared__ float sm_l[NW], sm_m[NW];
  __shared__ float4 sm_o[NW][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t seq = blockIdx.y;
  const int idx = SPLIT ? (int)blockIdx.x : (int)blockIdx.x * NW + warp;  // i * H + h
  if (idx >= T * H) return;
  const int i = idx / H, h = idx - i * H, G = H / Hkv, g = h / G;
  const int rr = i * G + (h - g * G), pair = rr / tile_rows, R = T * G, np = (R + tile_rows - 1) / tile_rows;
  const int64_t P = work.prefix[seq], tiles = work.prefix[seq + 1] - P, total = work.prefix[batch];
  const int64_t row = seq * T * H + idx;
  const int c = lane % LN, sub = lane / LN;
  if (tiles == 0) {
    if (SPLIT && warp != 0) return;
    if (sub == 0) *reinterpret_cast<uint2*>(o + row * D + 4 * c) = make_uint2(0u, 0u);
    if (lane == 0 && lse) lse[row] = -INFINITY;
    return;
  }
  const int64_t units = total * Hkv * np, ctas = range_ctas(units, grid);
  const int64_t u0 = P * Hkv * np + ((int64_t)g * np + pair) * tiles;
  const int64_t c0 = range_of(u0, units, ctas), c1 = range_of(u0 + tiles - 1, units, ctas);
  if (c0 == c1) return;
  const int n = (int)(c1 - c0) + 1;
  const int first_slot = range_begin(c0, units, ctas) == u0 ? 0 : 1;
  auto part_row = [&](int p) {
    return ((c0 + p) * 2 + (p == 0 ? first_slot : 0)) * (int64_t)tile_rows + (rr - pair * tile_rows);
  };
  const int p0 = SPLIT ? warp : 0, step = SPLIT ? NW : 1;
  // max and sum over the warp's parts, then over the warps'
  float m = -INFINITY, l = 0.f;
  for (int p = p0 + step * lane; p < n; p += step * 32) {
    const float2 ml = work.part_ml[part_row(p)];
    const float mn = fmaxf(m, ml.x);
    l = l * (m == -INFINITY ? 0.f : exp2f(m - mn)) + ml.y * (ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - mn));
    m = mn;
  }
  const float M = warp_max(m);
  l = warp_sum(l * (m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2f(m - M)));
  float4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int p = p0 + step * sub; p < n; p += step * PER) {
    const int64_t pr = part_row(p);
    const float2 ml = work.part_ml[pr];
    const float4 x = *reinterpret_cast<const float4*>(work.part_o + pr * D + 4 * c);
    if (ml.y == 0.f) continue;  // nothing visible there
    const float w = ml.x == -INFINITY ? 1.f : exp2f(ml.x - M);
    acc.x += w * x.x;
    acc.y += w * x.y;
    acc.z += w * x.z;
    acc.w += w * x.w;
  }
  if constexpr (PER == 2) {
    acc.x += __shfl_xor_sync(0xFFFFFFFFu, acc.x, 16);
    acc.y += __shfl_xor_sync(0xFFFFFFFFu, acc.y, 16);
    acc.z += __shfl_xor_sync(0xFFFFFFFFu, acc.z, 16);
    acc.w += __shfl_xor_sync(0xFFFFFFFFu, acc.w, 16);
  }
  float top = M;
  if constexpr (SPLIT) {
    if (lane == 0) {
      sm_m[warp] = M;
      sm_l[warp] = l;
    }
    sm_o[warp][lane] = acc;
    __syncthreads();
    if (warp != 0) return;
    top = -INFINITY;
    for (int w = 0; w < NW; ++w) top = fmaxf(top, sm_m[w]);
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < NW; ++w) {
      if (sm_l[w] == 0.f) continue;
      const float a = sm_m[w] == -INFINITY ? 1.f : exp2f(sm_m[w] - top);
      const float4 x = sm_o[w][lane];
      l += a * sm_l[w];
      acc.x += a * x.x;
      acc.y += a * x.y;
      acc.z += a * x.z;
      acc.w += a * x.w;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (sub == 0)
    *reinterpret_cast<uint2*>(o + row * D + 4 * c) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (lane == 0 && lse) lse[row] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
}

int row_tiles(const Shape& s) { return s.n_q * (s.H / s.Hkv) > kRows ? 2 : 1; }

struct Layout {
  size_t prefix, part_o, part_ml, lse, weight, total;
};
Layout layout(const Shape& s, bool with_weight) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = (size_t)kMaxCtas * 2 * row_tiles(s) * kRows;
  Layout L;
  L.prefix = 0;
  L.part_o = up((size_t)(s.batch + 1) * sizeof(int64_t));
  L.part_ml = L.part_o + up(rows * s.d * sizeof(float));
  L.lse = L.part_ml + up(rows * sizeof(float2));
  L.weight = L.lse + (with_weight ? up((size_t)s.n_query * s.H * sizeof(float)) : 0);
  L.total = L.weight;
  if (with_weight) L.total += up(cache_weight_workspace_bytes(s));
  return L;
}

template <int D, int NT>
cudaError_t launch(const Shape& s, const void* q, const void* k, const void* v, const int32_t* kv_len,
                   const int32_t* parent, void* o, float* lse, Work work, int32_t* status, cudaStream_t st) {
  using C = Cfg<D, NT>;
  CUtensorMap mk, mv;
  if (!map_cache_rows(&mk, k, D, (uint64_t)s.Hkv, (uint64_t)s.n_kv, (uint64_t)s.batch, kRows) ||
      !map_cache_rows(&mv, v, D, (uint64_t)s.Hkv, (uint64_t)s.n_kv, (uint64_t)s.batch, kRows))
    return cudaErrorNotSupported;
  cudaError_t e = ensure_smem((const void*)tree_attn_kernel<D, NT>, C::kSmem);
  if (e != cudaSuccess) return e;
  const int R = (int)s.n_q * (s.H / s.Hkv), np = (R + NT * kRows - 1) / (NT * kRows);
  const int64_t items = (int64_t)s.batch * s.Hkv * np, most = items * ((s.n_kv + kRows - 1) / kRows);
  const int ctas = (int)(most < kMaxCtas ? most : kMaxCtas);
  tree_attn_kernel<D, NT><<<ctas, C::kThreads, C::kSmem, st>>>(
      mk, mv, static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(v), kv_len, parent,
      static_cast<uint16_t*>(o), lse, work, status, s.batch, (int)s.n_q, s.n_kv, s.H, s.Hkv,
      s.scale * kLog2e);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // a CTA per row where an item's parts are many, or where the rows are so few that one wave of CTAs
  // takes them all
  const bool split = items * 16 < ctas || (items * 4 < ctas && s.n_query * s.H <= 8 * kMaxCtas);
  const int rows = (int)s.n_q * s.H, per = split ? 1 : kMergeThreads / 32;
  return launch_after(split ? tree_attn_merge_kernel<D, true> : tree_attn_merge_kernel<D, false>,
                      dim3((unsigned)((rows + per - 1) / per), (unsigned)s.batch), kMergeThreads, st, work,
                      static_cast<uint16_t*>(o), lse, s.batch, (int)s.n_q, s.H, s.Hkv, NT * kRows, ctas);
}

}  // namespace

size_t tree_attn_workspace_bytes(const Shape& s, bool with_weight) { return layout(s, with_weight).total; }

cudaError_t launch_tree_attn(const Shape& s, const void* q, const void* k, const void* v, const int32_t* kv_len,
                             const int32_t* parent, void* o, float* lse, float* weight, int32_t* status, void* ws,
                             cudaStream_t st) {
  const Layout L = layout(s, weight != nullptr);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const Work work = {reinterpret_cast<int64_t*>(w + L.prefix), reinterpret_cast<float*>(w + L.part_o),
                     reinterpret_cast<float2*>(w + L.part_ml)};
  if (weight && !lse) lse = reinterpret_cast<float*>(w + L.lse);
  const auto run = s.d == 64 ? (row_tiles(s) == 1 ? launch<64, 1> : launch<64, 2>)
                             : (row_tiles(s) == 1 ? launch<128, 1> : launch<128, 2>);
  const cudaError_t e = run(s, q, k, v, kv_len, parent, o, lse, work, status, st);
  if (e != cudaSuccess || !weight) return e;
  return launch_cache_weight(s, q, k, kv_len, parent, nullptr, lse, weight, nullptr, w + L.weight, st);
}

}  // namespace hisa
