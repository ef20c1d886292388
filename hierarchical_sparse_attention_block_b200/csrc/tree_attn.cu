// hisa_tree_attn_fwd: attention of drafted tokens over a cache, on the 5th-generation tensor cores.
//
//   z(t) = scale q[i,h].k[t,g],  lse = ln sum_{t in V(i)} e^z(t),  o = sum_{t in V(i)} e^(z(t) - lse) v[t,g],
//   V(i) = the context's rows [0, L) and the drafted rows L + j of i's ancestors and itself.
//
// The T tokens of a sequence and the G = H / Hk heads of one KV head make R = T G query rows that
// read the same K and V.  With few rows the call is bound by the cache's bytes, with many (R above
// about 128) by the tensor cores.  Up to 16 rows are tree_attn_few.cu's; here tiles of 128 query rows
// (padded) meet tiles of 128 keys.  A tile of 128 x 128 costs the tensor cores about half the time that
// its K and V take from HBM, so the padding of 17 to 128 rows costs little; R above 128 puts two row
// tiles on one CTA, which then reads every K/V tile once for 256 rows.
//
// Work.  A unit is one key tile of one (sequence, KV head, row-tile pair) item.  All units of the
// call, in that order, are cut into equal contiguous ranges, one per CTA (one CTA per SM), from the
// lengths on the device: ragged caches balance, and a long cache of a single sequence covers every
// SM.  An item that one CTA holds whole is written by it; the others leave (max, sum, unnormalised
// output) per range in the workspace, merged by tree_attn_merge_kernel.
//
// Roles of a CTA: two softmax groups of four warps, one thread per query row (TMEM lane = row); then
// one thread each for the K loads (TMA), the MMAs (tcgen05) and the V loads.  Two row tiles: each
// group has its tile.  One row tile: the groups take the key tiles in turn, each with its own running
// max, sum and output, joined at the segment's end; a group's softmax takes longer than a tile's
// bytes, two side by side do not.  Either way a group's scores of the next tile follow the product with
// its weights of this one, and one group's products run while the other's weights are formed.
// Scores and weights share columns of tensor memory: a row's scores are read 32 at a time, and its
// weights written over them, as bf16: rounding the weights to 8 bits moves an output of n comparable
// weights by about as much as its own rounding to bf16 does; a second product with the weights' low
// parts took a quarter of the call (16 x 32K rows, 128 query rows a KV head: 210 us with it, 161
// without).
//
// Rows that a slot does not see get weight 0 by a bit mask in the key tiles from L on; there, V rows
// that no token holds are zeroed in shared memory, and values that are no finite numbers are taken out
// and added, at the end, to the rows that see them (0 x inf would reach the others).
// Every wait is bounded (1 s): a timeout sets status bit 1 and the CTA stops.
#include <math.h>

#include "row_ref.h"
#include "tree_attn.cuh"

namespace hisa {
namespace {

using namespace tc;

constexpr uint32_t kTmemCols = 512;

// What another item costs a CTA, in key tiles (a tile takes about 1.5 us with one row tile, 2.5 with two).
template <int NT>
constexpr int kLead = NT == 1 ? 5 : 6;
constexpr int kSoftmax = 256;  // two groups
constexpr int kThreads = kSoftmax + 96;
constexpr int kWarpK = 8, kWarpMMA = 9, kWarpV = 10;
// Tensor memory: scores / weights of group t at 128 t, its output at col_o(t).
__host__ __device__ constexpr uint32_t col_o(int t) { return 256u + 128u * (uint32_t)t; }

// NT: row tiles of an item.
template <int D, int NT>
struct Cfg {
  static constexpr int kTile = kHalf * (D / 64);
  // ring slots of K and of V: what 227 KB hold beside Q and the tree
  static constexpr int KS = D == 64 ? 5 : NT == 1 ? 3 : 2, VS = D == 64 ? 4 : 2;
  static constexpr int K_OFF = NT * kTile, V_OFF = K_OFF + KS * kTile, TREE_OFF = V_OFF + VS * kTile;
  static constexpr int JOIN_OFF = (TREE_OFF + (int)sizeof(DraftTree) + 15) / 16 * 16;  // float2 [2][kRows]
  static constexpr int BAR_OFF = JOIN_OFF + 2 * kRows * (int)sizeof(float2);
  enum : int {
    B_QFULL = 0,
    B_KFULL,                   // [KS]
    B_KEMPTY = B_KFULL + KS,   // [KS]
    B_VFULL = B_KEMPTY + KS,   // [VS]
    B_VEMPTY = B_VFULL + VS,   // [VS]
    B_SFULL = B_VEMPTY + VS,   // [2]: per group
    B_PREADY = B_SFULL + 2,    // [2]
    B_PFREE = B_PREADY + 2,    // [2]
    B_SYNC = B_PFREE + 2,      // the softmax warps among themselves
    B_GO,                      // the first segment's query rows are asked for
    B_DRAIN,
    kNBar
  };
  static constexpr int WALK_OFF = BAR_OFF + kNBar * 8;
  static constexpr int MISC_OFF = WALK_OFF + (int)sizeof(WalkShared<kThreads>);
  static constexpr int kSmem = MISC_OFF + 4 * (2 + 2 * kDraftWords) + 1024;  // + slack for the 1024-byte alignment
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ TreeArgs args) {
  const int32_t* const parent = args.parent;
  int32_t* const status = args.status;
  const Work& work = args.work;
  const int T = args.T, H = args.H, Hkv = args.Hkv;
  const int64_t n_kv = args.n_kv;
  const float qscale = args.qscale;
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
  uint32_t* odd_rows = misc + 2;  // [2][kDraftWords] by segment parity: drafted V rows not all finite
  auto fail = [&]() {
    *abort_flag = 1;
    if (status) atomicOr(status, kStatusTimeout);
  };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == kWarpMMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < C::kNBar; ++i) {
      const bool group = i >= C::B_PREADY && i < C::B_PFREE;
      mbar_init(bar(i), group ? kRows : i == C::B_SYNC || i == C::B_QFULL || i == C::B_GO ? kSoftmax : 1);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (tid < 2 * kDraftWords) odd_rows[tid] = 0u;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what the kernels before wrote, and read of the workspace
  const int G = H / Hkv, R = T * G, np = (R + NT * kRows - 1) / (NT * kRows);  // items: (KV head, row-tile pair)
  tc_fence_before();
  Walk walk = walk_begin<kThreads>(args.kv_len, n_kv, T, args.batch, Hkv * np, kLead<NT>,
                                   *reinterpret_cast<WalkShared<kThreads>*>(smem + C::WALK_OFF), work.prefix,
                                   status);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kWarpK || warp == kWarpV) {
    // ---------------- TMA producers ----------------
    if (lane == 0) {
      const bool is_k = warp == kWarpK;
      const CUtensorMap* map = is_k ? &map_k : &map_v;
      const int full = is_k ? C::B_KFULL : C::B_VFULL, empty = is_k ? C::B_KEMPTY : C::B_VEMPTY;
      const int NS = is_k ? C::KS : C::VS;
      const uint32_t base = sb + (uint32_t)(is_k ? C::K_OFF : C::V_OFF);
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
      // K and V pass through the L2 once, unless several row-tile pairs read them
      const uint64_t policy = np > 1 ? l2_evict_normal() : l2_evict_first();
      int slot = 0, issued = 0;
      uint32_t phase = 1;  // parity of the slot's last release
      bool ok = true;
      while (ok && walk.next()) {
        const int g = walk.item / np;
        for (int x = 0; x < walk.n; ++x) {
          // The query rows go first: behind the first tiles of every SM they would wait for all of those.  (A CTA
          // whose units hold no tile has none, and asks for none.)
          if ((issued == 0 && !mbar_wait_or_abort(bar(C::B_GO), 0, abort_flag)) ||
              (issued >= NS && !mbar_wait_or_abort(bar(empty + slot), phase, abort_flag))) {
            fail();
            ok = false;
            break;
          }
          const uint32_t dst = base + (uint32_t)(slot * C::kTile);
          mbar_expect_tx(bar(full + slot), C::kTile);
#pragma unroll
          for (int h2 = 0; h2 < D / 64; ++h2)
            tma_load_4d(dst + h2 * kHalf, map, 64 * h2, g, (walk.j0 + x) * kRows, walk.s, bar(full + slot), policy);
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
  } else if (warp == kWarpMMA) {
    // ---------------- MMA issuer ----------------
    {
      auto waited = [&](uint32_t barrier, uint32_t parity) {
        return warp_wait_or_abort(barrier, parity, abort_flag);
      };
      constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);  // Q and K both K-major
      constexpr uint32_t kIdO = idesc_bf16(128, D, false, true);     // weights (tensor memory), V MN-major
      bool ok = true;
      int kit = 0, vit = 0, seg = 0;  // K and V tiles taken so far, segments
      int cnt[2] = {0, 0};            // products with the weights of each group
      auto wait_k = [&]() {
        const bool r = waited(bar(C::B_KFULL + kit % C::KS), (uint32_t)(kit / C::KS) & 1u);
        tc_fence_after();
        return r;
      };
      auto scores_of = [&](int t) {  // group t's scores with the K tile kit
        const uint32_t kt = sb + (uint32_t)(C::K_OFF + (kit % C::KS) * C::kTile);
        const uint32_t qb = sb + (uint32_t)(NT == 2 ? t * C::kTile : 0);
        if (elect_one()) {
#pragma unroll
          for (int h2 = 0; h2 < D / 64; ++h2)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16(tmem + 128u * (uint32_t)t, desc_kmajor_sw128(qb + h2 * kHalf + kk * 32),
                        desc_kmajor_sw128(kt + h2 * kHalf + kk * 32), kIdS, (h2 | kk) ? 1u : 0u);
          umma_commit(bar(C::B_SFULL + t));
        }
      };
      auto free_k = [&]() {
        if (elect_one()) umma_commit(bar(C::B_KEMPTY + kit % C::KS));
        ++kit;
      };
      auto output_of = [&](int t, bool first) {  // O_t += group t's weights x the V tile vit
        const uint32_t vt = sb + (uint32_t)(C::V_OFF + (vit % C::VS) * C::kTile);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kRows / 16; ++kk)
            umma_bf16_ta(tmem + col_o(t), tmem + 128u * (uint32_t)t + (uint32_t)(32 * (kk >> 1) + 8 * (kk & 1)),
                         desc_mnmajor_sw128(vt + kk * 2048, kHalf), kIdO, (!first || kk) ? 1u : 0u);
          umma_commit(bar(C::B_PFREE + t));
        }
        ++cnt[t];
      };
      auto wait_weights = [&](int t) {
        const bool r = waited(bar(C::B_PREADY + t), (uint32_t)cnt[t] & 1u);
        tc_fence_after();
        return r;
      };
      auto wait_v = [&]() {
        return waited(bar(C::B_VFULL + vit % C::VS), (uint32_t)(vit / C::VS) & 1u);
      };
      auto free_v = [&]() {
        if (elect_one()) umma_commit(bar(C::B_VEMPTY + vit % C::VS));
        ++vit;
      };
      while (ok && walk.next()) {
        const int n = walk.n;
        ok = waited(bar(C::B_QFULL), (uint32_t)seg & 1u) && wait_k();
        ++seg;
        if (!ok) break;
        if constexpr (NT == 1) {
          // key tile x belongs to group x & 1
          scores_of(0);
          free_k();
          if (n > 1) {
            ok = wait_k();
            if (!ok) break;
            scores_of(1);
            free_k();
          }
          for (int x = 0; ok && x < n; x += 2)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok || x + t >= n) continue;
              ok = wait_v() && wait_weights(t);
              if (!ok) continue;
              output_of(t, x == 0);
              free_v();
              if (x + t + 2 < n) {
                ok = wait_k();
                if (!ok) continue;
                scores_of(t);
                free_k();
              }
            }
        } else {
          const int pair = walk.item % np;
          const bool two = R - pair * 256 > kRows;
          scores_of(0);
          if (two) scores_of(1);
          free_k();
          for (int x = 0; ok && x < n; ++x) {
            const bool more = x + 1 < n;
            ok = wait_v() && wait_weights(0);
            if (!ok) break;
            output_of(0, x == 0);
            if (more) {
              ok = wait_k();
              if (!ok) break;
              scores_of(0);
            }
            if (two) {
              ok = wait_weights(1);
              if (!ok) break;
              output_of(1, x == 0);
              if (more) scores_of(1);
            }
            free_v();
            if (more) free_k();
          }
        }
      }
      if (!ok && lane == 0) fail();
      if (elect_one()) umma_commit(bar(C::B_DRAIN));
      mbar_wait(bar(C::B_DRAIN), 0);
    }
  } else {
    // ---------------- softmax and output: group t = warps 4 t .. 4 t + 3, thread = query row ----------------
    const int t = warp >> 2;
    const int r = tid & (kRows - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 128u * (uint32_t)t;
    const float lim = rise_limit(qscale);
    float2* join = reinterpret_cast<float2*>(smem + C::JOIN_OFF);
    bool ok = true;
    int cnt = 0, seg = 0;  // key tiles of this group so far, segments
    int vit = 0;           // V tiles of the segments before
    uint32_t sync_phase = 0;
    auto sync = [&]() {
      mbar_arrive(bar(C::B_SYNC));
      ok = warp_wait_or_abort(bar(C::B_SYNC), sync_phase, abort_flag) && ok;
      sync_phase ^= 1u;
    };
    while (ok && walk.next()) {
      const int64_t seq = walk.s;
      const int g = walk.item / np, pair = walk.item - g * np;
      const int L = (int)walk.L;
      const int base = NT == 2 ? pair * 256 + t * kRows : 0;  // first query row of the group
      const int nr = min(kRows, R - base);                     // its rows (none: below 1)
      if (seg > 0) sync();  // the segment before is read out everywhere
      if (!ok) break;
      // Q rows, 16 bytes a copy, all in flight at once
      if (nr > 0) {
        constexpr int CH = D / 8;  // 16-byte chunks of a row; rows that hold no query are 0
        for (int e = NT == 2 ? r : tid; e < kRows * CH; e += NT == 2 ? kRows : kSoftmax) {
          const int row = e / CH, c = e % CH;
          const bool held = row < nr;
          const int i = (base + row) / G, hg = (base + row) - i * G;
          cp_async16(smem + (NT == 2 ? t * C::kTile : 0) + (c >> 3) * kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                     args.q + (held ? ((seq * T + i) * H + g * G + hg) * D + c * 8 : 0), held);
        }
        cp_async_commit();
      }
      if (seg == 0) mbar_arrive(bar(C::B_GO));
      cp_async_wait<0>();
      fence_async_smem();
      mbar_arrive(bar(C::B_QFULL));
      if (tid < kDraftWords) odd_rows[((seg + 1) & 1) * kDraftWords + tid] = 0u;
      uint32_t* odd = odd_rows + (seg & 1) * kDraftWords;
      const bool treed = parent && (walk.j0 + walk.n) * kRows > L;  // the segment reaches behind the context
      if (treed) {
        if (draft_tree_build<kSoftmax>(tree, parent + seq * T, T, tid, sync) && status)
          atomicOr(status, kStatusBadIndex);
      }
      if (!ok) break;
      ++seg;
      const int vit0 = vit;
      vit += walk.n;
      if (NT == 2 && nr <= 0) continue;  // this group has no rows here
      const int slot_i = min(base + r, R - 1) / G;  // drafted token of this row
      // an empty slot; where the segment ends within the context, the merge learns it from another part
      const bool empty = treed && tree.end[slot_i] != kRoot;
      const bool warp_rows = (r & ~31) < nr;        // the warp has rows
      float m_run = -INFINITY;                      // running max of the row's scores
      float2 l2 = {0.f, 0.f};                       // sum of the row's weights, relative to m_run
      bool any = false;                             // the group had a key tile
      const int ahead_at = max(0, (walk.n - 10) & ~1);
      for (int x = NT == 2 ? 0 : t; x < walk.n; x += NT == 2 ? 1 : 2, ++cnt) {
        const int t0 = (walk.j0 + x) * kRows;
        const bool tail = t0 + kRows > L;
        if (t == 0 && x == ahead_at) prefetch_next<D>(walk, args, np, NT * kRows, r);
        ok = warp_wait_or_abort(bar(C::B_SFULL + t), (uint32_t)cnt & 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (warp_rows) {
          // 32 columns at a time, the next load in flight: first the row's max, then, from the two blocks
          // that are still in registers on, the weights
          uint32_t xa[32], xb[32];
          auto issue = [&](int c4, uint32_t(&x)[32]) { tmem_ld32_issue(ts + (uint32_t)(32 * c4), x); };
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          auto mask = [&](int c4, uint32_t(&x)[32]) {
            if (!tail) return;
            const int off = t0 + 32 * c4 - L;
            const uint32_t w = parent ? mask_word(tree.anc[slot_i], off) : chain_word(slot_i, off);
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = ((w >> c) & 1u) ? x[c] : 0xFF800000u;  // -inf
          };
          auto look = [&](int c4, uint32_t(&x)[32]) {
            mask(c4, x);
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              m4[(c >> 1) & 3] = fmax3(m4[(c >> 1) & 3], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
          };
          issue(0, xa);
          tmem_wait_ld(xa);
          issue(1, xb);
          look(0, xa);
          tmem_wait_ld(xb);
          issue(2, xa);
          look(1, xb);
          tmem_wait_ld(xa);
          issue(3, xb);
          look(2, xa);
          tmem_wait_ld(xb);
          look(3, xb);
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
          const float m0 = m_run == -INFINITY ? 0.f : m_run, qs = row_scale(m0, qscale), nmq = -m0 * qs;
          const float2 qs2 = {qs, qs}, nmq2 = {nmq, nmq};
          // the weights of a block over its scores: pairs (2 i, 2 i + 1) in the block's first 16 columns
          float2 ls[2] = {{0.f, 0.f}, {0.f, 0.f}};
          auto weigh = [&](int c4, const uint32_t(&x)[32]) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 e = ffma2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), qs2, nmq2);
              const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));  // 0 where masked
              ls[i & 1] = fadd2(ls[i & 1], p);
              w[i] = pack_bf16(p.x, p.y);
            }
            tmem_st16_issue(ts + (uint32_t)(32 * c4), w);
          };
          weigh(2, xa);
          issue(0, xa);
          weigh(3, xb);
          tmem_wait_ld(xa);
          issue(1, xb);
          mask(0, xa);
          weigh(0, xa);
          tmem_wait_ld(xb);
          mask(1, xb);
          weigh(1, xb);
          l2 = fadd2(l2, fadd2(ls[0], ls[1]));
          if (__any_sync(0xFFFFFFFFu, resc)) {  // the group's output holds earlier tiles: rescale it once they are in
            if (!warp_wait_or_abort(bar(C::B_PFREE + t), (uint32_t)(cnt - 1) & 1u, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t ov[16];
              tmem_ld<16>(tmem + lanes + col_o(t) + c, ov);
#pragma unroll
              for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
              tmem_st16_issue(tmem + lanes + col_o(t) + c, ov);
            }
          }
          tmem_wait_st();
        }
        if (tail && (NT == 1 || t == 0)) {
          // V rows behind the context.  The scores are in, and with them this
          // group's product before, so the wait cannot take an earlier fill of the V slot for this one.
          const int vs = (vit0 + x) % C::VS;
          ok = warp_wait_or_abort(bar(C::B_VFULL + vs), (uint32_t)((vit0 + x) / C::VS) & 1u, abort_flag);
          if (!ok) break;
          clear_tail_values<D>(smem + C::V_OFF + vs * C::kTile, t0, L, T, parent != nullptr, tree, odd, r);
          fence_async_smem();
          __syncwarp();
        }
        tc_fence_before();
        mbar_arrive(bar(C::B_PREADY + t));
        any = true;
      }
      if (!ok) break;
      if (any) {
        ok = warp_wait_or_abort(bar(C::B_PFREE + t), (uint32_t)(cnt - 1) & 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
      }
      float l = l2.x + l2.y;
      float m = m_run == -INFINITY ? -INFINITY : m_run * qscale;  // log2 domain
      // What the row's two outputs count: w0 O_0 + w1 O_1; one row tile: both groups' key tiles joined, each
      // group taking half of the columns.
      int c0 = 0, c1 = D;
      float w0 = t == 0 ? 1.f : 0.f, w1 = t == 1 ? 1.f : 0.f;
      bool use0 = t == 0, use1 = t == 1;
      if constexpr (NT == 1) {
        join[t * kRows + r] = make_float2(m, l);
        tc_fence_before();
        sync();
        if (!ok) break;
        tc_fence_after();
        const float2 a = join[r], b = join[kRows + r];
        m = fmaxf(a.x, b.x);
        w0 = a.y == 0.f ? 0.f : a.x == -INFINITY ? 1.f : exp2f(a.x - m);
        w1 = b.y == 0.f ? 0.f : b.x == -INFINITY ? 1.f : exp2f(b.x - m);
        l = (w0 == 0.f ? 0.f : w0 * a.y) + (w1 == 0.f ? 0.f : w1 * b.y);
        use0 = true;
        use1 = walk.n > 1;
        c0 = t * (D / 2);
        c1 = c0 + D / 2;
      }
      if (empty) {
        l = 0.f;
        m = INFINITY;
      }
      const bool whole = walk.whole();
      const int64_t part = (int64_t)blockIdx.x * 2 + walk.slot();
      const uint32_t any_odd = odd[0] | odd[1] | odd[2] | odd[3] | odd[4] | odd[5] | odd[6] | odd[7];
      // Four columns of a row of this item: its slot, its sum.
      auto put = [&](int row, int c, float4 x, float sum) {
        const int i = (base + row) / G;
        if (sum == 0.f) x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (any_odd && !(treed && tree.end[i] != kRoot)) {
          // values that are not finite, of the rows this token sees in this segment
          for (int j = 0; j < T; ++j) {
            if (!((odd[j >> 5] >> (j & 31)) & 1u)) continue;
            if (!sees(tree, parent != nullptr, i, j)) continue;
            const uint2 y = *reinterpret_cast<const uint2*>(args.v + ((seq * n_kv + L + j) * Hkv + g) * D + c);
            if ((y.x & 0x7F80u) == 0x7F80u) x.x += bf16_lo(y.x);
            if ((y.x & 0x7F800000u) == 0x7F800000u) x.y += bf16_hi(y.x);
            if ((y.y & 0x7F80u) == 0x7F80u) x.z += bf16_lo(y.y);
            if ((y.y & 0x7F800000u) == 0x7F800000u) x.w += bf16_hi(y.y);
          }
        }
        if (whole) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const int64_t at = (seq * T + i) * H + g * G + (base + row - i * G);
          *reinterpret_cast<uint2*>(args.o + at * D + c) =
              make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
        } else {
          work.part_o[(part * (D / 4) + c / 4) * (NT * kRows) + (NT == 2 ? t * kRows : 0) + row] = x;
        }
      };
      auto read16 = [&](int c, float(&ov)[16]) {  // 16 columns of this lane's share; the whole warp calls
        uint32_t x0[16], x1[16];
        __syncwarp();
        if (use0) tmem_ld<16>(tmem + lanes + col_o(0) + c, x0);
        if (use1) tmem_ld<16>(tmem + lanes + col_o(1) + c, x1);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          // an output that saw nothing is left out: it may hold 0 x inf
          ov[i] = use0 && w0 != 0.f ? w0 * __uint_as_float(x0[i]) : 0.f;
          if (use1 && w1 != 0.f) ov[i] = fmaf(w1, __uint_as_float(x1[i]), ov[i]);
        }
      };
      if (warp_rows) {
#pragma unroll 1
        for (int c = c0; c < c1; c += 16) {
          float ov[16];
          read16(c, ov);
          if (r < nr) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) put(r, c + i, make_float4(ov[i], ov[i + 1], ov[i + 2], ov[i + 3]), l);
          }
        }
      }
      __syncwarp();
      if (r < nr && (NT == 2 || t == 0)) {
        if (!whole)
          work.part_ml[part * (NT * kRows) + (NT == 2 ? t * kRows : 0) + r] = make_float2(m, l);
        else if (args.lse)
          args.lse[(seq * T + slot_i) * H + g * G + (base + r - slot_i * G)] =
              l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
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

// Rows whose item several CTAs hold: the parts joined; rows of sequences whose length is out of
// range: 0 and -inf.  A CTA takes up to 32 rows of an item: lane = row, and where the item has fewer
// rows the lanes share its parts; a warp takes 16 columns, and kSplits sets of warps share the parts.
constexpr int kSplits = 4;
struct MergeState {
  float m, l;
  float o[16];
  bool empty;
  __device__ void add(float m2, float l2, const float* o2) {
    if (l2 == 0.f) return;
    const float top = fmaxf(m, m2);
    const float a = l == 0.f ? 0.f : m == -INFINITY ? 1.f : exp2f(m - top), b = m2 == -INFINITY ? 1.f : exp2f(m2 - top);
    m = top;
    l = a * l + b * l2;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = (a == 0.f ? 0.f : a * o[i]) + b * o2[i];
  }
};
template <int D>
__global__ void __launch_bounds__(32 * (D / 16) * kSplits)
    tree_attn_merge_kernel(Work work, uint16_t* __restrict__ o, float* __restrict__ lse, int batch, int T, int H,
                           int Hkv, int tile_rows, int row_lanes, int grid) {
  constexpr int CW = D / 16;  // warps side by side
  __shared__ float sm_ml[kSplits / 2][CW][32][2];
  __shared__ float4 sm_o[kSplits / 2][CW][4][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cw = warp % CW, split = warp / CW;
  const int64_t seq = blockIdx.y;
  const int G = H / Hkv, R = T * G, np = (R + tile_rows - 1) / tile_rows, blocks = (R + row_lanes - 1) / row_lanes;
  const int g = blockIdx.x / blocks, r = (blockIdx.x - g * blocks) * row_lanes + lane % row_lanes;  // query row
  const int pair = (blockIdx.x - g * blocks) * row_lanes / tile_rows;  // row_lanes divides tile_rows
  const int64_t P = work.prefix[seq], length = work.prefix[seq + 1] - P, total = work.prefix[batch];
  const int i = r / G;
  const int64_t row = (seq * T + i) * H + g * G + (r - i * G);
  const bool mine = r < R && lane < row_lanes && split == 0;  // writes the row
  MergeState st;
  st.m = -INFINITY;
  st.l = 0.f;
  st.empty = false;
#pragma unroll
  for (int x = 0; x < 16; ++x) st.o[x] = 0.f;
  if (length > 0) {
    const int64_t units = total * Hkv * np, ctas = range_ctas(units, grid);
    const int64_t u0 = P * Hkv * np + ((int64_t)g * np + pair) * length;
    // the CTAs that hold the item's first and last tile
    const int64_t first = range_of(u0 + work.prefix[batch + 1], units, ctas);
    const int64_t last = range_of(u0 + length - 1, units, ctas);
    if (first == last) return;  // written by that CTA
    const int n = (int)(last - first) + 1;
    const int first_slot = range_begin(first, units, ctas) >= u0 ? 0 : 1;
    const int groups = 32 / row_lanes * kSplits, pr = min(r, R - 1) - pair * tile_rows;
#pragma unroll 2
    for (int p = split * (32 / row_lanes) + lane / row_lanes; p < n; p += groups) {
      const int64_t part = (first + p) * 2 + (p == 0 ? first_slot : 0);
      const float2 ml = work.part_ml[part * tile_rows + pr];
      float4 x[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = work.part_o[(part * (D / 4) + cw * 4 + c) * tile_rows + pr];
      st.empty = st.empty || (ml.x == INFINITY && ml.y == 0.f);
      st.add(ml.x, ml.y, reinterpret_cast<const float*>(x));
    }
    // the lanes of a row, then the sets of warps
    for (int off = row_lanes; off < 32; off *= 2) {
      float o2[16];
      const float m2 = __shfl_xor_sync(0xFFFFFFFFu, st.m, off), l2 = __shfl_xor_sync(0xFFFFFFFFu, st.l, off);
#pragma unroll
      for (int x = 0; x < 16; ++x) o2[x] = __shfl_xor_sync(0xFFFFFFFFu, st.o[x], off);
      const bool e2 = __shfl_xor_sync(0xFFFFFFFFu, (int)st.empty, off) != 0;
      st.empty = st.empty || e2;
      st.add(m2, l2, o2);
    }
#pragma unroll
    for (int half = kSplits / 2; half >= 1; half /= 2) {
      if (split >= half && split < 2 * half) {
        sm_ml[split - half][cw][lane][0] = st.empty ? INFINITY : st.m;
        sm_ml[split - half][cw][lane][1] = st.empty ? 0.f : st.l;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sm_o[split - half][cw][c][lane] = make_float4(st.o[4 * c], st.o[4 * c + 1], st.o[4 * c + 2], st.o[4 * c + 3]);
      }
      __syncthreads();
      if (split < half) {
        const float m2 = sm_ml[split][cw][lane][0], l2 = sm_ml[split][cw][lane][1];
        float4 x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = sm_o[split][cw][c][lane];
        st.empty = st.empty || (m2 == INFINITY && l2 == 0.f);
        st.add(m2, l2, reinterpret_cast<const float*>(x));
      }
      __syncthreads();
    }
  }
  if (!mine) return;
  const bool none = st.empty || st.l == 0.f;
  const float inv = none ? 0.f : 1.f / st.l;
  uint32_t w[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) w[x] = none ? 0u : pack_bf16(st.o[2 * x] * inv, st.o[2 * x + 1] * inv);
  uint4* out = reinterpret_cast<uint4*>(o + row * D + 16 * cw);
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  out[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (cw == 0 && lse) lse[row] = none ? -INFINITY : (st.m + log2f(st.l)) * kLn2;
}

// The weights the rows received, from the scores that the attention kept: thread = 4 rows of the
// cache, the query rows added in order.
constexpr int kWeighThreads = 128, kWeighRows = 512;
__global__ void __launch_bounds__(kWeighThreads)
    tree_attn_weigh_kernel(const float* __restrict__ scores, int64_t score_stride, const float* __restrict__ lse,
                           const int32_t* __restrict__ kv_len, float* __restrict__ weight, int T, int64_t n_kv, int H,
                           int Hkv) {
  __shared__ float nlse2[kWeighRows];  // minus the LSE in the log2 domain; -inf: an empty slot
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t seq = blockIdx.y, L = context_len(kv_len, seq, T, n_kv);
  const int64_t t = ((int64_t)blockIdx.x * kWeighThreads + threadIdx.x) * 4;
  if (L < 0 || (int64_t)blockIdx.x * kWeighThreads * 4 >= L + T) return;
  const int G = H / Hkv, R = T * G, rows = T * H;
  float4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int r0 = 0; r0 < rows; r0 += kWeighRows) {
    const int n = min(kWeighRows, rows - r0);
    __syncthreads();
    for (int x = threadIdx.x; x < n; x += kWeighThreads) {
      const int g = (r0 + x) / R, r = r0 + x - g * R, i = r / G;
      const float l = lse[(seq * T + i) * H + g * G + (r - i * G)];
      nlse2[x] = l == -INFINITY ? -INFINITY : l * -kLog2e;
    }
    __syncthreads();
    if (t >= L + T) continue;
    const float* z = scores + (seq * rows + r0) * score_stride + t;
#pragma unroll 8
    for (int x = 0; x < n; ++x) {
      const float nl = nlse2[x];
      const float4 s = *reinterpret_cast<const float4*>(z + x * score_stride);
      if (nl == -INFINITY) continue;
      sum.x += fast_exp2(s.x + nl);
      sum.y += fast_exp2(s.y + nl);
      sum.z += fast_exp2(s.z + nl);
      sum.w += fast_exp2(s.w + nl);
    }
  }
  float* w = weight + seq * n_kv + t;
  if (t < L + T) w[0] = t < L ? w[0] + sum.x : sum.x;
  if (t + 1 < L + T) w[1] = t + 1 < L ? w[1] + sum.y : sum.y;
  if (t + 2 < L + T) w[2] = t + 2 < L ? w[2] + sum.z : sum.z;
  if (t + 3 < L + T) w[3] = t + 3 < L ? w[3] + sum.w : sum.w;
}

int row_tiles(const Shape& s) { return s.n_q * (s.H / s.Hkv) > kRows ? 2 : 1; }
// Query rows of an item, which are also its rows in the partial results.
int item_rows(const Shape& s) { return s.n_q * (s.H / s.Hkv) <= kFewRows ? kFewRows : row_tiles(s) * kRows; }

// Up to 8 query rows of a KV head the weights come from kept scores: writing and reading those moves 8 bytes a
// query row and key, reading K again 2 d bytes a key, and forms the scores again.  us with kept scores and with K
// read again, in a replayed graph, by query rows:
//   8 x 32K rows, 4 KV heads, d = 128:    1: 115, 156   4: 122, 155   8: 136, 156   16: 168, 155
//   2 x 16K rows, 16 KV heads, d = 128:   1: 64, 96     4: 72, 96     8: 82, 96     16: 108, 97
//   8 x 32K rows, 4 KV heads, d = 64:     1: 99, 121    4: 106, 121   8: 115, 121   16: 135, 121
//   2 x 16K rows, 16 KV heads, d = 64:    1: 63, 81     4: 74, 81     8: 89, 81     16: 121, 81
constexpr int kKeptRows = 8;
bool keeps_scores(const Shape& s) { return s.n_q * (s.H / s.Hkv) <= kKeptRows; }
int64_t score_stride(const Shape& s) { return (s.n_kv + kRows - 1) / kRows * kRows; }

struct Layout {
  size_t prefix, part_o, part_ml, lse, weight, total;
};
Layout layout(const Shape& s, bool with_weight) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = (size_t)kMaxCtas * 2 * item_rows(s);
  Layout L;
  L.prefix = 0;
  L.part_o = up((size_t)(s.batch + 2) * sizeof(int64_t));
  L.part_ml = L.part_o + up(rows * s.d * sizeof(float));
  L.lse = L.part_ml + up(rows * sizeof(float2));
  L.weight = L.lse + (with_weight ? up((size_t)s.n_query * s.H * sizeof(float)) : 0);
  L.total = L.weight;
  if (with_weight)
    L.total += up(keeps_scores(s) ? (size_t)s.n_query * s.H * score_stride(s) * sizeof(float)
                                  : cache_weight_workspace_bytes(s));
  return L;
}

template <int D, int NT>
cudaError_t launch(const Shape& s, const void* k, const void* v, const TreeArgs& a, int ctas, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!map_cache_rows(&mk, k, D, (uint64_t)s.Hkv, (uint64_t)s.n_kv, (uint64_t)s.batch, kRows) ||
      !map_cache_rows(&mv, v, D, (uint64_t)s.Hkv, (uint64_t)s.n_kv, (uint64_t)s.batch, kRows))
    return cudaErrorNotSupported;
  const cudaError_t e = ensure_smem((const void*)tree_attn_kernel<D, NT>, Cfg<D, NT>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_after(tree_attn_kernel<D, NT>, dim3((unsigned)ctas), kThreads, st, Cfg<D, NT>::kSmem, mk, mv, a);
}

template <int D>
cudaError_t launch_merge(const Shape& s, const TreeArgs& a, int tile_rows, int ctas, cudaStream_t st) {
  const int R = a.T * (a.H / a.Hkv);
  int lanes = 1;  // lanes for rows
  while (lanes < 32 && lanes < R) lanes *= 2;
  return launch_after(tree_attn_merge_kernel<D>, dim3((unsigned)(s.Hkv * ((R + lanes - 1) / lanes)), (unsigned)s.batch),
                      32 * (D / 16) * kSplits, st, 0, a.work, a.o, a.lse, s.batch, a.T, a.H, a.Hkv, tile_rows, lanes,
                      ctas);
}

}  // namespace

size_t tree_attn_workspace_bytes(const Shape& s, bool with_weight) { return layout(s, with_weight).total; }

cudaError_t launch_tree_attn(const Shape& s, const void* q, const void* k, const void* v, const int32_t* kv_len,
                             const int32_t* parent, void* o, float* lse, float* weight, int32_t* status, void* ws,
                             cudaStream_t st) {
  const Layout L = layout(s, weight != nullptr);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const bool kept = weight && keeps_scores(s);
  TreeArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.v = static_cast<const uint16_t*>(v);
  a.kv_len = kv_len;
  a.parent = parent;
  a.o = static_cast<uint16_t*>(o);
  a.lse = weight && !lse ? reinterpret_cast<float*>(w + L.lse) : lse;
  a.scores = kept ? reinterpret_cast<float*>(w + L.weight) : nullptr;
  a.score_stride = score_stride(s);
  a.work = {reinterpret_cast<int64_t*>(w + L.prefix), reinterpret_cast<float4*>(w + L.part_o),
            reinterpret_cast<float2*>(w + L.part_ml)};
  a.status = status;
  a.batch = s.batch;
  a.T = (int)s.n_q;
  a.n_kv = s.n_kv;
  a.H = s.H;
  a.Hkv = s.Hkv;
  a.qscale = s.scale * kLog2e;
  const int R = a.T * (s.H / s.Hkv), nt = row_tiles(s), tile_rows = item_rows(s);
  const int64_t most = (int64_t)s.batch * s.Hkv * ((R + tile_rows - 1) / tile_rows) * ((s.n_kv + kRows - 1) / kRows);
  const int ctas = (int)(most < kMaxCtas ? most : kMaxCtas);
  cudaError_t e;
  if (R <= kFewRows)
    e = launch_tree_attn_few(s, k, v, a, ctas, st);
  else if (s.d == 64)
    e = nt == 1 ? launch<64, 1>(s, k, v, a, ctas, st) : launch<64, 2>(s, k, v, a, ctas, st);
  else
    e = nt == 1 ? launch<128, 1>(s, k, v, a, ctas, st) : launch<128, 2>(s, k, v, a, ctas, st);
  if (e == cudaSuccess)
    e = s.d == 64 ? launch_merge<64>(s, a, tile_rows, ctas, st) : launch_merge<128>(s, a, tile_rows, ctas, st);
  if (e != cudaSuccess || !weight) return e;
  if (!kept) return launch_cache_weight(s, q, k, kv_len, parent, nullptr, a.lse, weight, nullptr, w + L.weight, st);
  const int64_t per = 4 * kWeighThreads;
  return launch_after(tree_attn_weigh_kernel, dim3((unsigned)((s.n_kv + per - 1) / per), (unsigned)s.batch),
                      kWeighThreads, st, 0, a.scores, a.score_stride, a.lse, kv_len, weight, a.T, s.n_kv, s.H, s.Hkv);
}

}  // namespace hisa
