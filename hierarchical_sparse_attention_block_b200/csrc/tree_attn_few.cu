// hisa_tree_attn_fwd for up to 16 query rows per KV head (a plain decode step, small trees), on the
// 5th-generation tensor cores with the keys as the product's rows:
//
//   S^T = K Q^T  (128 keys x N),   O^T += V^T P^T  (D x N),   N = 16 >= T H / Hk query rows.
//
// The call is bound by the cache's bytes (K and V once): 8 x 64K rows of different lengths, one query row a KV
// head, take 421 to 444 us (GPUs differ), 6.5 to 6.8 TB/s.  With the query rows as the M = 128 of the products, as
// tree_attn.cu has them, one to 16 of 128 rows would be padding (446 us, with weights of 8 bits).  Here the products
// shrink with N, a thread, which owns a key, forms that key's weights of all rows, and keeping the scores for the
// weights that the rows receive is a coalesced store.  From 17 rows on the stores of the weights, two bytes at a
// time, take longer than the tile's bytes (8 x 32K rows, 32 query rows: 150 us this way with N = 32, 129 the other).
//
// Work and ring buffers are those of tree_attn.cu (one row tile).  Scores and weights have two buffers,
// used by the key tiles in turn; the two softmax groups of four warps take half of the query rows each.
// A row's softmax runs over the lanes here.  Its reference max is one number for the group's warps; it
// starts as the score of the segment's first key and moves, for all of them, when a score exceeds it by
// 2^8: each tile the warps look for that while they form the weights (no reduction over lanes), agree at a
// barrier, and only where one found it, rarely, reduce the rows' max, rescale and form the weights again (once a
// tile: after that no score of the tile exceeds it; row_ref.h has the arithmetic).
// (Starting from the first tile's max instead: 1 x 1K rows, 16 query rows, 18.2 us, 15.7 this way with the
// sums by halving.)  A row's sum stays a partial sum per thread until the segment's end.  The weights go to
// shared memory, in the layout of the second product's operand, as two bf16 numbers each (16 significant bits).
// Every wait is bounded (1 s): a timeout sets status bit 1 and the CTA stops.
#include <math.h>

#include "row_ref.h"
#include "tree_attn.cuh"

namespace hisa {
namespace {

using namespace tc;

constexpr int kLead = 4;       // what another item costs a CTA, in key tiles of about 1.5 us
constexpr int kSoftmax = 256;  // two groups
constexpr int kThreads = kSoftmax + 96;
constexpr int kWarpK = 8, kWarpMMA = 9, kWarpV = 10;
constexpr uint32_t kTmemCols = 256;  // score buffer b at 64 b, the output at 128

constexpr int N = kFewRows;

template <int D>
struct Cfg {
  static constexpr int kTile = kHalf * (D / 64);   // a K or V tile
  static constexpr int kQHalf = N * 128;           // 64 columns of the query rows
  static constexpr int kWeights = N * 256;         // one part (high, low) of a tile's weights: N rows x 128 keys
  // ring slots of K and of V: what 227 KB hold beside the rest
  static constexpr int KS = D == 64 ? 6 : 3, VS = D == 64 ? 6 : 3;
  // V before the weights and the rest: with D = 64 the second product's upper 64 rows, which nobody
  // reads, come from the 16 KB behind a V tile
  static constexpr int K_OFF = 0, V_OFF = K_OFF + KS * kTile, P_OFF = V_OFF + VS * kTile;
  static constexpr int Q_OFF = P_OFF + 4 * kWeights;  // weight buffer b, part p at P_OFF + (2 b + p) * kWeights
  static constexpr int TREE_OFF = Q_OFF + kQHalf * (D / 64);
  static constexpr int ROW_OFF = TREE_OFF + (int)sizeof(DraftTree);     // RowRef [N]
  static constexpr int ALPHA_OFF = ROW_OFF + N * (int)sizeof(float2);    // float [N]
  static constexpr int MAX_OFF = ALPHA_OFF + N * 4;                      // float [4][N]: per warp; then the sums
  static constexpr int JOIN_OFF = MAX_OFF + 4 * N * 4;                   // float2 [N]: max, sum
  static constexpr int SLOT_OFF = JOIN_OFF + N * 8;                      // int16 [N]: the rows' slots
  static constexpr int BAR_OFF = SLOT_OFF + N * 2;
  enum : int {
    B_QFULL = 0,
    B_KFULL,                  // [KS]
    B_KEMPTY = B_KFULL + KS,  // [KS]
    B_VFULL = B_KEMPTY + KS,  // [VS]
    B_VEMPTY = B_VFULL + VS,  // [VS]
    B_SFULL = B_VEMPTY + VS,  // [2]: per buffer
    B_PREADY = B_SFULL + 2,   // [2]
    B_PFREE = B_PREADY + 2,   // [2]
    B_AGREE = B_PFREE + 2,    // [2]: a group's warps among themselves
    B_SYNC = B_AGREE + 2,     // both groups
    B_GO,                     // the first segment's query rows are asked for
    B_DRAIN,
    kNBar
  };
  static constexpr int WALK_OFF = BAR_OFF + kNBar * 8;
  static constexpr int MISC_OFF = WALK_OFF + (int)sizeof(WalkShared<kThreads>);
  static constexpr int kSmem = MISC_OFF + 4 * (6 + 2 * kDraftWords) + 1024;  // + slack for the 1024-byte alignment
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(P_OFF % 1024 == 0 && Q_OFF % 1024 == 0 && kQHalf % 1024 == 0, "swizzle atoms stay 1024-byte aligned");
  static_assert(P_OFF - V_OFF >= kTile && 4 * kWeights >= kHalf, "what lies behind a V tile is this block's memory");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_few_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ TreeArgs args) {
  using C = Cfg<D>;
  const int32_t* const parent = args.parent;
  int32_t* const status = args.status;
  const int T = args.T, H = args.H, Hkv = args.Hkv, G = H / Hkv, R = T * G;
  const int64_t n_kv = args.n_kv;
  const float qscale = args.qscale;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) { return sb + (uint32_t)C::BAR_OFF + 8u * (uint32_t)i; };
  DraftTree& tree = *reinterpret_cast<DraftTree*>(smem + C::TREE_OFF);
  int16_t* slots = reinterpret_cast<int16_t*>(smem + C::SLOT_OFF);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  uint32_t* tmem_slot = misc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  // [2][2] by group and key tile parity: a row of the group exceeds its reference.  A warp may be a tile ahead of the
  // others: past a tile's barrier, it waits for none of them until the next tile's.
  volatile int* raise_flags = reinterpret_cast<volatile int*>(misc + 2);
  uint32_t* odd_rows = misc + 6;  // [2][kDraftWords] by segment parity: drafted V rows not all finite
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
      const bool group = i >= C::B_AGREE && i < C::B_SYNC, all = i >= C::B_PREADY && i < C::B_PFREE;
      mbar_init(bar(i), group ? kRows : all || i == C::B_SYNC || i == C::B_QFULL || i == C::B_GO ? kSoftmax : 1);
    }
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) raise_flags[i] = 0;
    mbar_init_fence();
  }
  if (tid < 2 * kDraftWords) odd_rows[tid] = 0u;
  if (tid < N) slots[tid] = (int16_t)(min(tid, R - 1) / G);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what the kernels before wrote, and read of the workspace
  tc_fence_before();
  Walk walk = walk_begin<kThreads>(args.kv_len, n_kv, T, args.batch, Hkv, kLead,
                                   *reinterpret_cast<WalkShared<kThreads>*>(smem + C::WALK_OFF), args.work.prefix,
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
      const uint64_t policy = l2_evict_first();  // K and V pass through the L2 once
      int slot = 0, issued = 0;
      uint32_t phase = 1;  // parity of the slot's last release
      bool ok = true;
      while (ok && walk.next()) {
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
            tma_load_4d(dst + h2 * kHalf, map, 64 * h2, walk.item, (walk.j0 + x) * kRows, walk.s, bar(full + slot),
                        policy);
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
      constexpr uint32_t kIdS = idesc_bf16(kRows, N, false, false);  // K and Q both K-major
      constexpr uint32_t kIdO = idesc_bf16(128, N, true, false);     // V with its columns as rows, weights K-major
      bool ok = true;
      int kit = 0, vit = 0, seg = 0;  // K and V tiles taken (the score and weight buffers go with them), segments
      auto scores_of = [&]() {        // of the K tile kit
        const uint32_t kt = sb + (uint32_t)(C::K_OFF + (kit % C::KS) * C::kTile);
        if (elect_one()) {
#pragma unroll
          for (int h2 = 0; h2 < D / 64; ++h2)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16(tmem + 64u * (uint32_t)(kit & 1), desc_kmajor_sw128(kt + h2 * kHalf + kk * 32),
                        desc_kmajor_sw128(sb + (uint32_t)(C::Q_OFF + h2 * C::kQHalf + kk * 32)), kIdS, (h2 | kk) ? 1u : 0u);
          umma_commit(bar(C::B_SFULL + (kit & 1)));
          umma_commit(bar(C::B_KEMPTY + kit % C::KS));
        }
        ++kit;
      };
      auto wait_k = [&]() {
        const bool r = waited(bar(C::B_KFULL + kit % C::KS), (uint32_t)(kit / C::KS) & 1u);
        tc_fence_after();
        return r;
      };
      while (ok && walk.next()) {
        const int n = walk.n;
        ok = waited(bar(C::B_QFULL), (uint32_t)seg & 1u) && wait_k();
        ++seg;
        if (!ok) break;
        scores_of();
        if (n > 1) {
          ok = wait_k();
          if (!ok) break;
          scores_of();
        }
        for (int x = 0; ok && x < n; ++x) {
          const int buf = vit & 1;
          ok = waited(bar(C::B_PREADY + buf), (uint32_t)(vit >> 1) & 1u) &&
               waited(bar(C::B_VFULL + vit % C::VS), (uint32_t)(vit / C::VS) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint32_t vt = sb + (uint32_t)(C::V_OFF + (vit % C::VS) * C::kTile);
          const uint32_t pt = sb + (uint32_t)(C::P_OFF + 2 * buf * C::kWeights);
          if (elect_one()) {
#pragma unroll
            for (int part = 0; part < 2; ++part)  // the weights' high and low parts
#pragma unroll
              for (int kk = 0; kk < kRows / 16; ++kk)  // keys 16 kk .. 16 kk + 15
                umma_bf16(tmem + 128u, desc_mnmajor_sw128(vt + kk * 2048, kHalf),
                          desc_kmajor_sw128(pt + (uint32_t)(part * C::kWeights + (kk >> 2) * C::kQHalf + (kk & 3) * 32)),
                          kIdO, (x > 0 || part || kk) ? 1u : 0u);
            umma_commit(bar(C::B_PFREE + buf));
            umma_commit(bar(C::B_VEMPTY + vit % C::VS));
          }
          ++vit;
          if (x + 2 < n) {  // the buffer of tile x: its scores have been read
            ok = wait_k();
            if (!ok) break;
            scores_of();
          }
        }
      }
      if (!ok && lane == 0) fail();
      if (elect_one()) umma_commit(bar(C::B_DRAIN));
      mbar_wait(bar(C::B_DRAIN), 0);
    }
  } else {
    // ---------------- softmax and output: group t has the rows [row0, row0 + NR); thread = key of the tile, then
    // column of the output ----------------
    constexpr int NR = N / 2;
    const int t = warp >> 2, row0 = t * NR;
    const int r = tid & (kRows - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lanes + 128u + (uint32_t)row0;
    RowRef* rows = reinterpret_cast<RowRef*>(smem + C::ROW_OFF) + row0;
    const float limit = rise_limit(qscale);
    float* alphas = reinterpret_cast<float*>(smem + C::ALPHA_OFF) + row0;
    float* per_warp = reinterpret_cast<float*>(smem + C::MAX_OFF) + row0;  // [4] at pitch N
    float2* join = reinterpret_cast<float2*>(smem + C::JOIN_OFF) + row0;
    // this key's place in a row of the weights: 16-byte chunk (swizzled by the row), bytes within it
    const int p_half = (r >> 6) * C::kQHalf, p_chunk = (r & 63) >> 3, p_byte = (r & 7) * 2;
    bool ok = true;
    int cnt = 0, seg = 0;  // key tiles so far, segments
    uint32_t sync_phase = 0, agree_phase = 0;
    auto sync = [&]() {
      mbar_arrive(bar(C::B_SYNC));
      ok = warp_wait_or_abort(bar(C::B_SYNC), sync_phase, abort_flag) && ok;
      sync_phase ^= 1u;
    };
    auto agree = [&]() {
      mbar_arrive(bar(C::B_AGREE + t));
      ok = warp_wait_or_abort(bar(C::B_AGREE + t), agree_phase, abort_flag) && ok;
      agree_phase ^= 1u;
    };
    while (ok && walk.next()) {
      const int64_t seq = walk.s;
      const int g = walk.item;
      const int L = (int)walk.L;
      if (seg > 0) sync();  // the segment before is read out everywhere
      if (!ok) break;
      {
        constexpr int CH = D / 8;  // 16-byte chunks of a row; rows that hold no query are 0
        for (int e = tid; e < N * CH; e += kSoftmax) {
          const int row = e / CH, c = e % CH, i = row / G;
          const bool held = row < R;
          cp_async16(smem + C::Q_OFF + (c >> 3) * C::kQHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                     args.q + (held ? ((seq * T + i) * H + g * G + (row - i * G)) * D + c * 8 : 0), held);
        }
        cp_async_commit();
        if (seg == 0) mbar_arrive(bar(C::B_GO));
        cp_async_wait<0>();
        fence_async_smem();
      }
      mbar_arrive(bar(C::B_QFULL));
      if (tid < kDraftWords) odd_rows[((seg + 1) & 1) * kDraftWords + tid] = 0u;
      if (r < NR) rows[r] = {0.f, -INFINITY};
      uint32_t* odd = odd_rows + (seg & 1) * kDraftWords;
      const bool treed = parent && (walk.j0 + walk.n) * kRows > L;  // the segment reaches behind the context
      if (treed) {
        if (draft_tree_build<kSoftmax>(tree, parent + seq * T, T, tid, sync) && status)
          atomicOr(status, kStatusBadIndex);
      }
      agree();  // the rows' state
      if (!ok) break;
      ++seg;
      float* scores =
          args.scores && row0 < R ? args.scores + ((seq * Hkv + g) * R + row0) * args.score_stride + r : nullptr;
      float l[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) l[i] = 0.f;
      const int ahead_at = max(0, walk.n - 10);
      for (int x = 0; x < walk.n; ++x, ++cnt) {
        const int t0 = (walk.j0 + x) * kRows, buf = cnt & 1;
        const uint32_t ts = tmem + lanes + 64u * (uint32_t)buf + (uint32_t)row0;
        volatile int* raise = raise_flags + 2 * t + buf;
        const bool tail = t0 + kRows > L;
        const int j = t0 + r - L;  // drafted row of this key, from the context's end on
        if (t == 0 && x == ahead_at) prefetch_next<D>(walk, args, 1, kFewRows, r);
        ok = warp_wait_or_abort(bar(C::B_SFULL + buf), (uint32_t)(cnt >> 1) & 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
        // the rows' scores of this key, -inf where a row does not see it
        auto load = [&](uint32_t(&s)[NR]) {
          __syncwarp();
          tmem_ld<NR>(ts, s);
          if (tail && j >= 0) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
              if (j >= T || !sees(tree, parent != nullptr, slots[row0 + i], j)) s[i] = 0xFF800000u;
          }
        };
        if (x == 0) {
          // A reference to start from: the score of the segment's first key, where the row sees it.
          if ((warp & 3) == 0) {
            uint32_t s[NR];
            load(s);
            if (lane == 0) {
#pragma unroll
              for (int i = 0; i < NR; ++i) {
                const float z = __uint_as_float(s[i]);
                if (z > -INFINITY && z < INFINITY) rows[i] = {z, limit};
              }
            }
          }
          agree();
          if (!ok) break;
        }
        float p[NR];
        // The weights; formed a second time, and for good, if a score asks for another reference.
        for (bool raised = false;; raised = true) {
          bool up = false;
          uint32_t s[NR];
          load(s);
          if (scores && !raised) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
              if (row0 + i < R) scores[i * args.score_stride + t0] = __uint_as_float(s[i]) * qscale;
          }
#pragma unroll
          for (int i = 0; i < NR; i += 2) {
            const float4 st = *reinterpret_cast<const float4*>(rows + i);
            const RowRef r0 = {st.x, st.y}, r1 = {st.z, st.w};
            const float s0 = __uint_as_float(s[i]), s1 = __uint_as_float(s[i + 1]);
            up |= exceeds(s0, r0);
            up |= exceeds(s1, r1);
            p[i] = fast_exp2(exponent(s0, r0, qscale));  // 0 where masked
            p[i + 1] = fast_exp2(exponent(s1, r1, qscale));
          }
          if (raised) break;
          if (__any_sync(0xFFFFFFFFu, up) && lane == 0) *raise = 1;
          agree();
          if (!ok || !*raise) break;
          // the rows' max over the tile, per warp and then over the warps
          float mine = -INFINITY;
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            const float top = warp_max(__uint_as_float(s[i]));
            if (lane == i) mine = top;
          }
          if (lane < NR) per_warp[(warp & 3) * N + lane] = mine;
          agree();
          if (!ok) break;
          if (r == 0) *raise = 0;
          if (r < NR) {
            const RowRef st = rows[r];
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) top = fmaxf(top, per_warp[w * N + r]);
            float alpha = 1.f;
            if (exceeds(top, st)) {
              const RowRef moved = {top, limit};
              if (st.limit != -INFINITY) alpha = exp2f(exponent(st.ref, moved, qscale));  // else nothing to rescale
              rows[r] = moved;
            }
            alphas[r] = alpha;
          }
          agree();
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < NR; ++i) l[i] *= alphas[i];
          if (x > 0) {  // the output holds earlier tiles: rescale it once they are in
            ok = warp_wait_or_abort(bar(C::B_PFREE + (buf ^ 1)), (uint32_t)((cnt - 1) >> 1) & 1u, abort_flag);
            if (!ok) break;
            tc_fence_after();
            uint32_t ov[NR];
            __syncwarp();
            tmem_ld<NR>(to, ov);
#pragma unroll
            for (int i = 0; i < NR; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alphas[i]);
            tmem_st<NR>(to, ov);
          }
        }
        if (!ok) break;
        // the weight buffer is free once the product of two tiles ago is in
        if (cnt >= 2) {
          ok = warp_wait_or_abort(bar(C::B_PFREE + buf), (uint32_t)((cnt >> 1) - 1) & 1u, abort_flag);
          if (!ok) break;
        }
        uint8_t* at = smem + C::P_OFF + 2 * buf * C::kWeights + p_half + row0 * 128 + p_byte;
#pragma unroll
        for (int i = 0; i < NR; i += 2) {
          l[i] += p[i];
          l[i + 1] += p[i + 1];
          const uint32_t hi = pack_bf16(p[i], p[i + 1]), lo = pack_bf16(p[i] - bf16_lo(hi), p[i + 1] - bf16_hi(hi));
          uint8_t* a0 = at + i * 128 + ((p_chunk ^ (i & 7)) << 4);
          uint8_t* a1 = at + (i + 1) * 128 + ((p_chunk ^ ((i + 1) & 7)) << 4);
          *reinterpret_cast<uint16_t*>(a0) = (uint16_t)hi;
          *reinterpret_cast<uint16_t*>(a1) = (uint16_t)(hi >> 16);
          *reinterpret_cast<uint16_t*>(a0 + C::kWeights) = (uint16_t)lo;
          *reinterpret_cast<uint16_t*>(a1 + C::kWeights) = (uint16_t)(lo >> 16);
        }
        if (tail && t == 0) {
          // The product of two tiles ago is in, so the wait cannot take an earlier fill of the V slot for this one.
          const int vs = cnt % C::VS;
          ok = warp_wait_or_abort(bar(C::B_VFULL + vs), (uint32_t)(cnt / C::VS) & 1u, abort_flag);
          if (!ok) break;
          clear_tail_values<D>(smem + C::V_OFF + vs * C::kTile, t0, L, T, parent != nullptr, tree, odd, r);
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(bar(C::B_PREADY + buf));
      }
      if (!ok) break;
      ok = warp_wait_or_abort(bar(C::B_PFREE + ((cnt - 1) & 1)), (uint32_t)((cnt - 1) >> 1) & 1u, abort_flag);
      if (!ok) break;
      tc_fence_after();
      // the rows' sums: over the lanes, then over the warps
      // (half of the rows change lanes at each step: lane 4 i ends with row i)
      static_assert(NR == 8, "three halvings leave one row a lane");
#pragma unroll
      for (int h = NR / 2; h >= 1; h /= 2) {
        const bool upper = (lane & (4 * h)) != 0;
#pragma unroll
        for (int i = 0; i < h; ++i)
          l[i] = (upper ? l[i + h] : l[i]) + __shfl_xor_sync(0xFFFFFFFFu, upper ? l[i] : l[i + h], 4 * h);
      }
      l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], 2);
      l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], 1);
      if ((lane & 3) == 0) per_warp[(warp & 3) * N + lane / 4] = l[0];
      agree();
      if (!ok) break;
      if (r < NR) {
        const RowRef st = rows[r];
        float m = st.limit == -INFINITY ? -INFINITY : st.ref * qscale;  // log2 domain
        float sum = (per_warp[r] + per_warp[N + r]) + (per_warp[2 * N + r] + per_warp[3 * N + r]);
        // an empty slot; where the segment ends within the context, the merge learns it from another part
        if (treed && tree.end[slots[row0 + r]] != kRoot) {
          sum = 0.f;
          m = INFINITY;
        }
        join[r] = make_float2(m, sum);
        alphas[r] = sum == 0.f ? 0.f : 1.f / sum;
      }
      agree();
      if (!ok) break;
      const bool whole = walk.whole();
      const int64_t part = (int64_t)blockIdx.x * 2 + walk.slot();
      const uint32_t any_odd = odd[0] | odd[1] | odd[2] | odd[3] | odd[4] | odd[5] | odd[6] | odd[7];
      // Output: thread = column.
      uint32_t ov[NR];
      __syncwarp();
      tmem_ld<NR>(to, ov);
      if (r < D) {
        float y[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) y[i] = join[i].y == 0.f ? 0.f : __uint_as_float(ov[i]);
        if (any_odd) {
          // values that are not finite, of the rows that a token sees in this segment
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            const int slot = slots[row0 + i];
            if (row0 + i >= R || (treed && tree.end[slot] != kRoot)) continue;
            for (int jj = 0; jj < T; ++jj) {
              if (!((odd[jj >> 5] >> (jj & 31)) & 1u) || !sees(tree, parent != nullptr, slot, jj)) continue;
              const uint32_t b = args.v[((seq * n_kv + L + jj) * Hkv + g) * D + r];
              if ((b & 0x7F80u) == 0x7F80u) y[i] += bf16_lo(b);
            }
          }
        }
        if (whole) {
          __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(args.o) + (seq * T * H + g * G) * D + r;
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            const int row = row0 + i, slot = slots[row];
            if (row < R)
              o[((int64_t)slot * H + (row - slot * G)) * D] =
                  __float2bfloat16_rn(join[i].y == 0.f ? y[i] : y[i] * alphas[i]);
          }
        } else {
          float* o = reinterpret_cast<float*>(args.work.part_o + (part * (D / 4) + r / 4) * N + row0) + (r & 3);
#pragma unroll
          for (int i = 0; i < NR; ++i)
            if (row0 + i < R) o[4 * i] = y[i];
        }
      }
      __syncwarp();
      if (r < NR && row0 + r < R) {
        const float2 ms = join[r];
        const int row = row0 + r, slot = slots[row];
        if (!whole)
          args.work.part_ml[part * N + row] = ms;
        else if (args.lse)
          args.lse[(seq * T + slot) * H + g * G + (row - slot * G)] =
              ms.y == 0.f ? -INFINITY : (ms.x + log2f(ms.y)) * kLn2;
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

template <int D>
cudaError_t launch(const Shape& s, const void* k, const void* v, const TreeArgs& a, int ctas, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!map_cache_rows(&mk, k, D, (uint64_t)s.Hkv, (uint64_t)s.n_kv, (uint64_t)s.batch, kRows) ||
      !map_cache_rows(&mv, v, D, (uint64_t)s.Hkv, (uint64_t)s.n_kv, (uint64_t)s.batch, kRows))
    return cudaErrorNotSupported;
  const cudaError_t e = ensure_smem((const void*)tree_attn_few_kernel<D>, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_after(tree_attn_few_kernel<D>, dim3((unsigned)ctas), kThreads, st, Cfg<D>::kSmem, mk, mv, a);
}

}  // namespace

cudaError_t launch_tree_attn_few(const Shape& s, const void* k, const void* v, const TreeArgs& a, int ctas,
                                 cudaStream_t st) {
  return s.d == 64 ? launch<64>(s, k, v, a, ctas, st) : launch<128>(s, k, v, a, ctas, st);
}

}  // namespace hisa
