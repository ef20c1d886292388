// hisa_cache_compact: rows of the cache moved towards the front, in place.
//
//   array[s][begin + j] = array[s][rows[s][j]],  rows ascending, rows[s][j] >= begin + j.
//
// In place, a destination row may be the source of another entry.  Every source is at or behind its
// own destination, so a sweep over j in ascending order that has read the rows of entries [0, j1) may
// write the destinations [0, j1): a later entry's source lies at begin + j1 or behind.  A slice (128
// bytes) of every row of one sequence is swept in tiles: the next tile's rows are loaded into
// registers, a barrier is passed (every load of the current tile is then in), the current tile is
// written.  Slices share no byte, so nothing else has to be ordered.  Where the slices are too few for
// the SMs (few sequences), a cluster of up to 8 CTAs sweeps a slice together, a part of each tile
// each, and the barrier is the cluster's (1 x 128K rows, a quarter kept: 201 us by CTAs alone, 110 by
// clusters of 4).
// The bound is HBM: each moved byte is read and written once; the next tile's loads are in flight
// while the current one is stored.  8 x 32K rows, a quarter kept: 91 us, 5.5 TB/s; slices of 256 bytes
// take 125 us, of 64 bytes 121.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace hisa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kUnroll = 8;    // row loads in flight per thread and tile
constexpr int kMaxCluster = 8;
constexpr int kLanesMax = 8, kLanesShort = 64;  // threads per row slice: long lists, lists of one tile

struct Array {
  uint8_t* base;
  int64_t row_bytes;
  int first_slice;  // first slice id of this array
  int vec;          // bytes per access: 16, or 4 where the rows are no multiple of 16
  int lanes;        // threads per row slice, a power of two
};
struct Arrays {
  Array a[kMaxRowArrays];
  int n;
};

// Plain loads (never the read-only path: the kernel writes the same array).
template <class V>
__device__ __forceinline__ V load_once(const uint8_t* p) {
  return *reinterpret_cast<const V*>(p);
}

// This CTA's entries of one tile: src[j] = the source row, or -1 for an entry that moves nothing.
struct Tile {
  int32_t src[kThreads * kUnroll];  // a row a thread at the most
};

template <class V>
__device__ __forceinline__ void sweep(const Array& A, int slice, const int32_t* __restrict__ list, int n, int64_t begin,
                                      int64_t n_kv, int64_t seq, Tile (&tile)[2], int32_t* status) {
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x;
  const int per = kThreads / A.lanes;  // rows per step
  const int rows = per * kUnroll;      // entries of a CTA's part of a tile
  const int r0 = tid / A.lanes, c = tid & (A.lanes - 1);
  const int64_t col = ((int64_t)slice * A.lanes + c) * (int64_t)sizeof(V);
  const bool mine = col < A.row_bytes;
  uint8_t* base = A.base + seq * n_kv * A.row_bytes + col;
  __shared__ int dirty;        // an entry broke the order: from then on the entries are looked at one by one
  __shared__ int64_t scanned;  // entries looked at so
  __shared__ int32_t last_in;  // the largest in range among them
  auto barrier = [&]() {
    if (nc == 1)
      __syncthreads();
    else
      cluster.sync();
  };
  if (tid == 0) {
    dirty = 0;
    scanned = 0;
    last_in = -1;
  }
  barrier();

  // Reads the entries [j0, j0 + rows) into t; those out of range move nothing.  An ascending list with its
  // padding at the end passes the test of neighbours; any other makes the whole cluster look closer.  All
  // threads call; ends synchronised.
  auto stage = [&](int64_t j0, Tile& t) {
    bool clean = true;
    for (int i = tid; i < rows; i += kThreads) {
      const int64_t j = j0 + i;
      int32_t r = -1;
      if (j < n) {
        r = list[j];
        const int32_t before = j > 0 ? list[j - 1] : -1;
        const bool in = r >= begin + j && r < n_kv;
        clean = clean && (r == -1 || (in && r > before && (j == 0 || before >= 0)));
        if (!in) r = -1;
      }
      t.src[i] = r;
    }
    if (!__syncthreads_and(clean) && tid < nc) *(volatile int*)cluster.map_shared_rank(&dirty, tid) = 1;
  };
  // Entries that are not greater than every in-range entry before them move nothing either.
  auto look = [&](int64_t j0, Tile& t) {
    if (tid == 0) {
      int32_t last = last_in;
      bool bad = false;
      int64_t j = scanned;
      for (; j < j0 + rows && j < n; ++j) {
        const int32_t r = list[j];
        if (r == -1) continue;
        const bool ok = r >= begin + j && r < n_kv && r > last;
        if (ok) last = r;
        if (!ok && j >= j0) {
          t.src[j - j0] = -1;
          bad = true;
        }
      }
      scanned = j;
      last_in = last;
      if (bad && status) atomicOr(status, kStatusBadIndex);
    }
    __syncthreads();
  };

  V cur[kUnroll], nxt[kUnroll];
  auto load = [&](const Tile& t, V (&x)[kUnroll]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t r = t.src[u * per + r0];
      if (mine && r >= 0) x[u] = load_once<V>(base + (int64_t)r * A.row_bytes);
    }
  };
  const int64_t part = (int64_t)rank * rows, whole = (int64_t)nc * rows;
  stage(part, tile[0]);
  load(tile[0], cur);
  int b = 0;
  for (int64_t t0 = 0; t0 < n; t0 += whole, b ^= 1) {
    const int64_t j0 = t0 + part;
    if (t0 + whole < n) {
      stage(j0 + whole, tile[b ^ 1]);
      load(tile[b ^ 1], nxt);
    }
    barrier();  // the rows of the current tile are read by every thread
    // A CTA of the cluster that is ahead may set this flag for its next tile by now, so the threads agree on one
    // answer (early is fine: the look then finds nothing).  Alone, no one is ahead.
    const int seen = *(volatile int*)&dirty;
    if (nc == 1 ? seen : __syncthreads_or(seen)) look(j0, tile[b]);
    const Tile& t = tile[b];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int e = u * per + r0;
      const int32_t r = t.src[e];
      if (mine && r >= 0 && r != begin + j0 + e) *reinterpret_cast<V*>(base + (begin + j0 + e) * A.row_bytes) = cur[u];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) cur[u] = nxt[u];
    __syncthreads();  // tile[b] may be filled again
  }
}

__global__ void __launch_bounds__(kThreads)
    cache_compact_kernel(const __grid_constant__ Arrays arrays, const int32_t* __restrict__ rows, int n_rows,
                         const int32_t* __restrict__ dst_begin, int64_t n_kv, int32_t* __restrict__ status, int nc) {
  __shared__ Tile tile[2];
  const int64_t seq = blockIdx.y;
  const int id = (int)blockIdx.x / nc;
  int a = 0;
  while (a + 1 < arrays.n && id >= arrays.a[a + 1].first_slice) ++a;
  const Array& A = arrays.a[a];
  const int slice = id - A.first_slice;
  const int64_t begin = dst_begin ? dst_begin[seq] : 0;
  if (begin < 0) {
    if (threadIdx.x == 0 && status) atomicOr(status, kStatusBadIndex);
    return;
  }
  if (A.vec == 16)
    sweep<uint4>(A, slice, rows + seq * n_rows, n_rows, begin, n_kv, seq, tile, status);
  else
    sweep<uint32_t>(A, slice, rows + seq * n_rows, n_rows, begin, n_kv, seq, tile, status);
}

}  // namespace

cudaError_t launch_cache_compact(const Shape& s, const int32_t* rows, int n_rows, const int32_t* dst_begin,
                                 const hisa_rows_t* arrays, int n_arrays, int32_t* status, cudaStream_t st) {
  Arrays p;
  p.n = n_arrays;
  int64_t slices = 0;
  for (int i = 0; i < n_arrays; ++i) {
    Array& A = p.a[i];
    A.base = static_cast<uint8_t*>(arrays[i].base);
    A.row_bytes = arrays[i].row_bytes;
    A.vec = A.row_bytes % 16 == 0 ? 16 : 4;
    const int64_t units = A.row_bytes / A.vec;
    // Long lists: slices of 128 bytes, so that even one sequence's sweeps cover the SMs.  A list that
    // is one tile all the same takes wider ones: fewer CTAs, each of a few rows.
    A.lanes = 1;
    while (A.lanes < units &&
           (A.lanes < kLanesMax || (A.lanes < kLanesShort && (int64_t)kThreads / (2 * A.lanes) * kUnroll >= n_rows)))
      A.lanes *= 2;
    A.first_slice = (int)slices;
    slices += (units + A.lanes - 1) / A.lanes;
  }
  // CTAs that sweep a slice together: while two a SM take them all, and each has a tile of its own.
  int nc = 1;
  while (nc < kMaxCluster && slices * s.batch * nc * 2 <= 2 * 148 &&
         n_rows >= (int64_t)nc * 2 * (kThreads / kLanesMax * kUnroll))
    nc *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(slices * nc), (unsigned)s.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)nc;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_compact_kernel, p, rows, n_rows, dst_begin, s.n_kv, status, nc);
}

}  // namespace hisa
