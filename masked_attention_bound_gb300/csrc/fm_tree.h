// Attention over the paged cache: what its kernels share.
//
// Work is cut into units and tiles.  A unit is one (sequence, K/V head, row
// tile): up to R rows, row r of a sequence being node r / G of query head hk *
// G + r % G, so the G query heads that share a K/V head share its loads.  A
// unit walks the 128-key tiles [0, tiles) of its sequence up to its last
// node.  All tiles of all units, in order, form one line; each block takes an
// equal run of it, whatever the lengths, so one long sequence keeps every SM
// busy and a full batch is balanced.  Where a run ends inside a unit, each
// block leaves its unnormalised part (running max, sum, O) in the workspace
// and tree_join_kernel adds the parts in ascending order.
#pragma once
#include <cuda_bf16.h>

#include "fm_cache.h"
#include "fm_ptx.cuh"
#include "fm_tmap.h"

namespace fm {

struct TreeParams {
  int B, H, Hkv, G, total, max_nodes, page_size, n_pages, max_pages;
  int tree;                // 0: chain (no parents)
  float scale_log2;        // scale * log2(e)
  const __nv_bfloat16* q;
  int64_t q_stride[2];
  __nv_bfloat16* o;
  int64_t o_stride[2];
  float* lse;
  const __nv_bfloat16* v_pool;   // for values that are not finite (see fix_row)
  int64_t v_stride[3];           // page, slot, head
  const int32_t *table, *lens, *cu, *parents;
  int4* rec;               // [grid] see Parts
  int part_rows;           // rows that a part has room for
  float2* part_ml;         // [2 * grid][part_rows] running max (base-2 exponent) and sum
  float* part_o;           // [2 * grid][part_rows][D]
  int* status;
  uint64_t wait_ns;
  int withhold;
};

// What a block leaves for the join: rec.x = the unit it starts and does not
// finish (a part in slot 2 * block + 1), -1 if none: sequence in .x, K/V head
// in .y, row tile in .z; rec.w = 0, or 1: its first run finishes a unit that
// an earlier block started, 2: belongs to one and does not finish it (a part
// in slot 2 * block).

// Per sequence: packed rows, nodes, context length (-1: out of range).
struct TreeSeq {
  int row0, n, base;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& P, int b) {
  TreeSeq s;
  const int c0 = P.cu[b], c1 = P.cu[b + 1], len = P.lens[b];
  s.row0 = c0;
  s.n = c1 - c0;
  s.base = len - s.n;
  if (c0 < 0 || s.n < 0 || c1 > P.total || s.n > P.max_nodes || len < s.n ||
      len > P.max_pages * P.page_size) {
    // the rows that can be written get zeros
    const int lo = max(c0, 0), hi = min(c1, P.total);
    s.row0 = lo;
    s.n = max(hi - lo, 0);
    s.base = -1;
  }
  return s;
}

// Row tiles of a sequence, keys and tiles of one of them.
template <int R>
__device__ __forceinline__ int row_tiles(const TreeParams& P, const TreeSeq& s) {
  return static_cast<int>((static_cast<int64_t>(s.n) * P.G + R - 1) / R);
}
template <int R>
__device__ __forceinline__ int unit_keys(const TreeParams& P, const TreeSeq& s, int rt) {
  if (s.base < 0) return 0;
  const int64_t rows = static_cast<int64_t>(s.n) * P.G;
  const int64_t end = min(rows, static_cast<int64_t>(rt + 1) * R);
  return s.base + static_cast<int>((end - 1) / P.G) + 1;
}
__device__ __forceinline__ int key_tiles(int keys) {
  return keys > 0 ? (keys + kTile - 1) / kTile : 1;
}
// Tiles of all units of one K/V head of a sequence.
template <int R>
__device__ __forceinline__ int64_t seq_tiles(const TreeParams& P, const TreeSeq& s) {
  const int nr = row_tiles<R>(P, s);
  int64_t w = 0;
  for (int rt = 0; rt < nr; ++rt) w += key_tiles(unit_keys<R>(P, s, rt));
  return w;
}

// A place on the line of tiles.
struct TreePlace {
  int b, hk, rt, tile;
};

// The run [begin, end) of a block and where it starts; all threads of the
// block call it.
struct TreeRun {
  int64_t left;       // tiles of the run
  TreePlace at;
};

struct TreeScan {
  int64_t warp[32];
  int64_t begin, end;
  int64_t before;     // tiles before sequence b
  int b;
};

template <int R, int NT>
__device__ __forceinline__ TreeRun tree_run(const TreeParams& P, TreeScan& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = NT / 32;
  int64_t w_first = 0;            // this thread's sequence of the first round
  auto weight = [&](int b) -> int64_t {
    if (b >= P.B) return 0;
    const TreeSeq s = tree_seq(P, b);
    if (s.base < 0 && blockIdx.x == 0 && P.status) atomicOr(P.status, DEV_CACHE);
    return seq_tiles<R>(P, s) * P.Hkv;
  };
  int64_t sum = 0;
  for (int b = tid; b < P.B; b += NT) {
    const int64_t w = weight(b);
    if (b == tid) w_first = w;
    sum += w;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sh.warp[warp] = sum;
  if (tid == 0) sh.b = -1;
  __syncthreads();
  int64_t all = 0;
  for (int i = 0; i < NW; ++i) all += sh.warp[i];
  // no more blocks than tiles: the runs of the others are empty
  const int64_t blocks = min(all, static_cast<int64_t>(gridDim.x));
  const bool idle = blockIdx.x >= blocks;
  const int64_t begin = idle ? all : all * blockIdx.x / blocks;
  const int64_t end = idle ? all : all * (blockIdx.x + 1) / blocks;
  int64_t before = 0;
  for (int b0 = 0; b0 < P.B; b0 += NT) {
    __syncthreads();
    const int b = b0 + tid;
    const int64_t w = b0 == 0 ? w_first : weight(b);
    int64_t inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) sh.warp[warp] = inc;
    __syncthreads();
    int64_t pre = before;
    for (int i = 0; i < NW; ++i) {
      if (i < warp) pre += sh.warp[i];
      before += sh.warp[i];
    }
    const int64_t lo = pre + inc - w;
    if (w > 0 && lo <= begin && begin < lo + w) {
      sh.b = b;
      sh.before = lo;
    }
    if (before > begin) break;
  }
  __syncthreads();
  TreeRun run;
  run.left = end - begin;
  run.at = TreePlace{sh.b, 0, 0, 0};
  if (sh.b < 0) run.left = 0;     // no tiles at all
  if (run.left > 0) {
    const TreeSeq s = tree_seq(P, sh.b);
    const int64_t per = seq_tiles<R>(P, s);
    int64_t off = begin - sh.before;
    run.at.hk = static_cast<int>(off / per);
    off -= run.at.hk * per;
    int rt = 0;
    while (true) {
      const int t = key_tiles(unit_keys<R>(P, s, rt));
      if (off < t) break;
      off -= t;
      ++rt;
    }
    run.at.rt = rt;
    run.at.tile = static_cast<int>(off);
  }
  return run;
}

// One stretch of tiles of one unit, as a block works on it.
struct TreePiece {
  int b, hk, rt;
  TreeSeq s;
  int keys;            // keys of the unit (the last node's position + 1)
  int t0, t1, tiles;   // tiles [t0, t1) of [0, tiles)
  int row_first, rows; // first row of the unit within its sequence, rows
  int origin;          // the first key that not every row of the unit sees for certain
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// Every role of a block walks its run piece by piece in the same order.
template <int R>
struct TreeWalk {
  TreeRun run;
  __device__ __forceinline__ bool next(const TreeParams& P, TreePiece& u) {
    if (run.left <= 0) return false;
    TreePlace& at = run.at;
    TreeSeq s = tree_seq(P, at.b);
    // on to the next sequence with rows
    while (at.hk >= P.Hkv || s.n <= 0) {
      at.hk = 0;
      at.rt = 0;
      at.tile = 0;
      ++at.b;
      if (at.b >= P.B) return false;
      s = tree_seq(P, at.b);
    }
    u.b = at.b;
    u.hk = at.hk;
    u.rt = at.rt;
    u.s = s;
    u.keys = unit_keys<R>(P, s, at.rt);
    u.tiles = key_tiles(u.keys);
    u.t0 = at.tile;
    u.t1 = static_cast<int>(min(static_cast<int64_t>(u.tiles), at.tile + run.left));
    run.left -= u.t1 - u.t0;
    u.row_first = at.rt * R;
    u.rows = static_cast<int>(min(static_cast<int64_t>(R), static_cast<int64_t>(s.n) * P.G - u.row_first));
    u.origin = s.base + (P.tree ? 0 : u.row_first / P.G);
    at.tile = u.t1;
    if (u.t1 == u.tiles) {
      at.tile = 0;
      if (++at.rt >= row_tiles<R>(P, s)) {
        at.rt = 0;
        ++at.hk;
      }
    }
    return true;
  }
};

// Parent of node t of sequence s as the kernels use it: -1 a root, -2 padding.
__device__ __forceinline__ int tree_parent(const TreeParams& P, const TreeSeq& s, int t) {
  const int p = P.parents[s.row0 + t];
  if (p >= -2 && p < t) return p;
  if (P.status) atomicOr(P.status, DEV_CACHE);
  return -1;
}

// Ancestors of node t and itself as bits [0, 256) of w (all 0 for padding).
__device__ __forceinline__ void tree_ancestors(const TreeParams& P, const TreeSeq& s, int t,
                                               uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0;
  int a = t;
  if (tree_parent(P, s, t) == -2) return;
  while (a >= 0) {
    const int p = tree_parent(P, s, a);
    if (p == -2) break;      // a node drafted after a padding node is a root
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] |= (a >> 5) == i ? 1u << (a & 31) : 0u;
    a = p;
  }
}

// ---------------------------------------------------------------- K/V loads
// One 128-key tile of K or V (a pool's tensor map) into shared memory:
// page_size rows of 64 columns per copy, the tile's two 64-column slabs 16 KB
// apart.  Pages past the unit's keys are not loaded.  All 32 lanes call it;
// `pages`: this lane's page (see tile_pages).
template <int D>
struct TileLoad {
  static constexpr int SLABS = D / 64;
  // pages of the tile that hold keys of the unit
  __device__ static __forceinline__ int pages(const TreeParams& P, const TreePiece& u, int tile) {
    const int keys = min(u.keys - tile * kTile, kTile);
    return keys <= 0 ? 0 : (keys + P.page_size - 1) / P.page_size;
  }
  // lane l: page index of the pool for page l / SLABS of the tile, one past
  // the pool (which TMA reads as zeros) if the table's entry is out of range
  __device__ static __forceinline__ int lane_page(const TreeParams& P, const TreePiece& u, int tile,
                                                  int lane) {
    const int j = lane / SLABS;
    if (j >= pages(P, u, tile)) return 0;
    const int pg = P.table[static_cast<int64_t>(u.b) * P.max_pages +
                           tile * (kTile / P.page_size) + j];
    if (pg >= 0 && pg < P.n_pages) return pg;
    if (P.status) atomicOr(P.status, DEV_CACHE);
    return P.n_pages;
  }
  __device__ static __forceinline__ void issue(const TreeParams& P, const TreePiece& u, int tile,
                                               int lane, int page, const CUtensorMap* tm,
                                               uint32_t dst, uint32_t bar) {
    const int n = pages(P, u, tile);
    if (lane == 0) mbar_arrive_expect_tx(bar, n * P.page_size * D * 2);
    __syncwarp();
    const int j = lane / SLABS, slab = lane % SLABS;
    if (j < n)
      tma_load_4d(dst + slab * (kTile * 128) + j * P.page_size * 128, tm, bar, slab * 64, u.hk, 0,
                  page);
  }
};

// ---------------------------------------------------------------- values that are not finite
// A row's P is 0 at a key that it does not see, but 0 times a NaN or an
// infinity of V is not 0.  Keys at or past `origin` (drafted nodes, which not
// every row sees) are therefore cleaned: their elements that are not finite
// become 0 in shared memory, a bit per key remembers it, and the epilogue
// applies them to the rows that do see the key (fix_value).  A weight of the
// softmax is positive, so the sum over visible keys has +-inf where one of
// them has, and NaN where one has NaN or both infinities meet.
__device__ __forceinline__ bool bf16x2_not_finite(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t bf16x2_clean(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}

// Row tiles of the two kernels.
constexpr int kNarrowRows = 16, kWideRows = 256;

// Adds to x what the keys flagged in nf (bit i: key origin + i) and seen
// (bit i of `seen`) hold in column c, if that is not finite.
__device__ __forceinline__ float fix_value(const TreeParams& P, const TreePiece& u,
                                           const uint32_t* nf, const uint32_t* seen, int c,
                                           float x) {
  for (int w = 0; w < 8; ++w) {
    uint32_t bits = nf[w] & seen[w];
    while (bits) {
      const int i = w * 32 + __ffs(bits) - 1;
      bits &= bits - 1;
      const int pos = u.origin + i;
      const int pg = P.table[static_cast<int64_t>(u.b) * P.max_pages + pos / P.page_size];
      if (pg < 0 || pg >= P.n_pages) continue;
      const float v = __bfloat162float(P.v_pool[pg * P.v_stride[0] +
                                                (pos % P.page_size) * P.v_stride[1] +
                                                u.hk * P.v_stride[2] + c]);
      if (!isfinite(v)) x += v;
    }
  }
  return x;
}

// fix_value over columns [c0, c1) of a row that has been written (bf16 or fp32).
template <typename T>
__device__ __noinline__ void fix_row(const TreeParams& P, const TreePiece& u, const uint32_t* nf,
                                     const uint32_t* seen, int c0, int c1, T* row) {
  for (int c = c0; c < c1; ++c) {
    const float x = static_cast<float>(row[c]);
    const float y = fix_value(P, u, nf, seen, c, x);
    if (!(x == y)) row[c] = static_cast<T>(y);
  }
}

// The kernel for units of up to 256 rows (fm_tree_wide.cu) and the join of
// either kernel's parts (fm_tree.cu).
fm_status launch_tree_wide(const TreeParams& P, int d, const CUtensorMap& tk, const CUtensorMap& tv,
                           int grid, cudaStream_t s);

}  // namespace fm
