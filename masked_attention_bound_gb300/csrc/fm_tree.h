// Attention over the paged cache: what its kernels share.
//
// Work is cut into units and tiles.  A unit is one (sequence, K/V head, row
// tile): up to R rows, row r of a sequence being node r / G of query head hk *
// G + r % G, so the G query heads that share a K/V head share its loads.  A
// unit walks the 64- or 128-key tiles [0, tiles) of its sequence up to its last
// node.  All units, in order, form one line on which a unit is as long as its
// tiles and its fixed cost (writing its rows, fetching the next one's; END
// tiles); each block takes an equal run of it, whatever the lengths, so one
// long sequence keeps every SM busy and a full batch is balanced.  Where a run ends inside a unit, each
// block leaves its unnormalised part (running max, sum, O) in the workspace
// and tree_join_kernel adds the parts in ascending order.
#pragma once
#include <cuda_bf16.h>

#include "fm_cache.h"
#include "fm_ptx.cuh"
#include "fm_tmap.h"

namespace fm {

struct TreeParams {
  int B, H, Hkv, G, total, max_nodes, page_shift, n_pages, max_pages;
  int box_shift;           // log2 of the rows of a TMA box, min(page_size, tile)
  int tree;                // 0: chain (no parents)
  int q_tma;               // the wide kernel loads Q by TMA: G divides 128
  int whole;               // units are not cut: no parts, no join
  FastDiv by_G, by_grid;
  float scale_log2;        // scale * log2(e)
  const __nv_bfloat16* q;
  int64_t q_stride[2];
  __nv_bfloat16* o;
  int64_t o_stride[2];
  float* lse;
  const __nv_bfloat16* v_pool;   // for values that are not finite (see fix_row)
  int64_t v_stride[3];           // page, slot, head
  const int32_t *table, *lens, *cu, *parents;
  int4* rec;               // [grid] what a block leaves for the join, see below
  int part_rows;           // rows that a part has room for
  float2* part_ml;         // [2 * grid][part_rows] running max (base-2 exponent) and sum
  float* part_o;           // [2 * grid][part_rows][D]
  int* status;
  uint32_t wait_ns;        // limit of every mbarrier wait
  int withhold;            // test hook: 8 = the consumers skip their first arrival, see fm_test_hooks
};

// What a block leaves for the join: the unit that it starts and does not
// finish (its part is in slot 2 * block + 1): sequence in rec.x (-1: none),
// K/V head in .y, row tile in .z; rec.w = 0, or 1: its first run finishes a
// unit that an earlier block started, 2: belongs to one and does not finish
// it (its part is in slot 2 * block).

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
  if (c0 < 0 || c1 < c0 || c1 > P.total || s.n > P.max_nodes || len < s.n ||
      len > (P.max_pages << P.page_shift)) {
    // the rows that can be written get zeros
    const int lo = min(max(c0, 0), P.total), hi = min(max(c1, 0), P.total);
    s.row0 = lo;
    s.n = max(hi - lo, 0);
    s.base = -1;
  }
  return s;
}

// What the kernels of few rows load their operands and meet by.
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Geometry of the kernels: rows of a unit, keys of a tile, a unit's fixed cost
// in tiles, and the shortest run of a block in tiles (a part of 128 rows is as
// many bytes as two 64-key tiles, written and read again).  HEADS_FIRST: the
// order of the units on the line, heads outside of sequences.
struct NarrowGeo {
  static constexpr bool HEADS_FIRST = false;
  static constexpr int R = 16, KT = 64, LEAST = 2;
  __device__ static __forceinline__ int end(int) { return 2; }
};
struct MidGeo {
  static constexpr bool HEADS_FIRST = false;
  static constexpr int R = 128, KT = 64, LEAST = 4;
  __device__ static __forceinline__ int end(int) { return 8; }
};
struct WideGeo {
  static constexpr bool HEADS_FIRST = false;
  static constexpr int R = 256, KT = 128, LEAST = 2;
  // a block with a unit's end in its run took 12000 (256 rows) to 20000
  // cycles (128 rows) longer, where a tile takes 3100 and 2800; with Q by TMA
  // 3, 4 and 5 tiles are within 3 % of each other
  __device__ static __forceinline__ int end(int rows) { return rows > 128 ? 5 : 10; }
};

struct Wide8Geo {
  static constexpr bool HEADS_FIRST = false;
  static constexpr int R = 256, KT = 64, LEAST = 4;
  // a tile takes 2200 cycles, a unit's ends some 15000; with 6, 8, 10 and 14 tiles
  // 64 nodes over 16384 tokens took 200.7, 200.8, 201.6 and 204 us, four prompts'
  // pieces of 480 tokens 93.1, 92.8, 91.7 and 93.6
  __device__ static __forceinline__ int end(int) { return 10; }
};

// Row tiles of a sequence, keys and tiles of one of them (total * H is at
// most 2^30: 32 bits hold every row).
template <class Geo>
__device__ __forceinline__ int row_tiles(const TreeParams& P, const TreeSeq& s) {
  return (s.n * P.G + Geo::R - 1) / Geo::R;
}
template <class Geo>
__device__ __forceinline__ int unit_keys(const TreeParams& P, const TreeSeq& s, int rt) {
  if (s.base < 0) return 0;
  return s.base + P.by_G(min(s.n * P.G, (rt + 1) * Geo::R) - 1) + 1;
}
template <class Geo>
__device__ __forceinline__ int key_tiles(int keys) {
  return keys > 0 ? (keys + Geo::KT - 1) / Geo::KT : 1;
}
// A unit's length on the line.  With P.whole a unit is a point of the line and
// never cut.
template <class Geo>
__device__ __forceinline__ int unit_length(const TreeParams& P, const TreeSeq& s, int rt, int tiles) {
  return P.whole ? 1 : tiles + Geo::end(s.n * P.G - rt * Geo::R);
}
// Length of all units of one K/V head of a sequence.  (The launch checks that
// the line's length fits in 31 bits.)
template <class Geo>
__device__ __forceinline__ uint32_t seq_length(const TreeParams& P, const TreeSeq& s) {
  const int nr = row_tiles<Geo>(P, s);
  uint32_t w = 0;
#pragma unroll 1
  for (int rt = 0; rt < nr; ++rt) w += unit_length<Geo>(P, s, rt, key_tiles<Geo>(unit_keys<Geo>(P, s, rt)));
  return w;
}

// The first touch of a memory page by an SM costs 2 to 3 us (address
// translation, behind the K/V stream): the small inputs and this block's
// places in the workspace are touched at once, while the block sets up.
__device__ __forceinline__ void touch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
template <int D>
__device__ __forceinline__ void touch_memory(const TreeParams& P, int lane, int block) {
  const int64_t part = 2 * static_cast<int64_t>(block) * P.part_rows;
  if (lane == 0) touch(P.lens);
  if (lane == 1) touch(P.cu);
  if (lane == 2) touch(P.table);
  if (lane == 3) touch(P.q);
  if (lane == 4 && P.tree) touch(P.parents);
  if (lane >= 5 && P.whole) return;
  if (lane == 5) touch(P.part_o + part * D);
  if (lane == 6) touch(P.part_o + (part + P.part_rows) * D);
  if (lane == 7) touch(P.part_ml + part);
}

// A block's run: the place where it starts, and its length.
struct TreeRun {
  int b, hk, rt, tile, left;
  TreeSeq s;          // sequence b
};

// Every warp of the block finds the run by itself (no shared memory and no
// barrier: the start of the kernel is on the path of every call).  Lane l
// adds up the lengths of sequences [l m, l m + m), m = ceil(B / 32); one scan
// over the lanes, and the lane whose sequences hold the run's start looks for
// it among them.
template <class Geo>
__device__ __forceinline__ TreeRun tree_run(const TreeParams& P, int block) {
  constexpr unsigned ALL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int m = (P.B + 31) >> 5;
  const int b0 = lane * m, b1 = min(b0 + m, P.B);
  TreeSeq s{0, 0, 0};
  uint32_t w = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    s = tree_seq(P, b);
    if (s.base < 0 && block == 0 && P.status) atomicOr(P.status, DEV_CACHE);
    w += seq_length<Geo>(P, s) * (Geo::HEADS_FIRST ? 1 : P.Hkv);
  }
  uint32_t inc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(ALL, inc, o);
    if (lane >= o) inc += y;
  }
  const uint32_t once = __shfl_sync(ALL, inc, 31);           // HEADS_FIRST: of one head
  const uint32_t all = Geo::HEADS_FIRST ? once * P.Hkv : once;
  TreeRun run{0, 0, 0, 0, 0, s};
  const uint32_t me = block, grid = gridDim.x, least = P.whole ? 1 : Geo::LEAST;
  uint32_t each = P.by_grid(all), more = all - each * grid;   // the first blocks take one more
  if (each < least) {                  // on a short line the last blocks have nothing
    each = least;
    more = 0;
  }
  uint32_t begin = each * me + min(me, more);
  if (begin >= all) return run;
  run.left = min(each + (me < more), all - begin);
  if (Geo::HEADS_FIRST) {
    run.hk = begin / once;
    begin -= run.hk * once;
  }
  const unsigned owner = __ballot_sync(ALL, inc > begin);
  const int from = __ffs(owner) - 1;
  if (lane == from) {
    uint32_t off = begin - (inc - w), per = 0;
    int b = b0;
#pragma unroll 1
    for (;; ++b) {
      if (m > 1) s = tree_seq(P, b);
      per = seq_length<Geo>(P, s);
      const uint32_t span = Geo::HEADS_FIRST ? per : per * P.Hkv;
      if (off < span) break;
      off -= span;
    }
    run.b = b;
    if (!Geo::HEADS_FIRST) {
      run.hk = off / per;
      off -= run.hk * per;
    }
#pragma unroll 1
    while (true) {
      const uint32_t t = unit_length<Geo>(P, s, run.rt, key_tiles<Geo>(unit_keys<Geo>(P, s, run.rt)));
      if (off < t) break;
      off -= t;
      ++run.rt;
    }
    run.tile = off;
  }
  run.b = __shfl_sync(ALL, run.b, from);
  run.hk = __shfl_sync(ALL, run.hk, from);
  run.rt = __shfl_sync(ALL, run.rt, from);
  run.tile = __shfl_sync(ALL, run.tile, from);
  run.s.row0 = __shfl_sync(ALL, s.row0, from);
  run.s.n = __shfl_sync(ALL, s.n, from);
  run.s.base = __shfl_sync(ALL, s.base, from);
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

// Every role of a block walks its run piece by piece in the same order.  The
// walk is the piece: each field is held once.
template <class Geo>
struct TreeWalk : TreePiece {
  int left;            // of the run, in units of the line
  int next_tile;       // where the next piece starts; -1: at the next unit
  __device__ __forceinline__ explicit TreeWalk(const TreeRun& run) {
    b = run.b;
    hk = run.hk;
    rt = run.rt;
    s = run.s;
    left = run.left;
    next_tile = run.tile;
  }
  __device__ __forceinline__ bool next(const TreeParams& P) {
#pragma unroll 1
    while (true) {
      if (left <= 0) return false;
      if (next_tile < 0) {
        next_tile = 0;
        if (++rt >= row_tiles<Geo>(P, s)) {
          rt = 0;
          if (Geo::HEADS_FIRST) s.n = 0;         // on to the next sequence
          else ++hk;
        }
      }
      // on to the next sequence with rows
      if (Geo::HEADS_FIRST) {
        if (s.n <= 0) {
          rt = next_tile = 0;
          if (++b >= P.B) {
            b = 0;
            if (++hk >= P.Hkv) return false;
          }
          s = tree_seq(P, b);
          continue;
        }
      } else if (hk >= P.Hkv || s.n <= 0) {
        hk = rt = next_tile = 0;
        if (++b >= P.B) return false;
        s = tree_seq(P, b);
        continue;
      }
      keys = unit_keys<Geo>(P, s, rt);
      tiles = key_tiles<Geo>(keys);
      t0 = next_tile;
      t1 = P.whole ? tiles : min(tiles, t0 + left);
      const bool ends = t1 >= tiles;
      left -= (ends ? unit_length<Geo>(P, s, rt, tiles) : t1) - t0;
      next_tile = ends ? -1 : t1;
      if (t0 < tiles) break;           // else the run starts in a unit's fixed cost
    }
    row_first = rt * Geo::R;
    rows = min(Geo::R, s.n * P.G - row_first);
    origin = s.base + (P.tree ? 0 : P.by_G(row_first));
    return true;
  }
};

// A piece's share of the block's record (its first thread's; the block starts
// with {-1, 0, 0, 0}).
__device__ __forceinline__ void leave_record(const TreeParams& P, const TreePiece& u, int block) {
  if (u.whole()) return;
  int* rec = reinterpret_cast<int*>(P.rec + block);
  if (u.t0 == 0) {
    rec[0] = u.b;
    rec[1] = u.hk;
    rec[2] = u.rt;
  } else {
    rec[3] = u.t1 == u.tiles ? 1 : 2;
  }
}

// Parent of node t of sequence s as the kernels use it: -1 a root, -2 padding.
__device__ __forceinline__ int tree_parent(const TreeParams& P, const TreeSeq& s, int t) {
  const int p = P.parents[s.row0 + t];
  if (p >= -2 && p < t) return p;
  if (P.status) atomicOr(P.status, DEV_CACHE);
  return -1;
}

// Ancestors of node t and itself as bits [0, 256) of w (all 0 for padding);
// parent(a): tree_parent of node a.
template <typename F>
__device__ __forceinline__ void tree_ancestors(int t, F parent, uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0;
#pragma unroll 1
  for (int a = t; a >= 0;) {
    const int p = parent(a);
    if (p == -2) break;      // a node drafted after a padding node is a root
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] |= (a >> 5) == i ? 1u << (a & 31) : 0u;
    a = p;
  }
}

// ---------------------------------------------------------------- waits
// Code that a block runs once costs its instruction fetches, which queue
// behind the K/V stream in L2: the first version of the wide kernel (149 KB,
// rare paths unrolled everywhere) spent 21000 cycles on its first masked tile
// and 10000 on writing O.  So the rare paths are kept small: short waits,
// loops that are not unrolled.
__device__ __forceinline__ uint32_t globaltimer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
// mbar_wait with the limit in 32 bits; false (with the status and the abort
// flag set) when it runs out, or when another warp's did.
__device__ __forceinline__ bool tree_wait(uint32_t bar, uint32_t parity, const TreeParams& P,
                                          volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = globaltimer_lo();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (globaltimer_lo() - t0 > P.wait_ns) {
      if (P.status) atomicOr(P.status, DEV_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// ---------------------------------------------------------------- K/V loads
// One KT-key tile of K or V (a pool's tensor map) into shared memory: boxes of
// min(page_size, KT) rows of 64 columns, the tile's two 64-column slabs KT *
// 128 bytes apart.  Boxes past the unit's keys are not loaded.  All 32 lanes
// call it; `page`: this lane's (lane_page); `policy`: evict first, since a
// stream of K and V through L2 would push out what the next piece needs, the
// kernel's own instructions among it (a fetch from DRAM behind the stream took
// 5000 cycles).
template <int D, int KT>
struct TileLoad {
  static constexpr int SLABS = D / 64;
  // boxes of the tile that hold keys of the unit
  __device__ static __forceinline__ int boxes(const TreeParams& P, const TreePiece& u, int tile) {
    const int keys = min(u.keys - tile * KT, KT);
    return keys <= 0 ? 0 : (keys + (1 << P.box_shift) - 1) >> P.box_shift;
  }
  // lane l: page of the pool that holds box l / SLABS of the tile, one past
  // the pool (which TMA reads as zeros) if the table's entry is out of range
  __device__ static __forceinline__ int lane_page(const TreeParams& P, const TreePiece& u, int tile,
                                                  int lane) {
    const int j = lane / SLABS;
    if (j >= boxes(P, u, tile)) return 0;
    const int pg = P.table[static_cast<int64_t>(u.b) * P.max_pages +
                           ((tile * KT + (j << P.box_shift)) >> P.page_shift)];
    if (pg >= 0 && pg < P.n_pages) return pg;
    if (P.status) atomicOr(P.status, DEV_CACHE);
    return P.n_pages;
  }
  __device__ static __forceinline__ void issue(const TreeParams& P, const TreePiece& u, int tile,
                                               int lane, int page, const CUtensorMap* tm,
                                               uint32_t dst, uint32_t bar, uint64_t policy) {
    const int n = boxes(P, u, tile);
    if (lane == 0) mbar_arrive_expect_tx(bar, (n << P.box_shift) * D * 2);
    __syncwarp();
    const int j = lane / SLABS, slab = lane % SLABS;
    if (j < n)
      tma_load_4d_hint(dst + slab * (KT * 128) + (j << P.box_shift) * 128, tm, bar, slab * 64, u.hk,
                       (tile * KT + (j << P.box_shift)) & ((1 << P.page_shift) - 1), page, policy);
  }
};

// ---------------------------------------------------------------- values that are not finite
// A row's P is 0 at a key that it does not see, but 0 times a NaN or an
// infinity of V is not 0.  Keys at or past `origin` (drafted nodes, which not
// every row sees) are therefore cleaned: their elements that are not finite
// become 0 in shared memory, a bit per key remembers it, and the epilogue
// applies them to the rows that do see the key (fix_row).  A weight of the
// softmax is positive, so the sum over visible keys has +-inf where one of
// them has, and NaN where one has NaN or both infinities meet.
__device__ __forceinline__ bool bf16x2_not_finite(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
// x * 0 + sum of both halves.
__device__ __forceinline__ uint32_t bf16x2_times_zero(uint32_t x, uint32_t sum) {
  uint32_t y;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(0u), "r"(sum));
  return y;
}
__device__ __forceinline__ uint32_t bf16x2_clean(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}

// Adds to elements [0, n) of a row that has been written (bf16 or fp32, row[i]
// is column c0 + i) what the keys flagged in nf (bit i: key origin + i) and
// seen (bit i of s0, s1) hold there, where that is not finite.  Arguments by
// value: what has its address taken lives in local memory, and the little L1
// that shared memory leaves does not hold it.
template <typename T>
static __device__ __noinline__ void fix_row(const TreeParams& P, int b, int hk, int origin,
                                            const uint32_t* nf, uint4 s0, uint4 s1, int c0, int n,
                                            T* row) {
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const float x = static_cast<float>(row[i]);
    float y = x;
#pragma unroll 1
    for (int w = 0; w < 8; ++w) {
      const uint4 s = w < 4 ? s0 : s1;
      const uint32_t seen = (w & 3) == 0 ? s.x : (w & 3) == 1 ? s.y : (w & 3) == 2 ? s.z : s.w;
      uint32_t bits = nf[w] & seen;
#pragma unroll 1
      while (bits) {
        const int pos = origin + w * 32 + __ffs(bits) - 1;
        bits &= bits - 1;
        const int pg = P.table[static_cast<int64_t>(b) * P.max_pages + (pos >> P.page_shift)];
        if (pg < 0 || pg >= P.n_pages) continue;
        const float v = __bfloat162float(P.v_pool[pg * P.v_stride[0] +
                                                  (pos & ((1 << P.page_shift) - 1)) * P.v_stride[1] +
                                                  hk * P.v_stride[2] + c0 + i]);
        if (!isfinite(v)) y += v;
      }
    }
    if (!(x == y)) row[i] = static_cast<T>(y);
  }
}

// The kernels for units of up to 128 and 256 rows (fm_tree_wide.cu); the one
// for up to 16 rows and the join of their parts are in fm_tree.cu.
fm_status launch_tree_mid(const TreeParams& P, int d, const CUtensorMap& tq, const CUtensorMap& tk,
                          const CUtensorMap& tv, int grid, cudaStream_t s);
fm_status launch_tree_wide(const TreeParams& P, const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& tv, int grid, cudaStream_t s);   // d = 128

}  // namespace fm
